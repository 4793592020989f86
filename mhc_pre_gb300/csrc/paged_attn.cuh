// paged_attn.cuh -- what the paged-attention kernels share: the plan that
// splits a ragged batch evenly over the CTAs, the masks, and the joining of
// partial results.
//
// Work.  For each sequence and key head, the query heads that share the key
// head and the sequence's new tokens form one list of rows (row r is token
// r / G, head r % G of the group, G = Hq/Hk); a tile is up to `tile_rows`
// consecutive rows, and it reads the keys that any of its rows sees in blocks
// of `block_keys`.  The unit of work is one block of one tile of one key head.
// A tile of a key head begins with `lead` units that stand for its fixed costs
// (queries in, sums out), so that many short tiles weigh what they take.
// All units are laid end to end (tiles, then key heads, then blocks) and CTA c
// takes the `per_cta` consecutive units from c * per_cta: every CTA has the
// same share whatever the lengths are, a long sequence is split over as many
// CTAs as it needs, and at most two of a CTA's pieces (its first and its last)
// are incomplete.  A tile of a key head that costs at most 1/8 of a share is
// not split: the border moves to its nearer end, which unbalances the shares
// by less than joining its parts would take (14 tiles of 7 units a CTA: 216 ->
// 203 us).  Incomplete pieces go to the workspace as unnormalised sums
// with their row maxima, and the CTA that finishes a tile last joins them in
// the order of the CTAs, so that results do not depend on timing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_common.cuh"

namespace mhc {

constexpr unsigned ATTN_ERR_TIMEOUT = 1u, ATTN_ERR_RANGE = 2u;

// Join counters of a tile and key head: each warp's rows are joined by
// themselves.
constexpr int JOINS = 8;

// One tile of rows of one sequence, for every key head.
struct alignas(16) AttnTile {
    int64_t start;      // its first unit
    int64_t q0;         // the sequence's first row of q
    int seq;
    int qlen, kvlen;    // new tokens; cached tokens including them
    int row0;           // first row of the tile in the sequence's list
    int blk0, nblk;     // key blocks that any of its rows sees
    int cnt;            // index of its join counters (JOINS per key head)
    int pad;
};
static_assert(sizeof(AttnTile) == 48, "AttnTile is read as three 16-byte words");

struct AttnHead {       // start of the plan
    int64_t per_cta;    // units of a CTA
    int64_t T;          // this and the sizes below: for the check that plan and call agree
    int64_t max_q, max_kv;
    int ntiles;
    int ncta;
    int Hq, Hk, B, tile_rows, block_keys, window, lead;
    int spent;          // a wait ran out in a call with this plan: parts of its tiles never
                        // came, and their join counters stand where the next call would
                        // take them for its own
};
static_assert(sizeof(AttnHead) <= 256, "the header has 256 bytes");

// Sizes both the host and the device need.
struct AttnPlan {
    int ncta;           // CTAs of the launch
    int tile_rows, block_keys;
    int lane_rows;      // rows of one softmax lane (tensor cores): whole tokens
    int lead;           // fixed cost of a tile, in blocks
    int slot_rows;      // rows a partial result can have
    int64_t max_tiles;
    size_t start_off, tile_off, count_off, part_off, part_slot_bytes, total;
};

struct AttnParams {
    const void *q, *k_cache, *v_cache;
    void* o;
    float* lse;                    // may be null
    const int32_t* page_table;     // [B, table_stride]
    unsigned char* ws;
    int64_t q_stride, table_stride, num_pages;
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int64_t T, max_q, max_kv;
    int B, Hq, Hk, G, Dh, page_size, page_shift, window;
    unsigned g_mul, g_shift;       // r / G = umulhi(r, g_mul) >> g_shift for 0 <= r < 2^31
    float scale, softcap;
    unsigned force_timeout;
    AttnPlan plan;
};

// A CTA's share: its units, tile, key head and unit of the tile, and the tile itself
// (one read instead of two on the way to the first queries and keys).
struct alignas(16) AttnStart {
    int64_t begin, end;     // the CTA's units
    int tile, head, unit, pad;
    AttnTile t;
};
static_assert(sizeof(AttnStart) == 80, "AttnStart is read as five 16-byte words");

__device__ __forceinline__ const AttnHead* attn_head(const AttnParams& p) {
    return reinterpret_cast<const AttnHead*>(p.ws);
}
__device__ __forceinline__ const AttnStart* attn_starts(const AttnParams& p) {
    return reinterpret_cast<const AttnStart*>(p.ws + p.plan.start_off);
}
__device__ __forceinline__ const AttnTile* attn_tiles(const AttnParams& p) {
    return reinterpret_cast<const AttnTile*>(p.ws + p.plan.tile_off);
}
__device__ __forceinline__ int* attn_counts(const AttnParams& p) {
    return reinterpret_cast<int*>(p.ws + p.plan.count_off);
}

// Whether the plan in the workspace is the one that this call's sizes ask for (a
// larger max_q would overrun the parts, a larger max_kv the page table) and its
// counters are at zero.
__device__ __forceinline__ bool attn_plan_agrees(const AttnParams& p) {
    const AttnHead* h = attn_head(p);
    return h->T == p.T && h->max_q == p.max_q && h->max_kv == p.max_kv && h->Hq == p.Hq && h->Hk == p.Hk &&
           h->B == p.B && h->tile_rows == p.plan.tile_rows && h->block_keys == p.plan.block_keys &&
           h->window == p.window && h->ncta == p.plan.ncta && h->lead == p.plan.lead && h->ntiles >= 0 &&
           h->ntiles <= p.plan.max_tiles && h->per_cta > 0 && h->spent == 0;
}
__device__ __forceinline__ void attn_plan_spent(const AttnParams& p) { reinterpret_cast<AttnHead*>(p.ws)->spent = 1; }

// The token of row r.
__device__ __forceinline__ int attn_token(const AttnParams& p, int r) {
    return p.G == 1 ? r : static_cast<int>(__umulhi(static_cast<unsigned>(r), p.g_mul) >> p.g_shift);
}

// Keys [lo, hi) that token i of the sequence's new ones sees.  A token before the
// cached ones has end = 0: end - window stays in 32 bits for every window.
template <typename T>
__device__ __forceinline__ void attn_token_keys(const T& t, int i, int window, int& lo, int& hi) {
    const int end = max(0, t.kvlen - t.qlen + i + 1);
    hi = min(t.kvlen, end);
    lo = window > 0 ? max(0, end - window) : 0;
}

// A CTA's pieces one after the other.
struct AttnPiece {
    int64_t q0;
    int seq, qlen, kvlen, row0, head;
    int blk, nb;                // first key block and number of blocks (0: there is no piece)
    int whole;                  // the tile's only piece
    int cnt, slot;              // join counters; where a partial result goes
    int first_cta, last_cta;    // the CTAs with a part of the tile (unless whole)
    int lo, hi;                 // keys [lo, hi) that any row of the tile sees
};
struct AttnWalk {
    int64_t at, end, per;
    int tile, head, unit;
    AttnTile t;
    __device__ __forceinline__ bool begin(const AttnParams& p, int cta) {
        const AttnHead* h = attn_head(p);
        const AttnStart s = attn_starts(p)[cta];
        per = h->per_cta;
        at = s.begin;
        end = s.end;
        tile = s.tile;
        head = s.head;
        unit = s.unit;
        t = s.t;
        return at < end;
    }
    // The next piece that has blocks; false when the CTA's share is done.
    __device__ __forceinline__ bool next(const AttnParams& p, int cta, AttnPiece& out) {
        while (at < end) {
            const int lead = p.plan.lead, cost = t.nblk + lead;
            const int64_t left = end - at;
            const int n = left < cost - unit ? static_cast<int>(left) : cost - unit;
            const int b0 = max(0, unit - lead), b1 = max(0, unit + n - lead);
            out.q0 = t.q0;
            out.seq = t.seq;
            out.qlen = t.qlen;
            out.kvlen = t.kvlen;
            out.row0 = t.row0;
            out.head = head;
            out.blk = t.blk0 + b0;
            out.nb = b1 - b0;
            out.whole = b0 == 0 && b1 == t.nblk;
            int unused;
            attn_token_keys(t, attn_token(p, t.row0), p.window, out.lo, unused);
            attn_token_keys(t, attn_token(p, min(t.row0 + p.plan.tile_rows, t.qlen * p.G) - 1), p.window, unused, out.hi);
            out.cnt = (t.cnt + head) * JOINS;
            out.slot = 2 * cta + (b0 > 0 ? 0 : 1);
            if (!out.whole) {
                const int64_t u0 = t.start + static_cast<int64_t>(head) * cost + lead, u1 = u0 + t.nblk - 1;
                if (u1 >> 31 == 0) {   // the 64-bit division is a long subroutine
                    out.first_cta = static_cast<int>(static_cast<uint32_t>(u0) / static_cast<uint32_t>(per));
                    out.last_cta = static_cast<int>(static_cast<uint32_t>(u1) / static_cast<uint32_t>(per));
                } else {
                    out.first_cta = static_cast<int>(u0 / per);
                    out.last_cta = static_cast<int>(u1 / per);
                }
            }
            at += n;
            unit += n;
            if (unit == cost) {
                unit = 0;
                if (++head == p.Hk) {
                    head = 0;
                    ++tile;
                    if (at < end) t = attn_tiles(p)[tile];
                }
            }
            if (b1 > b0) return true;
        }
        out.nb = 0;
        return false;
    }
};

// Partial result of one piece: rows of `dp` sums, then the maxima (in the
// scores' own unit times log2 e), then the sums of the exponentials.
__device__ __forceinline__ float* attn_slot(const AttnParams& p, int slot) {
    return reinterpret_cast<float*>(p.ws + p.plan.part_off + static_cast<size_t>(slot) * p.plan.part_slot_bytes);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// One row's log sum exp from its maximum in base 2 and its sum.
__device__ __forceinline__ float attn_lse(float m2, float l) {
    return l != 0.0f ? fmaf(m2, LN2, logf(l)) : -INFINITY;
}

// Joins the partial results of rows [begin, end) of a tile (one warp, after the
// last part has arrived), R rows at a time.  Lane c first takes the maximum and
// the sum of part c for each row, so that the parts' weights come from one round
// of loads; then the lanes take 4 values of a row each and add the parts in
// order, the loads of U parts in flight together.  More than 32 parts go in
// rounds of 32 with a running maximum.
template <typename TA, int DP, int R, int U>
__device__ __forceinline__ void attn_join(const AttnParams& p, const AttnPiece& pc, int begin, int end, int lane) {
    constexpr int LPR = DP < 128 ? DP / 4 : 32;   // lanes of a row
    constexpr int NV = DP / 4 / LPR;              // pieces of 4 values a lane has of a row
    constexpr int RW = 32 / LPR;                  // rows side by side
    const int sub = lane % LPR, side = lane / LPR, sr = p.plan.slot_rows;
    auto part = [&](int c) { return attn_slot(p, 2 * c + (c == pc.first_cta ? 1 : 0)); };
    for (int r0 = begin; r0 < end; r0 += RW * R) {
        float M[RW * R], l[RW * R];
        float4 a[R][NV];
#pragma unroll
        for (int i = 0; i < RW * R; ++i) {
            M[i] = -INFINITY;
            l[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int v = 0; v < NV; ++v) a[i][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c0 = pc.first_cta; c0 <= pc.last_cta; c0 += 32) {
            const int n = min(32, pc.last_cta - c0 + 1);
            float w[RW * R], pl[RW * R];
#pragma unroll
            for (int i = 0; i < RW * R; ++i) {
                const float* s = part(c0 + min(lane, n - 1)) + static_cast<int64_t>(sr) * DP + min(r0 + i, end - 1);
                w[i] = lane < n ? __ldcg(s) : -INFINITY;
                pl[i] = lane < n ? __ldcg(s + sr) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < RW * R; ++i) {
                float top = w[i];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = fmaxf(top, M[i]);
                const float base = top == -INFINITY ? 0.0f : top, keep = ex2(M[i] - base);
                w[i] = ex2(w[i] - base);
                l[i] = fmaf(l[i], keep, warp_sum(pl[i] * w[i]));
                if (c0 > pc.first_cta) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (i % RW == side) {
                            float4& x = a[i / RW][v];
                            x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
                        }
                }
                M[i] = top;
            }
            for (int c = 0; c < n; c += U) {
                float4 pv[U][R][NV];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float* s = part(c0 + min(c + u, n - 1));
                        const int row = min(r0 + i * RW + side, end - 1);
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            pv[u][i][v] = __ldcg(reinterpret_cast<const float4*>(s + static_cast<int64_t>(row) * DP) +
                                                 v * LPR + sub);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        float f = 0.0f;
#pragma unroll
                        for (int q = 0; q < RW; ++q) {
                            const float x = __shfl_sync(0xffffffffu, w[i * RW + q], min(c + u, 31));
                            if (q == side) f = x;
                        }
                        if (c + u < n) {
#pragma unroll
                            for (int v = 0; v < NV; ++v) {
                                a[i][v].x = fmaf(pv[u][i][v].x, f, a[i][v].x);
                                a[i][v].y = fmaf(pv[u][i][v].y, f, a[i][v].y);
                                a[i][v].z = fmaf(pv[u][i][v].z, f, a[i][v].z);
                                a[i][v].w = fmaf(pv[u][i][v].w, f, a[i][v].w);
                            }
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = r0 + i * RW + side;
            if (row >= end) continue;
            float ml = M[i * RW], ll = l[i * RW];
#pragma unroll
            for (int q = 1; q < RW; ++q)
                if (q == side) {
                    ml = M[i * RW + q];
                    ll = l[i * RW + q];
                }
            const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
            const int r = pc.row0 + row, tok = attn_token(p, r);
            const int64_t out = (pc.q0 + tok) * p.Hq + pc.head * p.G + (r - tok * p.G);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int d = (v * LPR + sub) * 4;
                if (d >= p.Dh) continue;
                TA* o = static_cast<TA*>(p.o) + out * p.Dh + d;
                if (sizeof(TA) == 2) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(a[i][v].x * inv, a[i][v].y * inv);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(a[i][v].z * inv, a[i][v].w * inv);
                    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                                              *reinterpret_cast<const uint32_t*>(&y));
                } else {
                    *reinterpret_cast<float4*>(o) = make_float4(a[i][v].x * inv, a[i][v].y * inv, a[i][v].z * inv,
                                                                a[i][v].w * inv);
                }
            }
            if (sub == 0 && p.lse != nullptr) p.lse[out] = attn_lse(ml, ll);
        }
    }
}

}  // namespace mhc
