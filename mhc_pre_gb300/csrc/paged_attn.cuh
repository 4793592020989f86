// paged_attn.cuh -- what the paged-attention kernels share: the plan that
// splits a ragged batch evenly over the CTAs, the masks, and the joining of
// partial results.
//
// Work.  For each sequence and key head, the query heads that share the key
// head and the sequence's new tokens form one list of rows (row r is token
// r / G, head r % G of the group, G = Hq/Hk); a tile is up to `tile_rows`
// consecutive rows, and it reads the keys that any of its rows sees in blocks
// of `block_keys`.  The unit of work is one block of one tile of one key head.
// All units are laid end to end (tiles, then key heads, then blocks) and CTA c
// takes the `per_cta` consecutive units from c * per_cta: every CTA has the
// same share whatever the lengths are, a long sequence is split over as many
// CTAs as it needs, and at most two of a CTA's pieces (its first and its last)
// are incomplete.  Incomplete pieces go to the workspace as unnormalised sums
// with their row maxima, and the CTA that finishes a tile last joins them in
// the order of the CTAs, so that results do not depend on timing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_common.cuh"

namespace mhc {

constexpr unsigned ATTN_ERR_TIMEOUT = 1u, ATTN_ERR_RANGE = 2u;

// One tile of rows of one sequence, for every key head.
struct AttnTile {
    int64_t start;      // its first unit
    int64_t q0;         // the sequence's first row of q
    int seq;
    int qlen, kvlen;    // new tokens; cached tokens including them
    int row0;           // first row of the tile in the sequence's list
    int blk0, nblk;     // key blocks that any of its rows sees
    int cnt;            // index of its join counters (one per key head)
    int pad;
};
static_assert(sizeof(AttnTile) == 48, "AttnTile is read as three 16-byte words");

struct AttnHead {       // start of the plan
    int64_t units;      // all units
    int64_t per_cta;    // units of a CTA
    int64_t T;          // rows of q, for the check that plan and call agree
    int ntiles;
    int ncta;
    int Hq, Hk, B, tile_rows, block_keys, window;
};
static_assert(sizeof(AttnHead) <= 64, "the header has 64 bytes");

// Sizes both the host and the device need.
struct AttnPlan {
    int ncta;           // CTAs of the launch
    int tile_rows, block_keys;
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
    int64_t T;
    int B, Hq, Hk, G, Dh, page_size, page_shift, window;
    float scale, softcap;
    unsigned force_timeout;
    AttnPlan plan;
};

// Where a CTA starts: tile, key head and block.
struct AttnStart {
    int tile, head, blk, pad;
};

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

// Whether the plan in the workspace is the one that this call's sizes ask for.
__device__ __forceinline__ bool attn_plan_agrees(const AttnParams& p) {
    const AttnHead* h = attn_head(p);
    return h->T == p.T && h->Hq == p.Hq && h->Hk == p.Hk && h->B == p.B && h->tile_rows == p.plan.tile_rows &&
           h->block_keys == p.plan.block_keys && h->window == p.window && h->ncta == p.plan.ncta &&
           h->ntiles >= 0 && h->ntiles <= p.plan.max_tiles && h->per_cta > 0;
}

// A CTA's pieces one after the other.
struct AttnPiece {
    AttnTile t;
    int tile, head;
    int b0, b1;          // blocks [b0, b1) of the tile, relative to its first
    bool whole;          // the tile's only piece
    int slot;            // where a partial result goes
    int first_cta, last_cta;
};
struct AttnWalk {
    int64_t at, end;
    int tile, head, blk;
    __device__ __forceinline__ bool begin(const AttnParams& p, int cta) {
        const AttnHead* h = attn_head(p);
        const int64_t per = h->per_cta;
        at = static_cast<int64_t>(cta) * per;
        end = min(at + per, h->units);
        if (at >= end) return false;
        const AttnStart s = attn_starts(p)[cta];
        tile = s.tile;
        head = s.head;
        blk = s.blk;
        return true;
    }
    __device__ __forceinline__ bool next(const AttnParams& p, int cta, int64_t per, AttnPiece& out) {
        if (at >= end) return false;
        const int4* src = reinterpret_cast<const int4*>(attn_tiles(p) + tile);
        int4* dst = reinterpret_cast<int4*>(&out.t);
        dst[0] = src[0];
        dst[1] = src[1];
        dst[2] = src[2];
        out.tile = tile;
        out.head = head;
        out.b0 = blk;
        const int64_t left = end - at;
        const int n = left < out.t.nblk - blk ? static_cast<int>(left) : out.t.nblk - blk;
        out.b1 = blk + n;
        out.whole = out.b0 == 0 && out.b1 == out.t.nblk;
        out.slot = 2 * cta + (out.b0 > 0 ? 0 : 1);
        const int64_t u0 = out.t.start + static_cast<int64_t>(head) * out.t.nblk;
        out.first_cta = static_cast<int>(u0 / per);
        out.last_cta = static_cast<int>((u0 + out.t.nblk - 1) / per);
        at += n;
        blk += n;
        if (blk == out.t.nblk) {
            blk = 0;
            if (++head == p.Hk) {
                head = 0;
                ++tile;
            }
        }
        return true;
    }
};

// Keys [lo, hi) that row r of a tile's sequence sees.
__device__ __forceinline__ void attn_row_keys(const AttnTile& t, int r, int G, int window, int& lo, int& hi) {
    const int pos = t.kvlen - t.qlen + r / G;
    hi = max(0, min(t.kvlen, pos + 1));
    lo = window > 0 ? max(0, pos - window + 1) : 0;
}

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
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// One row's log sum exp from its maximum in base 2 and its sum.
__device__ __forceinline__ float attn_lse(float m2, float l) {
    return l != 0.0f ? fmaf(m2, LN2, logf(l)) : -INFINITY;
}

// Joins the partial results of a tile (nthr threads, all of them after a
// barrier that follows the last arrival): item i is 4 values of one row.
template <typename TA>
__device__ __forceinline__ void attn_join(const AttnParams& p, const AttnPiece& pc, int dp, int tid, int nthr) {
    const int rows_left = pc.t.qlen * p.G - pc.t.row0;
    const int rows = min(rows_left, p.plan.tile_rows);
    const int d4 = p.Dh / 4, sr = p.plan.slot_rows;
    for (int i = tid; i < rows * d4; i += nthr) {
        const int row = i / d4, d = (i - row * d4) * 4;
        float M = -INFINITY;
        for (int c = pc.first_cta; c <= pc.last_cta; ++c) {
            const float* s = attn_slot(p, 2 * c + (c == pc.first_cta ? 1 : 0));
            M = fmaxf(M, __ldcg(s + static_cast<int64_t>(sr) * dp + row));
        }
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float l = 0.0f;
        if (M > -INFINITY) {
            for (int c = pc.first_cta; c <= pc.last_cta; ++c) {
                const float* s = attn_slot(p, 2 * c + (c == pc.first_cta ? 1 : 0));
                const float w = ex2(__ldcg(s + static_cast<int64_t>(sr) * dp + row) - M);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(s + static_cast<int64_t>(row) * dp + d));
                l = fmaf(w, __ldcg(s + static_cast<int64_t>(sr) * (dp + 1) + row), l);
                a.x = fmaf(w, v.x, a.x);
                a.y = fmaf(w, v.y, a.y);
                a.z = fmaf(w, v.z, a.z);
                a.w = fmaf(w, v.w, a.w);
            }
        }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int r = pc.t.row0 + row;
        const int64_t out = (pc.t.q0 + r / p.G) * p.Hq + pc.head * p.G + r % p.G;
        TA* o = static_cast<TA*>(p.o) + out * p.Dh + d;
        if (sizeof(TA) == 2) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv);
            const __nv_bfloat162 y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
            *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                                      *reinterpret_cast<const uint32_t*>(&y));
        } else {
            *reinterpret_cast<float4*>(o) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        }
        if (d == 0 && p.lse != nullptr) p.lse[out] = attn_lse(M, l);
    }
}

}  // namespace mhc
