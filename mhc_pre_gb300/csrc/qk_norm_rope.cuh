// qk_norm_rope.cuh -- per-head RMSNorm of queries and keys with the position
// rotation in the same pass: what the forward, its cache-writing form
// (qk_norm_rope.cu), the backward (qk_norm_rope_bwd.cu) and the rotation without the
// norm (qk_norm_rope_bare.cu) share.
//
// For each head x in R^Dh of token t at position p, with weight w and angles
// (c, s) = (cos, sin)[p]:
//   r = 1/sqrt(mean(x^2) + eps),  z = r w x,  y = R z
//   R turns the pairs (a, b) of the first `rot` values: (a c - b s, b c + a s)
// so with the token's coefficients held in registers for all of its heads
//   y_a = r (a (w_a c) - b (w_b s)),   y_b = r (b (w_b c) + a (w_a s)).
// Backward of <g, y>: h = R^T g, u = w h,
//   dx = r u - x r^3 <u, x> / Dh,   dw = sum over heads of r h x.
//
// A head is the work of Dh/8 lanes (rounded up to a power of two, so that its
// sums are shuffles).  A lane holds four whole pairs, whatever the pairing, so
// nothing else is exchanged; values past `rot` are pairs with c = 1, s = 0.
// Arithmetic goes through packed pairs of float32.
//
// Every value is read once and written once at a few operations each: the
// floor is memory.  Many tokens: a team of warps keeps the rows of several
// tokens in flight to shared memory (bulk copies, one barrier per stage), so
// the bytes in flight do not depend on registers or on how many warps there
// are.  Few tokens: each group of lanes loads its head directly, one round
// trip, with a token's heads spread over blocks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "mhc_common.cuh"
#include "tc_ptx.cuh"

namespace mhc {

// Each translation unit has its own word: bit 0, a wait ran out; bit 1, a
// position or slot outside its range.
static __device__ unsigned g_qk_error;

namespace qk {

constexpr int THREADS = 128;
// Staged blocks of an SM (the kernels are compiled for that many).  Forward, at
// T = 32768 and 48 heads of 128: 4, 5 and 6 take 149, 145 and 150 us.
constexpr int FWD_BLOCKS = 5, BWD_BLOCKS = 4;
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;

// ------------------------------------------------------------- four pairs ---
// The a's and b's of a lane's four pairs, as (0, 1) and (2, 3).
struct Pairs {
    float2 a[2], b[2];
};

// Where a lane's pairs are in a head: two runs of four elements.
struct Lane {
    int sub;          // lane of the group
    int lo, hi;       // first elements of the runs
    int angle;        // first angle index, -1: these pairs do not turn
    bool on;          // the lane has pairs
};
template <int LPH, bool ADJ>
__device__ __forceinline__ Lane make_lane(int lane, int Dh, int rot) {
    Lane L;
    L.sub = lane & (LPH - 1);
    L.on = L.sub * 8 < Dh;
    const int j = L.sub * 4;   // pair index
    const bool turns = j < rot / 2;
    L.angle = turns ? j : -1;
    if (ADJ) {
        L.lo = L.sub * 8;
        L.hi = L.lo + 4;
    } else if (turns) {
        L.lo = j;
        L.hi = j + rot / 2;
    } else {
        L.lo = rot + j - rot / 2;
        L.hi = L.lo + (Dh - rot) / 2;
    }
    return L;
}

// Four consecutive elements in their storage type.
template <typename TA> struct Four;
template <> struct Four<__nv_bfloat16> {
    using T = uint2;
    __device__ __forceinline__ static T zero() { return make_uint2(0u, 0u); }
    __device__ __forceinline__ static void get(const T& u, float2& x, float2& y) {
        x = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
        y = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    }
    __device__ __forceinline__ static T put(const float2& x, const float2& y) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(y.x, y.y);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};
template <> struct Four<float> {
    using T = float4;
    __device__ __forceinline__ static T zero() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ static void get(const T& u, float2& x, float2& y) {
        x = make_float2(u.x, u.y);
        y = make_float2(u.z, u.w);
    }
    __device__ __forceinline__ static T put(const float2& x, const float2& y) {
        return make_float4(x.x, x.y, y.x, y.y);
    }
};

// A lane's pairs of one head as loaded.
template <typename TA> struct Raw {
    typename Four<TA>::T lo, hi;
    __device__ __forceinline__ void zero() { lo = hi = Four<TA>::zero(); }
    __device__ __forceinline__ void load(const TA* head, const Lane& L) {
        lo = *reinterpret_cast<const typename Four<TA>::T*>(head + L.lo);
        hi = *reinterpret_cast<const typename Four<TA>::T*>(head + L.hi);
    }
    __device__ __forceinline__ void stream(const TA* head, const Lane& L) {   // read once
        lo = __ldcs(reinterpret_cast<const typename Four<TA>::T*>(head + L.lo));
        hi = __ldcs(reinterpret_cast<const typename Four<TA>::T*>(head + L.hi));
    }
    __device__ __forceinline__ void store(TA* head, const Lane& L) const {
        *reinterpret_cast<typename Four<TA>::T*>(head + L.lo) = lo;
        *reinterpret_cast<typename Four<TA>::T*>(head + L.hi) = hi;
    }
};

// Two runs of four values to pairs and back.  Adjacent pairing: the runs are
// (a0 b0 a1 b1) (a2 b2 a3 b3); else the a's and the b's.
template <bool ADJ>
__device__ __forceinline__ Pairs to_pairs(const float2& l0, const float2& l1, const float2& h0, const float2& h1) {
    Pairs p;
    if (ADJ) {
        p.a[0] = make_float2(l0.x, l1.x);
        p.b[0] = make_float2(l0.y, l1.y);
        p.a[1] = make_float2(h0.x, h1.x);
        p.b[1] = make_float2(h0.y, h1.y);
    } else {
        p.a[0] = l0;
        p.a[1] = l1;
        p.b[0] = h0;
        p.b[1] = h1;
    }
    return p;
}
template <typename TA, bool ADJ>
__device__ __forceinline__ Pairs unpack(const Raw<TA>& r) {
    float2 l0, l1, h0, h1;
    Four<TA>::get(r.lo, l0, l1);
    Four<TA>::get(r.hi, h0, h1);
    return to_pairs<ADJ>(l0, l1, h0, h1);
}
template <typename TA, bool ADJ>
__device__ __forceinline__ Raw<TA> pack(const Pairs& p) {
    Raw<TA> r;
    if (ADJ) {
        r.lo = Four<TA>::put(make_float2(p.a[0].x, p.b[0].x), make_float2(p.a[0].y, p.b[0].y));
        r.hi = Four<TA>::put(make_float2(p.a[1].x, p.b[1].x), make_float2(p.a[1].y, p.b[1].y));
    } else {
        r.lo = Four<TA>::put(p.a[0], p.a[1]);
        r.hi = Four<TA>::put(p.b[0], p.b[1]);
    }
    return r;
}
template <bool ADJ>
__device__ __forceinline__ Pairs load_weight(const float* w, const Lane& L) {
    Raw<float> r;
    r.load(w, L);
    return unpack<float, ADJ>(r);
}

// Cosines and sines of the lane's pairs.
struct Angles {
    float2 c[2], s[2];
};
__device__ __forceinline__ Angles load_angles(const float* row, int rot, const Lane& L) {
    Angles g;
    if (L.angle >= 0) {
        const float4 c = *reinterpret_cast<const float4*>(row + L.angle);
        const float4 s = *reinterpret_cast<const float4*>(row + rot / 2 + L.angle);
        g.c[0] = make_float2(c.x, c.y);
        g.c[1] = make_float2(c.z, c.w);
        g.s[0] = make_float2(s.x, s.y);
        g.s[1] = make_float2(s.z, s.w);
    } else {
        g.c[0] = g.c[1] = make_float2(1.0f, 1.0f);
        g.s[0] = g.s[1] = make_float2(0.0f, 0.0f);
    }
    return g;
}

// Coefficients of one weight: y_a = r (a ac - b bs), y_b = r (b bc + a as).
struct Coef {
    float2 ac[2], bs[2], bc[2], as[2];   // bs holds -w_b s
};
__device__ __forceinline__ Coef make_coef(const Pairs& w, const Angles& g) {
    Coef k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 n = make_float2(-g.s[i].x, -g.s[i].y);
        k.ac[i] = __fmul2_rn(w.a[i], g.c[i]);
        k.bs[i] = __fmul2_rn(w.b[i], n);
        k.bc[i] = __fmul2_rn(w.b[i], g.c[i]);
        k.as[i] = __fmul2_rn(w.a[i], g.s[i]);
    }
    return k;
}

// The rotation alone; `sign` -1 turns back.
__device__ __forceinline__ Coef make_coef(const Angles& g, float sign) {
    Coef k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        k.ac[i] = k.bc[i] = g.c[i];
        k.as[i] = make_float2(sign * g.s[i].x, sign * g.s[i].y);
        k.bs[i] = make_float2(-k.as[i].x, -k.as[i].y);
    }
    return k;
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, LPH);
    return v;
}
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
    float2 s = __fmul2_rn(x.a[0], y.a[0]);
    s = __ffma2_rn(x.a[1], y.a[1], s);
    s = __ffma2_rn(x.b[0], y.b[0], s);
    s = __ffma2_rn(x.b[1], y.b[1], s);
    return s.x + s.y;
}

__device__ __forceinline__ Pairs turn(const Pairs& x, const Coef& k, float r) {
    const float2 rr = make_float2(r, r);
    Pairs y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        y.a[i] = __fmul2_rn(rr, __ffma2_rn(x.a[i], k.ac[i], __fmul2_rn(x.b[i], k.bs[i])));
        y.b[i] = __fmul2_rn(rr, __ffma2_rn(x.b[i], k.bc[i], __fmul2_rn(x.a[i], k.as[i])));
    }
    return y;
}

__device__ __forceinline__ Pairs turn(const Pairs& x, const Coef& k) {
    Pairs y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        y.a[i] = __ffma2_rn(x.a[i], k.ac[i], __fmul2_rn(x.b[i], k.bs[i]));
        y.b[i] = __ffma2_rn(x.b[i], k.bc[i], __fmul2_rn(x.a[i], k.as[i]));
    }
    return y;
}

// ------------------------------------------------------------- many tokens ---
// A team of W warps takes tokens team, team + teams, ...  Stage s of its ring
// holds a token's rows (q, k and, to append, v; backward: q, k and their
// gradients), its row of angles and a note.  The team's first lane starts the
// copies of the token S - 1 ahead.
struct Note {
    int64_t slot;   // -1: not to the cache
    int good;       // the position is in range
    int pad;
};
struct Ring {
    int rows[4];          // byte offsets in a stage: q, k, v | q, k, g_q, g_k
    int sizes[4];         // their bytes, 0: no such row
    int angles, note;     // byte offsets
    int stage_bytes, stages;
    int team_warps;       // 1, 2 or 4
};

__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 0 && ptx::globaltimer() - t0 > WAIT_LIMIT_NS) {
            atomicOr(&g_qk_error, 1u);
            return false;
        }
    }
}

// The team's place in its ring and among the tokens.
struct Team {
    unsigned char* base;        // first stage
    uint32_t full, empty;       // barriers of stage 0
    int64_t first, step, count; // tokens: first + n * step, n < count
    bool leads;                 // this lane starts the copies
    int next_pos;               // leader: position and slot of the next token to start
    int64_t next_slot;
};

__device__ __forceinline__ Team make_team(unsigned char* smem, const Ring& ring, int64_t T) {
    const int W = ring.team_warps, teams = THREADS / 32 / W;
    const int warp = threadIdx.x >> 5, team = warp / W;
    Team m;
    m.base = smem + team * ring.stages * ring.stage_bytes;
    m.full = ptx::smem_u32(smem) + teams * ring.stages * ring.stage_bytes + team * ring.stages * 16;
    m.empty = m.full + ring.stages * 8;
    m.first = static_cast<int64_t>(blockIdx.x) * teams + team;
    m.step = static_cast<int64_t>(gridDim.x) * teams;
    m.count = m.first < T ? (T - m.first + m.step - 1) / m.step : 0;
    m.leads = (threadIdx.x & 31) == 0 && warp % W == 0;
    if (m.leads) {
        for (int s = 0; s < ring.stages; ++s) {
            ptx::mbar_init(m.full + 8 * s, 1);
            ptx::mbar_init(m.empty + 8 * s, W);
        }
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    return m;
}

template <typename P>
__device__ __forceinline__ void fetch_numbers(const P& p, const int64_t* slots, Team& m, int64_t n) {
    if (n >= m.count) return;
    const int64_t t = m.first + n * m.step;
    m.next_pos = p.rot > 0 ? p.positions[t] : 0;
    m.next_slot = slots != nullptr ? slots[t] : -1;
}

// Leader: starts the copies of its n-th token (whose numbers have been
// fetched), then fetches the next one's numbers.
template <typename P>
__device__ __forceinline__ bool start_token(const P& p, const int64_t* slots, int64_t num_slots,
                                            const char* const (&src)[4], const int64_t (&stride)[4], const Ring& ring,
                                            Team& m, int64_t n) {
    if (n >= m.count) return true;
    const int s = static_cast<int>(n % ring.stages);
    const uint32_t round = static_cast<uint32_t>(n / ring.stages);
    if (round > 0 && !wait_full(m.empty + 8 * s, (round & 1) ^ 1)) return false;
    const int64_t t = m.first + n * m.step;
    unsigned char* stage = m.base + s * ring.stage_bytes;
    Note note;
    note.good = p.rot == 0 || (m.next_pos >= 0 && m.next_pos < p.max_pos);
    note.slot = m.next_slot;
    const bool bad_slot = note.slot < -1 || note.slot >= num_slots;
    if (bad_slot) note.slot = -1;
    if (!note.good || (slots != nullptr && bad_slot)) atomicOr(&g_qk_error, 2u);
    *reinterpret_cast<Note*>(stage + ring.note) = note;
    const uint32_t bar = m.full + 8 * s;
    uint32_t bytes = static_cast<uint32_t>(p.rot) * 4u;
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes += static_cast<uint32_t>(ring.sizes[i]);
    ptx::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (ring.sizes[i] > 0)
            ptx::bulk_load(ptx::smem_u32(stage + ring.rows[i]), src[i] + t * stride[i], ring.sizes[i], bar);
    if (p.rot > 0)
        ptx::bulk_load(ptx::smem_u32(stage + ring.angles),
                       p.cos_sin + static_cast<int64_t>(note.good ? m.next_pos : 0) * p.rot, p.rot * 4, bar);
    fetch_numbers(p, slots, m, n + 1);
    return true;
}

// The warp has read stage s.  The bulk copies that refill it are of the
// asynchronous proxy, which an arrive alone does not order behind these reads.
__device__ __forceinline__ void release_stage(const Team& m, int s, int lane) {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(m.empty + 8 * s);
}

// ------------------------------------------------------------------ host ---

inline int lanes_per_head(int Dh) {
    int l = 8;
    while (l * 8 < Dh) l *= 2;
    return l;
}

// The ring for rows of these sizes: teams of 1, 2 or 4 warps, blocks per SM, or
// stages = 0 where two stages do not fit or there are too few tokens.
struct RingPlan {
    Ring ring;
    int blocks;   // of the launch
    size_t smem;
};
constexpr int SM_SMEM = 224 * 1024;

// `values`: elements of a token's rows; `most`: blocks of an SM that the
// kernel's registers allow.
//
// A team's warps share the fixed work of a token (its barrier, angles and
// coefficients), so a team is as small as a token's rows allow: one warp up to
// 3072 values, two up to 6144, four above; but each team wants several tokens,
// or the last round leaves teams idle.  Forward, 32768 tokens of 48 heads of
// 128 (6144 values): 189, 138 and 145 us with one, two and four warps; 24 heads
// of 128: 74, 76 and 109; 9 heads of 128: 38, 51 and 77.  4096 tokens of 24
// heads: 17.9, 12.4 and 15.1.  Backward, 48 heads (12288 values): 378, 247 and
// 194; 24 heads: 131, 103 and 141.
inline RingPlan plan_ring(const int (&sizes)[4], int nrows, int rot, int64_t T, int values, int most) {
    RingPlan r = {};
    int at = 0;
    for (int i = 0; i < nrows; ++i) {
        r.ring.rows[i] = at;
        r.ring.sizes[i] = sizes[i];
        at += (sizes[i] + 127) & ~127;
    }
    r.ring.angles = at;
    at += (rot * 4 + 127) & ~127;
    r.ring.note = at;
    r.ring.stage_bytes = at + 128;
    const int sms = sm_count();
    int teams = 1;
    for (int warps = values <= 3072 ? 1 : values <= 6144 ? 2 : 4; warps <= 4; warps *= 2) {
        teams = THREADS / 32 / warps;
        r.ring.team_warps = warps;
        r.ring.stages = 0;
        // The most blocks of an SM that have two stages or more each: all of an
        // SM's stages together are what is in flight.
        for (int per_sm = most; per_sm >= 1; --per_sm) {
            const int each = SM_SMEM / per_sm - 1024 - teams * 8 * 16;
            const int stages = each / (teams * r.ring.stage_bytes);
            if (stages >= 2) {
                r.ring.stages = stages < 8 ? stages : 8;
                r.blocks = per_sm * sms;
                break;
            }
        }
        const int64_t tokens = warps == 1 ? 8 : 2;   // of a team, at least
        if (r.ring.stages > 0 && T >= tokens * r.blocks * teams) break;
    }
    // fewer than two tokens even for every team of four: the direct kernels
    if (r.ring.stages == 0 || T < 2ll * r.blocks * teams) {
        r.ring.stages = 0;
        return r;
    }
    r.smem = static_cast<size_t>(teams) * r.ring.stages * (r.ring.stage_bytes + 16);
    return r;
}

// cudaFuncSetAttribute to the most a block may have, once per device and kernel.
inline cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

}  // namespace qk
}  // namespace mhc
