// qk_norm_rope.cu -- per-head RMSNorm of queries and keys with the position
// rotation in the same pass: training forward and backward, and the serving
// form that writes keys and values into a paged cache.
//
// For each head x in R^Dh of token t at position p, with weight w and angles
// (c, s) = (cos, sin)[p]:
//   r = 1/sqrt(mean(x^2) + eps),  z = r w x,  y = R z
//   R turns the pairs (a, b) of the first `rot` values: (a c - b s, b c + a s)
// Element-wise that is y_j = r (A_j x_j + B_j x_j'), j' the pair's other
// element, A = w_j c, B = -+ w_j' s: the coefficients depend on the token
// only, so a group of lanes keeps them in registers for all of its heads.
// Backward of <g, y>: h = R^T g, u = w h,
//   dx = r u - x r^3 <u, x> / Dh,   dw = sum over heads of r h x.
//
// Every value is read once and written once and each costs a few operations,
// so these kernels are bound by memory (and by latency for a few tokens).  A
// head is Dh/8 lanes of 8 values (16 bytes of bf16, 32 of float32), lanes per
// head rounded up to a power of two so that the sums are shuffles; a block
// takes one token at a time and all of its lanes' head loads are issued
// before the first is used.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "mhc_common.cuh"
#include "tc_ptx.cuh"

namespace mhc {

__device__ unsigned g_qk_error;   // bit 1: a position or slot outside its range

cudaError_t read_and_clear_qk_error(unsigned* word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_qk_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_qk_error, &zero, sizeof(unsigned));
}

namespace qk {

constexpr int THREADS = 128;

// 8 consecutive values of one head, as loaded.
template <typename TA> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p) { a = ld16_stream(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const { Vec<__nv_bfloat16>::unpack(a, f); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = a; }
    __device__ __forceinline__ static void put(void* p, const float (&f)[8]) {
        *static_cast<uint4*>(p) = Vec<__nv_bfloat16>::pack(f);
    }
    // the same piece of lane `src` of the group
    template <int LPH> __device__ __forceinline__ Raw from(int src) const {
        Raw o;
        o.a.x = __shfl_sync(0xffffffffu, a.x, src, LPH);
        o.a.y = __shfl_sync(0xffffffffu, a.y, src, LPH);
        o.a.z = __shfl_sync(0xffffffffu, a.z, src, LPH);
        o.a.w = __shfl_sync(0xffffffffu, a.w, src, LPH);
        return o;
    }
};
template <> struct Raw<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p) {
        a = ld16_stream(p);
        b = ld16_stream(static_cast<const char*>(p) + 16);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
    __device__ __forceinline__ void store(void* p) const {
        static_cast<uint4*>(p)[0] = a;
        static_cast<uint4*>(p)[1] = b;
    }
    __device__ __forceinline__ static void put(void* p, const float (&f)[8]) {
        static_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
    template <int LPH> __device__ __forceinline__ Raw from(int src) const {
        Raw o;
        o.a.x = __shfl_sync(0xffffffffu, a.x, src, LPH);
        o.a.y = __shfl_sync(0xffffffffu, a.y, src, LPH);
        o.a.z = __shfl_sync(0xffffffffu, a.z, src, LPH);
        o.a.w = __shfl_sync(0xffffffffu, a.w, src, LPH);
        o.b.x = __shfl_sync(0xffffffffu, b.x, src, LPH);
        o.b.y = __shfl_sync(0xffffffffu, b.y, src, LPH);
        o.b.z = __shfl_sync(0xffffffffu, b.z, src, LPH);
        o.b.w = __shfl_sync(0xffffffffu, b.w, src, LPH);
        return o;
    }
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, LPH);
    return v;
}

// What a lane needs to know about the rotation: where the other elements of
// its 8 pairs are.
struct Lane {
    int sub;        // lane of the group
    int j0;         // its first element of the head
    bool on;        // j0 < Dh
    bool turns;     // j0 < rot
    int partner;    // lane that holds the other elements (halves)
    bool upper;     // this lane holds the b of each pair (halves)
};
template <int LPH, bool ADJ>
__device__ __forceinline__ Lane make_lane(int tid, int Dh, int rot) {
    Lane L;
    L.sub = tid & (LPH - 1);
    L.j0 = L.sub * 8;
    L.on = L.j0 < Dh;
    L.turns = L.j0 < rot;
    L.upper = !ADJ && L.turns && L.j0 >= rot / 2;
    L.partner = L.sub;
    if (!ADJ && L.turns) L.partner = L.upper ? L.sub - rot / 16 : L.sub + rot / 16;
    return L;
}

// Cosines and signed sines of the lane's elements: y_j = c_j z_j + s_j z_j'.
template <bool ADJ>
__device__ __forceinline__ void load_angles(const float* row, int rot, const Lane& L, float (&c)[8], float (&s)[8]) {
    if (!L.turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] = 1.0f;
            s[e] = 0.0f;
        }
        return;
    }
    if (ADJ) {
        const float4 cc = *reinterpret_cast<const float4*>(row + L.j0 / 2);
        const float4 ss = *reinterpret_cast<const float4*>(row + rot / 2 + L.j0 / 2);
        c[0] = c[1] = cc.x; c[2] = c[3] = cc.y; c[4] = c[5] = cc.z; c[6] = c[7] = cc.w;
        s[0] = -ss.x; s[1] = ss.x; s[2] = -ss.y; s[3] = ss.y;
        s[4] = -ss.z; s[5] = ss.z; s[6] = -ss.w; s[7] = ss.w;
    } else {
        const int i = L.upper ? L.j0 - rot / 2 : L.j0;
        load8(row + i, c);
        load8(row + rot / 2 + i, s);
        if (!L.upper) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];
        }
    }
}

// The pair's other element of each of the lane's values.
template <typename TA, int LPH, bool ADJ>
__device__ __forceinline__ void other_elements(const Raw<TA>& raw, const float (&x)[8], const Lane& L, float (&xp)[8]) {
    if (ADJ) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
    } else {
        raw.template from<LPH>(L.partner).get(xp);
    }
}

// Coefficients of one weight: A = w c, B = w' s.
template <bool ADJ>
__device__ __forceinline__ void coefficients(const float* w, const Lane& L, const float (&c)[8], const float (&s)[8],
                                             float (&A)[8], float (&B)[8]) {
    float a[8];
    load8(w + L.j0, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) A[e] = a[e] * c[e];
    if (ADJ) {
#pragma unroll
        for (int e = 0; e < 8; ++e) B[e] = a[e ^ 1] * s[e];
    } else {
        float b[8];
        load8(w + L.partner * 8, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) B[e] = b[e] * s[e];
    }
}

// Heads a group has in flight.
template <typename TA> constexpr int unroll() { return sizeof(TA) == 2 ? 6 : 3; }

template <typename TA, int LPH, bool ADJ, bool APPEND>
__global__ void __launch_bounds__(THREADS)
qk_norm_rope_kernel(const QkParams p) {
    constexpr int NGRP = THREADS / LPH, U = unroll<TA>();
    const Lane L = make_lane<LPH, ADJ>(threadIdx.x, p.Dh, p.rot);
    const int grp = threadIdx.x / LPH;
    const int heads = p.Hq + p.Hk + (APPEND ? p.Hk : 0);
    const int per = (heads + gridDim.y - 1) / gridDim.y;
    const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    const TA* q = static_cast<const TA*>(p.q);
    const TA* k = static_cast<const TA*>(p.k);
    const TA* v = static_cast<const TA*>(p.v);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int pos = p.rot > 0 ? p.positions[t] : 0;
        const bool good = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
        int64_t slot = -1;
        if (APPEND) {
            slot = p.slots[t];
            if (slot < -1 || slot >= p.num_slots) {
                if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_qk_error, 2u);
                slot = -1;
            }
        }
        if (!good && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_qk_error, 2u);
        int64_t at_k = 0, at_v = 0;
        if (APPEND && slot >= 0) {
            const int64_t page = slot / p.page_size, in = slot - page * p.page_size;
            at_k = page * p.k_page_stride + in * p.k_slot_stride;
            at_v = page * p.v_page_stride + in * p.v_slot_stride;
        }
        float Aq[8], Bq[8], Ak[8], Bk[8];
        if (L.on) {
            float c[8], s[8];
            load_angles<ADJ>(p.cos_sin + static_cast<int64_t>(good ? pos : 0) * p.rot, p.rot, L, c, s);
            coefficients<ADJ>(p.w_q, L, c, s, Aq, Bq);
            coefficients<ADJ>(p.w_k, L, c, s, Ak, Bk);
        }
        for (int hb = h0; hb < h1; hb += NGRP * U) {
            Raw<TA> x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                x[i].zero();
                if (h < h1 && L.on) {
                    if (h < p.Hq)
                        x[i].load(q + t * p.q_stride + static_cast<int64_t>(h) * p.Dh + L.j0);
                    else if (h < p.Hq + p.Hk)
                        x[i].load(k + t * p.k_stride + static_cast<int64_t>(h - p.Hq) * p.Dh + L.j0);
                    else
                        x[i].load(v + t * p.v_stride + static_cast<int64_t>(h - p.Hq - p.Hk) * p.Dh + L.j0);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                float f[8], xp[8], y[8];
                x[i].get(f);
                other_elements<TA, LPH, ADJ>(x[i], f, L, xp);
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
                ss = group_sum<LPH>(ss);
                if (h >= h1 || !L.on) continue;
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                const bool is_q = h < p.Hq;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = is_q ? Aq[e] : Ak[e], b = is_q ? Bq[e] : Bk[e];
                    y[e] = good ? r * fmaf(a, f[e], b * xp[e]) : 0.0f;
                }
                if (is_q) {
                    Raw<TA>::put(static_cast<TA*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(h) * p.Dh + L.j0, y);
                } else if (h < p.Hq + p.Hk) {
                    const int64_t hk = h - p.Hq;
                    if (!APPEND)
                        Raw<TA>::put(static_cast<TA*>(p.k_out) + t * p.k_out_stride + hk * p.Dh + L.j0, y);
                    else if (slot >= 0 && good)
                        Raw<TA>::put(static_cast<TA*>(p.k_out) + at_k + hk * p.k_head_stride + L.j0, y);
                } else if (APPEND && slot >= 0 && good) {
                    const int64_t hv = h - p.Hq - p.Hk;
                    x[i].store(static_cast<TA*>(p.v_out) + at_v + hv * p.v_head_stride + L.j0);
                }
            }
        }
    }
}

// Backward.  A block walks tokens blockIdx.x, + gridDim.x, ...; each lane sums
// r h x of its 8 elements over its heads and tokens in registers, the block's
// groups are added in a fixed order in shared memory, and the block writes one
// partial of dw_q and dw_k; qk_dw_kernel adds the partials in a fixed order.
template <typename TA> constexpr int unroll_bwd() { return sizeof(TA) == 2 ? 3 : 2; }

template <typename TA, int LPH, bool ADJ>
__global__ void __launch_bounds__(THREADS)
qk_norm_rope_bwd_kernel(const QkBwdParams p) {
    constexpr int NGRP = THREADS / LPH, U = unroll_bwd<TA>();
    __shared__ float red[NGRP][LPH * 8];
    const Lane L = make_lane<LPH, ADJ>(threadIdx.x, p.Dh, p.rot);
    const int grp = threadIdx.x / LPH;
    const int heads = p.Hq + p.Hk;
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    const TA* q = static_cast<const TA*>(p.q);
    const TA* k = static_cast<const TA*>(p.k);
    const TA* gq = static_cast<const TA*>(p.g_q);
    const TA* gk = static_cast<const TA*>(p.g_k);
    float dwq[8], dwk[8], wq[8], wk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = wq[e] = wk[e] = 0.0f;
    if (L.on) {
        load8(p.w_q + L.j0, wq);
        load8(p.w_k + L.j0, wk);
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int pos = p.rot > 0 ? p.positions[t] : 0;
        const bool good = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
        if (!good && threadIdx.x == 0) atomicOr(&g_qk_error, 2u);
        float c[8], s[8];
        if (L.on) load_angles<ADJ>(p.cos_sin + static_cast<int64_t>(good ? pos : 0) * p.rot, p.rot, L, c, s);
        for (int hb = 0; hb < heads; hb += NGRP * U) {
            Raw<TA> x[U], g[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                x[i].zero();
                g[i].zero();
                if (h < heads && L.on) {
                    if (h < p.Hq) {
                        x[i].load(q + t * p.q_stride + static_cast<int64_t>(h) * p.Dh + L.j0);
                        g[i].load(gq + t * p.gq_stride + static_cast<int64_t>(h) * p.Dh + L.j0);
                    } else {
                        x[i].load(k + t * p.k_stride + static_cast<int64_t>(h - p.Hq) * p.Dh + L.j0);
                        g[i].load(gk + t * p.gk_stride + static_cast<int64_t>(h - p.Hq) * p.Dh + L.j0);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                const bool is_q = h < p.Hq;
                float f[8], gg[8], gp[8], hh[8], u[8];
                x[i].get(f);
                g[i].get(gg);
                other_elements<TA, LPH, ADJ>(g[i], gg, L, gp);
                float ss = 0.0f, ux = 0.0f;
                if (L.on) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        hh[e] = fmaf(c[e], gg[e], -s[e] * gp[e]);   // R^T: the sines' signs turn
                        u[e] = hh[e] * (is_q ? wq[e] : wk[e]);
                        ss = fmaf(f[e], f[e], ss);
                        ux = fmaf(u[e], f[e], ux);
                    }
                }
                ss = group_sum<LPH>(ss);
                ux = group_sum<LPH>(ux);
                if (h >= heads || !L.on) continue;
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                const float m = r * r * ux * inv_d;
                float dx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dx[e] = good ? r * fmaf(-f[e], m, u[e]) : 0.0f;
                    const float d = good ? r * hh[e] * f[e] : 0.0f;
                    if (is_q) dwq[e] += d;
                    else dwk[e] += d;
                }
                if (is_q)
                    Raw<TA>::put(static_cast<TA*>(p.dq) + t * p.dq_stride + static_cast<int64_t>(h) * p.Dh + L.j0, dx);
                else
                    Raw<TA>::put(static_cast<TA*>(p.dk) + t * p.dk_stride + static_cast<int64_t>(h - p.Hq) * p.Dh + L.j0, dx);
            }
        }
    }
    ptx::griddep_launch_dependents();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[grp][L.j0 + e] = which ? dwk[e] : dwq[e];
        __syncthreads();
        for (int j = threadIdx.x; j < p.Dh; j += THREADS) {
            float a = 0.0f;
#pragma unroll
            for (int g = 0; g < NGRP; ++g) a += red[g][j];
            p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * p.Dh + j] = a;
        }
    }
}

// dw[which][j] = sum over blocks of the partials, in a fixed order: 32 rows of
// threads take every 32nd block each, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024)
qk_dw_kernel(const float* __restrict__ partial, int nblk, int Dh, float* __restrict__ dw_q, float* __restrict__ dw_k) {
    __shared__ float red[32][33];
    const int j = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
    ptx::griddep_wait();
    float a = 0.0f;
    if (j < Dh)
        for (int b = threadIdx.y; b < nblk; b += 32) a += partial[(static_cast<int64_t>(b) * 2 + which) * Dh + j];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && j < Dh) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
        (which ? dw_k : dw_q)[j] = v;
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 148;
    return n;
}

int lanes_per_head(int Dh) {
    int l = 4;
    while (l * 8 < Dh) l *= 2;
    return l;
}

template <typename TA, bool ADJ, bool APPEND>
cudaError_t launch_fwd(const QkParams& p, cudaStream_t s) {
    const int lph = lanes_per_head(p.Dh), ngrp = THREADS / lph;
    const int heads = p.Hq + p.Hk + (APPEND ? p.Hk : 0);
    // many tokens: a block per token (its groups share the token's angles);
    // few: the token's heads go to several blocks, one head per group, so that
    // a call of one token is one round trip to memory
    const int most = (heads + ngrp - 1) / ngrp;
    const int64_t want = 4 * sm_count();
    int64_t split = p.T >= want ? 1 : (want + p.T - 1) / p.T;
    if (split > most) split = most;
    const int64_t bx = p.T < 65536 ? p.T : 65536;
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(split));
    switch (lph) {
        case 4: qk_norm_rope_kernel<TA, 4, ADJ, APPEND><<<grid, THREADS, 0, s>>>(p); break;
        case 8: qk_norm_rope_kernel<TA, 8, ADJ, APPEND><<<grid, THREADS, 0, s>>>(p); break;
        case 16: qk_norm_rope_kernel<TA, 16, ADJ, APPEND><<<grid, THREADS, 0, s>>>(p); break;
        case 32: qk_norm_rope_kernel<TA, 32, ADJ, APPEND><<<grid, THREADS, 0, s>>>(p); break;
        default: return cudaErrorNotSupported;
    }
    return cudaGetLastError();
}

template <typename TA, bool ADJ>
cudaError_t launch_bwd(const QkBwdParams& p, int64_t nblk, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(nblk);
    switch (lanes_per_head(p.Dh)) {
        case 4: qk_norm_rope_bwd_kernel<TA, 4, ADJ><<<grid, THREADS, 0, s>>>(p); break;
        case 8: qk_norm_rope_bwd_kernel<TA, 8, ADJ><<<grid, THREADS, 0, s>>>(p); break;
        case 16: qk_norm_rope_bwd_kernel<TA, 16, ADJ><<<grid, THREADS, 0, s>>>(p); break;
        case 32: qk_norm_rope_bwd_kernel<TA, 32, ADJ><<<grid, THREADS, 0, s>>>(p); break;
        default: return cudaErrorNotSupported;
    }
    return cudaGetLastError();
}

}  // namespace qk

int64_t qk_bwd_blocks(int64_t T) {
    // one wave of persistent blocks: the dw partials stay few
    const int64_t most = 6ll * qk::sm_count();
    return T < most ? T : most;
}

cudaError_t launch_qk_norm_rope(bool bf16, bool adjacent, bool append, const QkParams& p, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (bf16) {
        if (append) return adjacent ? qk::launch_fwd<B, true, true>(p, s) : qk::launch_fwd<B, false, true>(p, s);
        return adjacent ? qk::launch_fwd<B, true, false>(p, s) : qk::launch_fwd<B, false, false>(p, s);
    }
    if (append) return adjacent ? qk::launch_fwd<float, true, true>(p, s) : qk::launch_fwd<float, false, true>(p, s);
    return adjacent ? qk::launch_fwd<float, true, false>(p, s) : qk::launch_fwd<float, false, false>(p, s);
}

cudaError_t launch_qk_norm_rope_bwd(bool bf16, bool adjacent, const QkBwdParams& p, float* dw_q, float* dw_k,
                                    cudaStream_t s) {
    using B = __nv_bfloat16;
    const int64_t nblk = qk_bwd_blocks(p.T);
    cudaError_t e;
    if (bf16) e = adjacent ? qk::launch_bwd<B, true>(p, nblk, s) : qk::launch_bwd<B, false>(p, nblk, s);
    else e = adjacent ? qk::launch_bwd<float, true>(p, nblk, s) : qk::launch_bwd<float, false>(p, nblk, s);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.Dh + 31) / 32), 2);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk::qk_dw_kernel, static_cast<const float*>(p.partial), static_cast<int>(nblk),
                              p.Dh, dw_q, dw_k);
}

}  // namespace mhc
