// qk_norm_rope_bwd.cu -- backward of the per-head RMSNorm with rotation.  The
// mathematics and the shared parts are in qk_norm_rope.cuh.
// Bound by memory traffic: at T = 32768, 40 + 8 heads of 128, bf16, 194 us,
// 6.2 TB/s, 0.93 of the measured copy rate.
#include "qk_norm_rope.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_qk_bwd_error(unsigned* word) { return g_error_word.read_and_clear(g_qk_error, word); }

namespace qk {

template <typename TA, int LPH, bool ADJ>
__device__ __forceinline__ void head_backward(const Raw<TA>& raw, const Raw<TA>& graw, const Angles& ang, const Pairs& w,
                                              Pairs& dw, bool good, float inv_d, float eps, TA* out, const Lane& L,
                                              bool there) {
    const Pairs x = unpack<TA, ADJ>(raw), g = unpack<TA, ADJ>(graw);
    Pairs h, u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // R^T: the sines' signs turn
        const float2 n = make_float2(-ang.s[i].x, -ang.s[i].y);
        h.a[i] = __ffma2_rn(g.a[i], ang.c[i], __fmul2_rn(g.b[i], ang.s[i]));
        h.b[i] = __ffma2_rn(g.b[i], ang.c[i], __fmul2_rn(g.a[i], n));
        u.a[i] = __fmul2_rn(h.a[i], w.a[i]);
        u.b[i] = __fmul2_rn(h.b[i], w.b[i]);
    }
    const float ss = group_sum<LPH>(dot(x, x)), ux = group_sum<LPH>(dot(u, x));
    if (!there) return;
    Raw<TA> o;
    if (good) {
        const float r = rsqrtf(fmaf(ss, inv_d, eps)), m = -r * r * ux * inv_d;
        const float2 rr = make_float2(r, r), mm = make_float2(m, m);
        Pairs d;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            d.a[i] = __fmul2_rn(rr, __ffma2_rn(x.a[i], mm, u.a[i]));
            d.b[i] = __fmul2_rn(rr, __ffma2_rn(x.b[i], mm, u.b[i]));
            dw.a[i] = __ffma2_rn(__fmul2_rn(rr, x.a[i]), h.a[i], dw.a[i]);
            dw.b[i] = __ffma2_rn(__fmul2_rn(rr, x.b[i]), h.b[i], dw.b[i]);
        }
        o = pack<TA, ADJ>(d);
    } else {
        o.zero();
    }
    o.store(out, L);
}

// Each lane sums r h x of its pairs over its heads and
// tokens in registers, the block's groups are added in a fixed order in shared
// memory, and the block writes one partial of dw_q and dw_k; qk_dw_kernel adds
// the partials in a fixed order.
template <typename TA, int LPH, bool ADJ>
__device__ __forceinline__ void write_partials(const QkBwdParams& p, const Lane& L, float* red, const Pairs& dq,
                                               const Pairs& dk) {
    constexpr int NGRP = THREADS / LPH;
    const int grp = threadIdx.x / LPH;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (L.on) pack<float, ADJ>(which ? dk : dq).store(red + grp * LPH * 8, L);
        __syncthreads();
        for (int j = threadIdx.x; j < p.Dh; j += THREADS) {
            float a = 0.0f;
#pragma unroll
            for (int g = 0; g < NGRP; ++g) a += red[g * LPH * 8 + j];
            p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * p.Dh + j] = a;
        }
    }
}

__device__ __forceinline__ void add(Pairs& to, const Pairs& d) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        to.a[e] = __fadd2_rn(to.a[e], d.a[e]);
        to.b[e] = __fadd2_rn(to.b[e], d.b[e]);
    }
}

template <typename TA, int LPH, bool ADJ>
__global__ void __launch_bounds__(THREADS)
qk_direct_bwd_kernel(const QkBwdParams p) {
    constexpr int NGRP = THREADS / LPH, U = 2;
    __shared__ float red[THREADS * 8];
    const Lane L = make_lane<LPH, ADJ>(threadIdx.x & 31, p.Dh, p.rot);
    const int grp = threadIdx.x / LPH;
    const int heads = p.Hq + p.Hk;
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    Pairs dwq = {}, dwk = {}, wq = {}, wk = {};
    if (L.on) {
        wq = load_weight<ADJ>(p.w_q, L);
        wk = load_weight<ADJ>(p.w_k, L);
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        Raw<TA> x[U], g[U];
        auto load = [&](int hb) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                x[i].zero();
                g[i].zero();
                if (h < p.Hq && L.on) {
                    x[i].stream(static_cast<const TA*>(p.q) + t * p.q_stride + h * p.Dh, L);
                    g[i].stream(static_cast<const TA*>(p.g_q) + t * p.gq_stride + h * p.Dh, L);
                } else if (h < heads && L.on) {
                    x[i].stream(static_cast<const TA*>(p.k) + t * p.k_stride + (h - p.Hq) * p.Dh, L);
                    g[i].stream(static_cast<const TA*>(p.g_k) + t * p.gk_stride + (h - p.Hq) * p.Dh, L);
                }
            }
        };
        load(0);
        const int pos = p.rot > 0 ? p.positions[t] : 0;
        const bool good = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
        if (!good && threadIdx.x == 0) atomicOr(&g_qk_error, 2u);
        Angles ang = {};
        if (L.on) ang = load_angles(p.cos_sin + static_cast<int64_t>(good ? pos : 0) * p.rot, p.rot, L);
        for (int hb = 0; hb < heads; hb += NGRP * U) {
            if (hb > 0) load(hb);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                const bool is_q = h < p.Hq;
                TA* out = is_q ? static_cast<TA*>(p.dq) + t * p.dq_stride + h * p.Dh
                               : static_cast<TA*>(p.dk) + t * p.dk_stride + (h - p.Hq) * p.Dh;
                Pairs d = {};
                head_backward<TA, LPH, ADJ>(x[i], g[i], ang, is_q ? wq : wk, d, good, inv_d, p.eps, out, L,
                                            h < heads && L.on);
                if (is_q) add(dwq, d);
                else add(dwk, d);
            }
        }
    }
    ptx::griddep_launch_dependents();
    write_partials<TA, LPH, ADJ>(p, L, red, dwq, dwk);
}

template <typename TA, int LPH, bool ADJ>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS)
qk_staged_bwd_kernel(const QkBwdParams p, const Ring ring) {
    const int W = ring.team_warps, NGRP = W * 32 / LPH;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Lane L = make_lane<LPH, ADJ>(lane, p.Dh, p.rot);
    const int grp = ((warp % W) * 32 + lane) / LPH;
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    constexpr int64_t E = sizeof(TA);
    const char* const src[4] = {static_cast<const char*>(p.q), static_cast<const char*>(p.k),
                                static_cast<const char*>(p.g_q), static_cast<const char*>(p.g_k)};
    const int64_t stride[4] = {p.q_stride * E, p.k_stride * E, p.gq_stride * E, p.gk_stride * E};
    Team m = make_team(smem, ring, p.T);
    bool ok = true;
    if (m.leads) {
        fetch_numbers(p, nullptr, m, 0);
        for (int n = 0; ok && n < ring.stages - 1; ++n) ok = start_token(p, nullptr, 0, src, stride, ring, m, n);
    }
    Pairs dwq = {}, dwk = {}, wq = {}, wk = {};
    if (L.on) {
        wq = load_weight<ADJ>(p.w_q, L);
        wk = load_weight<ADJ>(p.w_k, L);
    }
    int s = 0;
    uint32_t parity = 0;
    for (int64_t n = 0; n < m.count; ++n) {
        if (m.leads && ok) ok = start_token(p, nullptr, 0, src, stride, ring, m, n + ring.stages - 1);
        ok = __all_sync(0xffffffffu, ok && wait_full(m.full + 8 * s, parity));
        if (!ok) break;
        const unsigned char* stage = m.base + s * ring.stage_bytes;
        const int64_t t = m.first + n * m.step;
        const bool good = reinterpret_cast<const Note*>(stage + ring.note)->good != 0;
        Angles ang = {};
        if (L.on) ang = load_angles(reinterpret_cast<const float*>(stage + ring.angles), p.rot, L);
        const TA* q = reinterpret_cast<const TA*>(stage + ring.rows[0]);
        const TA* gq = reinterpret_cast<const TA*>(stage + ring.rows[2]);
        TA* dq = static_cast<TA*>(p.dq) + t * p.dq_stride;
#pragma unroll 2
        for (int hb = 0; hb < p.Hq; hb += NGRP) {
            const int h = hb + grp;
            const bool there = h < p.Hq && L.on;
            Raw<TA> x, g;
            x.zero();
            g.zero();
            if (there) {
                x.load(q + h * p.Dh, L);
                g.load(gq + h * p.Dh, L);
            }
            head_backward<TA, LPH, ADJ>(x, g, ang, wq, dwq, good, inv_d, p.eps, dq + h * p.Dh, L, there);
        }
        const TA* k = reinterpret_cast<const TA*>(stage + ring.rows[1]);
        const TA* gk = reinterpret_cast<const TA*>(stage + ring.rows[3]);
        TA* dk = static_cast<TA*>(p.dk) + t * p.dk_stride;
        for (int hb = 0; hb < p.Hk; hb += NGRP) {
            const int h = hb + grp;
            const bool there = h < p.Hk && L.on;
            Raw<TA> x, g;
            x.zero();
            g.zero();
            if (there) {
                x.load(k + h * p.Dh, L);
                g.load(gk + h * p.Dh, L);
            }
            head_backward<TA, LPH, ADJ>(x, g, ang, wk, dwk, good, inv_d, p.eps, dk + h * p.Dh, L, there);
        }
        release_stage(m, s, lane);
        if (++s == ring.stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (!ok) {
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000ull) {
        }
    }
    ptx::griddep_launch_dependents();
    // every stage has been read: the ring is free for the groups' sums
    write_partials<TA, LPH, ADJ>(p, L, reinterpret_cast<float*>(smem), dwq, dwk);
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

template <typename TA>
RingPlan plan_bwd(const QkBwdParams& p) {
    const int e = static_cast<int>(sizeof(TA));
    const int sizes[4] = {p.Hq * p.Dh * e, p.Hk * p.Dh * e, p.Hq * p.Dh * e, p.Hk * p.Dh * e};
    RingPlan r = plan_ring(sizes, 4, p.rot, p.T, 2 * (p.Hq + p.Hk) * p.Dh, BWD_BLOCKS);
    // the ring also holds the groups' sums at the end
    if (r.ring.stages > 0 && r.smem < THREADS * 8 * sizeof(float)) r.smem = THREADS * 8 * sizeof(float);
    return r;
}

template <typename TA, int LPH, bool ADJ>
cudaError_t launch_bwd_lph(const QkBwdParams& p, int64_t* nblk, cudaStream_t s) {
    const RingPlan r = plan_bwd<TA>(p);
    if (r.ring.stages > 0) {
        static std::atomic<uint64_t> done{0};
        auto kernel = qk_staged_bwd_kernel<TA, LPH, ADJ>;
        const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), done);
        if (err != cudaSuccess) return err;
        *nblk = r.blocks;
        kernel<<<r.blocks, THREADS, r.smem, s>>>(p, r.ring);
        return cudaGetLastError();
    }
    const int64_t most = qk_bwd_blocks(p.T);
    *nblk = p.T < most ? p.T : most;
    qk_direct_bwd_kernel<TA, LPH, ADJ><<<static_cast<unsigned>(*nblk), THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename TA, bool ADJ>
cudaError_t launch_bwd(const QkBwdParams& p, int64_t* nblk, cudaStream_t s) {
    switch (lanes_per_head(p.Dh)) {
        case 8: return launch_bwd_lph<TA, 8, ADJ>(p, nblk, s);
        case 16: return launch_bwd_lph<TA, 16, ADJ>(p, nblk, s);
        case 32: return launch_bwd_lph<TA, 32, ADJ>(p, nblk, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace qk

// Most blocks a backward launch has, each with one partial of dw.
int64_t qk_bwd_blocks(int64_t T) {
    const int64_t most = 6ll * sm_count();
    return T < most ? T : most;
}

cudaError_t launch_qk_norm_rope_bwd(bool bf16, bool adjacent, const QkBwdParams& p, float* dw_q, float* dw_k,
                                    cudaStream_t s) {
    g_error_word.may_be_set();
    using B = __nv_bfloat16;
    int64_t nblk = 0;
    cudaError_t e;
    if (bf16) e = adjacent ? qk::launch_bwd<B, true>(p, &nblk, s) : qk::launch_bwd<B, false>(p, &nblk, s);
    else e = adjacent ? qk::launch_bwd<float, true>(p, &nblk, s) : qk::launch_bwd<float, false>(p, &nblk, s);
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
