// qk_norm_rope_fwd.cuh -- the forward kernels of qk_norm_rope.cu (NORM) and of
// qk_norm_rope_bare.cu, the rotation alone.  The mathematics and the shared
// parts are in qk_norm_rope.cuh.
#pragma once

#include "qk_norm_rope.cuh"

namespace mhc {

namespace qk {

// One head, in and out (every lane of the group; `there` says whether it is one).
template <typename TA, int LPH, bool ADJ, bool NORM>
__device__ __forceinline__ void head_forward(const Raw<TA>& raw, const Coef& k, bool good, float inv_d, float eps,
                                             TA* out, const Lane& L, bool there) {
    const Pairs x = unpack<TA, ADJ>(raw);
    if (!NORM) {
        // values past the turned ones are copied: a product with a sine of zero would spread infinities
        if (!there) return;
        if (good && L.angle < 0) raw.store(out, L);
        else if (good) pack<TA, ADJ>(turn(x, k)).store(out, L);
        else {
            Raw<TA> z;
            z.zero();
            z.store(out, L);
        }
        return;
    }
    const float r = rsqrtf(fmaf(group_sum<LPH>(dot(x, x)), inv_d, eps));
    if (!there) return;
    if (good) pack<TA, ADJ>(turn(x, k, r)).store(out, L);
    else {
        Raw<TA> z;
        z.zero();
        z.store(out, L);
    }
}

// Where a token's keys and values go in the caches.
struct Place {
    int64_t k, v;
};
__device__ __forceinline__ Place cache_place(const QkParams& p, int64_t slot) {
    const int64_t page = slot / p.page_size, in = slot - page * p.page_size;
    return {page * p.k_page_stride + in * p.k_slot_stride, page * p.v_page_stride + in * p.v_slot_stride};
}

// -------------------------------------------------------------- few tokens ---
constexpr int DIRECT_HEADS = 4;   // of a group at a time

template <typename TA, int LPH, bool ADJ, bool APPEND, bool NORM>
__global__ void __launch_bounds__(THREADS)
qk_direct_kernel(const QkParams p) {
    constexpr int NGRP = THREADS / LPH, U = DIRECT_HEADS;
    const Lane L = make_lane<LPH, ADJ>(threadIdx.x & 31, p.Dh, p.rot);
    const int grp = threadIdx.x / LPH;
    const int heads = p.Hq + p.Hk + (APPEND ? p.Hk : 0);
    const int per = (heads + gridDim.y - 1) / gridDim.y;
    const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const TA* q = static_cast<const TA*>(p.q) + t * p.q_stride;
        const TA* k = static_cast<const TA*>(p.k) + t * p.k_stride;
        const TA* v = static_cast<const TA*>(p.v) + t * p.v_stride;
        Raw<TA> x[U];
        auto load = [&](int hb) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp;
                x[i].zero();
                if (h < h1 && L.on)
                    x[i].stream(h < p.Hq ? q + h * p.Dh
                                         : h < p.Hq + p.Hk ? k + (h - p.Hq) * p.Dh : v + (h - p.Hq - p.Hk) * p.Dh, L);
            }
        };
        // the heads are on their way before the position is known, and the
        // angles come after the position
        load(h0);
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
        Coef kq = {}, kk = {};
        if (L.on) {
            const Angles g = load_angles(p.cos_sin + static_cast<int64_t>(good ? pos : 0) * p.rot, p.rot, L);
            if (NORM) {
                kq = make_coef(load_weight<ADJ>(p.w_q, L), g);
                kk = make_coef(load_weight<ADJ>(p.w_k, L), g);
            } else {
                kq = kk = make_coef(g, p.sine_sign);
            }
        }
        const bool write = APPEND && slot >= 0 && good;
        const Place at = write ? cache_place(p, slot) : Place{0, 0};
        for (int hb = h0; hb < h1; hb += NGRP * U) {
            if (hb > h0) load(hb);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = hb + i * NGRP + grp, hk = h - p.Hq, hv = hk - p.Hk;
                const bool there = h < h1 && L.on;
                if (APPEND && __all_sync(0xffffffffu, hv >= 0)) {
                    if (there && write) x[i].store(static_cast<TA*>(p.v_out) + at.v + hv * p.v_head_stride, L);
                } else {
                    const bool is_q = hk < 0, is_v = hv >= 0;
                    TA* out = is_q ? static_cast<TA*>(p.q_out) + t * p.q_out_stride + h * p.Dh
                              : APPEND ? static_cast<TA*>(p.k_out) + at.k + hk * p.k_head_stride
                                       : static_cast<TA*>(p.k_out) + t * p.k_out_stride + hk * p.Dh;
                    head_forward<TA, LPH, ADJ, NORM>(x[i], is_q ? kq : kk, good, inv_d, p.eps, out, L,
                                               there && !is_v && (is_q || !APPEND || write));
                    if (APPEND && is_v && there && write)
                        x[i].store(static_cast<TA*>(p.v_out) + at.v + hv * p.v_head_stride, L);
                }
            }
        }
    }
}

// ------------------------------------------------------------- many tokens ---
template <typename TA, int LPH, bool ADJ, bool APPEND, bool NORM>
__global__ void __launch_bounds__(THREADS, FWD_BLOCKS)
qk_staged_kernel(const QkParams p, const Ring ring) {
    const int W = ring.team_warps, NGRP = W * 32 / LPH;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Lane L = make_lane<LPH, ADJ>(lane, p.Dh, p.rot);
    const int grp = ((warp % W) * 32 + lane) / LPH;
    const float inv_d = 1.0f / static_cast<float>(p.Dh);
    const char* const src[4] = {static_cast<const char*>(p.q), static_cast<const char*>(p.k),
                                static_cast<const char*>(p.v), nullptr};
    const int64_t stride[4] = {p.q_stride * static_cast<int64_t>(sizeof(TA)), p.k_stride * static_cast<int64_t>(sizeof(TA)),
                               p.v_stride * static_cast<int64_t>(sizeof(TA)), 0};
    const int64_t* slots = APPEND ? p.slots : nullptr;
    Team m = make_team(smem, ring, p.T);
    bool ok = true;
    if (m.leads) {
        fetch_numbers(p, slots, m, 0);
        for (int n = 0; ok && n < ring.stages - 1; ++n)
            ok = start_token(p, slots, p.num_slots, src, stride, ring, m, n);
    }
    Pairs wq = {}, wk = {};
    if (NORM && L.on) {
        wq = load_weight<ADJ>(p.w_q, L);
        wk = load_weight<ADJ>(p.w_k, L);
    }
    int s = 0;
    uint32_t parity = 0;
    for (int64_t n = 0; n < m.count; ++n) {
        if (m.leads && ok) ok = start_token(p, slots, p.num_slots, src, stride, ring, m, n + ring.stages - 1);
        ok = __all_sync(0xffffffffu, ok && wait_full(m.full + 8 * s, parity));
        if (!ok) break;
        const unsigned char* stage = m.base + s * ring.stage_bytes;
        const Note note = *reinterpret_cast<const Note*>(stage + ring.note);
        const int64_t t = m.first + n * m.step;
        const bool good = note.good != 0, write = APPEND && note.slot >= 0 && good;
        Coef kq = {}, kk = {};
        if (L.on) {
            const Angles g = load_angles(reinterpret_cast<const float*>(stage + ring.angles), p.rot, L);
            if (NORM) {
                kq = make_coef(wq, g);
                kk = make_coef(wk, g);
            } else {
                kq = kk = make_coef(g, p.sine_sign);
            }
        }
        const TA* q = reinterpret_cast<const TA*>(stage + ring.rows[0]);
        const TA* k = reinterpret_cast<const TA*>(stage + ring.rows[1]);
        TA* qo = static_cast<TA*>(p.q_out) + t * p.q_out_stride;
        const Place at = write ? cache_place(p, note.slot) : Place{0, 0};
#pragma unroll 2
        for (int hb = 0; hb < p.Hq; hb += NGRP) {
            const int h = hb + grp;
            const bool there = h < p.Hq && L.on;
            Raw<TA> x;
            x.zero();
            if (there) x.load(q + h * p.Dh, L);
            head_forward<TA, LPH, ADJ, NORM>(x, kq, good, inv_d, p.eps, qo + h * p.Dh, L, there);
        }
        TA* ko = APPEND ? static_cast<TA*>(p.k_out) + at.k : static_cast<TA*>(p.k_out) + t * p.k_out_stride;
        const int64_t ks = APPEND ? p.k_head_stride : p.Dh;
        for (int hb = 0; hb < p.Hk; hb += NGRP) {
            const int h = hb + grp;
            const bool there = h < p.Hk && L.on;
            Raw<TA> x;
            x.zero();
            if (there) x.load(k + h * p.Dh, L);
            head_forward<TA, LPH, ADJ, NORM>(x, kk, good, inv_d, p.eps, ko + h * ks, L, there && (!APPEND || write));
        }
        if (APPEND && write && L.on) {
            const TA* v = reinterpret_cast<const TA*>(stage + ring.rows[2]);
            TA* vo = static_cast<TA*>(p.v_out) + at.v;
            for (int h = grp; h < p.Hk; h += NGRP) {
                Raw<TA> x;
                x.load(v + h * p.Dh, L);
                x.store(vo + h * p.v_head_stride, L);
            }
        }
        release_stage(m, s, lane);
        if (++s == ring.stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (!ok) {   // let copies already issued land before the shared memory goes away
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000ull) {
        }
    }
}

template <typename TA, int LPH, bool ADJ, bool APPEND, bool NORM>
cudaError_t launch_fwd_lph(const QkParams& p, cudaStream_t s) {
    const int e = static_cast<int>(sizeof(TA));
    const int sizes[4] = {p.Hq * p.Dh * e, p.Hk * p.Dh * e, p.Hk * p.Dh * e, 0};
    const RingPlan r = plan_ring(sizes, APPEND ? 3 : 2, p.rot, p.T, (p.Hq + (APPEND ? 2 : 1) * p.Hk) * p.Dh, FWD_BLOCKS);
    if (r.ring.stages > 0) {
        static std::atomic<uint64_t> done{0};
        auto kernel = qk_staged_kernel<TA, LPH, ADJ, APPEND, NORM>;
        const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), done);
        if (err != cudaSuccess) return err;
        kernel<<<r.blocks, THREADS, r.smem, s>>>(p, r.ring);
        return cudaGetLastError();
    }
    // a token's heads go to several blocks until the GPU is covered
    const int heads = p.Hq + p.Hk + (APPEND ? p.Hk : 0), ngrp = THREADS / LPH;
    const int most = (heads + ngrp - 1) / ngrp;
    const int64_t want = 4ll * sm_count();
    int64_t split = p.T >= want ? 1 : (want + p.T - 1) / p.T;
    if (split > most) split = most;
    const int64_t bx = p.T < 65536 ? p.T : 65536;
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(split));
    qk_direct_kernel<TA, LPH, ADJ, APPEND, NORM><<<grid, THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename TA, bool ADJ, bool APPEND, bool NORM>
cudaError_t launch_fwd(const QkParams& p, cudaStream_t s) {
    switch (lanes_per_head(p.Dh)) {
        case 8: return launch_fwd_lph<TA, 8, ADJ, APPEND, NORM>(p, s);
        case 16: return launch_fwd_lph<TA, 16, ADJ, APPEND, NORM>(p, s);
        case 32: return launch_fwd_lph<TA, 32, ADJ, APPEND, NORM>(p, s);
    }
    return cudaErrorNotSupported;
}
}  // namespace qk

}  // namespace mhc
