// paged_attn_tree.cu -- attention of trees of drafted tokens over a paged cache:
// the choice of kernel, and the CUDA-core kernel with TREE on.
//
// A sequence's new tokens are the nodes of a tree (or of a forest; any mask is
// taken), in any order.  Node i sees every cached token before the new ones, and
// of the new ones those whose bits its row of the mask has:
//   z_ij = scale <q_i, k_j> over those keys,  o_i = sum_j softmax(z_i)_j v_j.
// All nodes read the same context, so the tiles and the kernels are those of a
// causal chunk (with each CTA finding its own share: tree_share); only the blocks
// with drafted tokens differ: there a row's bits take the place of the diagonal, 32
// keys to a word, and values that no row of a tile sees are zeroed like those past a
// sequence's end.
//
// Tiles of trees have many rows, and a tile that is split over CTAs leaves a part
// of every row with each of them. The last CTA joining them by itself, a warp for
// 32 rows, takes longer than all of the rest when contexts are short (one sequence
// of 13 tokens and 777 keys: 22 of 35 us), so the joins are a kernel of their own,
// 16 lanes for each row.
//
// Figures, 40 + 8 heads of 128 in bf16 on one GB300: 32 sequences of 16 to 32 drafted
// tokens on up to 8192 cached ones 96 us, 25 on 8192 each 187 us (5.8 TB/s), 4 of 64 on
// 65536 330 to 338 us (their 320 rows of a key head are two tiles, which read the context
// twice, at 6.4 TB/s; 350 to 372 after thousands of calls in a row, when the power cap has
// brought the SM clock down to 1.7 GHz), one of 13 on 777 16 us.  float32, 20 + 4 heads, 8 of 11 on 3200:
// 115 us.
#include "paged_attn_cc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tree_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_error, word); }

namespace attn {

// Lanes of a row, rows that a warp has side by side, parts on their way together,
// blocks of a tile: with 4 blocks one sequence of 64 and 32768 takes 90 us, with 8 79,
// with 16 or 32 72; 8 parts together cost registers, and with them blocks of an SM.
constexpr int JOIN_THREADS = 128, JOIN_WARPS = JOIN_THREADS / 32, JOIN_LANES = 16, JOIN_ROWS = 32 / JOIN_LANES;
constexpr int JOIN_AHEAD = 4, JOIN_SPLIT = 16;

// N consecutive floats of a part, a multiple of 4.
template <int N> struct Floats {
    float v[N];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + i));
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        }
    }
    // From value `at` of a head of Dh, a multiple of 8, whose rest is not there.
    __device__ __forceinline__ void store(float* head, int at, int Dh) const {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            if (at + i < Dh) *reinterpret_cast<float4*>(head + at + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* head, int at, int Dh) const {
        uint32_t u[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        if constexpr (N == 4) {
            if (at < Dh) *reinterpret_cast<uint2*>(head + at) = make_uint2(u[0], u[1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 8)
                if (at + i < Dh)
                    *reinterpret_cast<uint4*>(head + at + i) = make_uint4(u[i / 2], u[i / 2 + 1], u[i / 2 + 2], u[i / 2 + 3]);
        }
    }
};

// Block (c, y): of the tile and head whose first part is CTA c's (a CTA has at
// most one such, its last piece), a share of the rows, two at a time for a warp.
// Lane j of a row takes the maximum and the sum of its j-th part, so that all weights
// come from one round of loads; then the lanes have DP/16 values of the row each and
// the parts are added in their order, JOIN_AHEAD of them on their way together.
// Bound by instructions as much as by reads: 16 sequences of 25 drafted and 8192 cached
// tokens took 12 us at half the issue rate with a row for all 32 lanes.
template <typename TA, int DP>
__global__ void __launch_bounds__(JOIN_THREADS, DP <= 128 ? 8 : 4)
tree_join_kernel(const AttnParams p) {
    constexpr int N = DP / JOIN_LANES;
    ptx::griddep_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % JOIN_LANES, side = lane / JOIN_LANES;
    const AttnStart* starts = attn_starts(p);
    const AttnStart& s = starts[c + 1];   // where this CTA's share ends
    if (s.begin >= s.end || s.unit <= p.plan.lead) return;   // no tile goes on there
    const int64_t u0 = s.t.start + static_cast<int64_t>(s.head) * (s.t.nblk + p.plan.lead) + p.plan.lead;
    const int first = c;
    if (starts[c].begin > u0) return;     // it began before
    // the CTA in whose share the tile's last block is; all between have blocks of it
    int last = c + 1;
    while (true) {
        const int j = last + lane;
        const unsigned ends = __ballot_sync(0xffffffffu, j >= p.plan.ncta || starts[min(j, p.plan.ncta - 1)].end >= u0 + s.t.nblk);
        if (ends != 0u) {
            last += __ffs(ends) - 1;
            break;
        }
        last += 32;
    }
    last = min(last, p.plan.ncta - 1);
    const int rows = min(p.plan.tile_rows, s.t.qlen * p.G - s.t.row0), sr = p.plan.slot_rows;
    // the tile's parts, from the second on two slots apart
    auto part = [&](int j) { return attn_slot(p, 2 * j + (j == first ? 1 : 0)); };
    for (int r0 = (blockIdx.y * JOIN_WARPS + warp) * JOIN_ROWS; r0 < rows; r0 += gridDim.y * JOIN_WARPS * JOIN_ROWS) {
        const int row = min(r0 + side, rows - 1);
        const int stat = sr * DP + row, mine = row * DP + sub * N;   // in a part: below 2^31
        float M = -INFINITY, l = 0.0f;
        Floats<N> a;
#pragma unroll
        for (int e = 0; e < N; ++e) a.v[e] = 0.0f;
        for (int c0 = first; c0 <= last; c0 += JOIN_LANES) {
            const int n = min(JOIN_LANES, last - c0 + 1);
            const float* st = part(c0 + min(sub, n - 1)) + stat;
            float w = sub < n ? __ldcg(st) : -INFINITY;
            const float pl = sub < n ? __ldcg(st + sr) : 0.0f;
            Floats<N> x[JOIN_AHEAD];
            auto fetch = [&](int j0) {
#pragma unroll
                for (int u = 0; u < JOIN_AHEAD; ++u)
                    if (j0 + u < n) x[u].load(part(c0 + j0 + u) + mine);
            };
            fetch(0);   // on their way with the weights
            float top = w;
#pragma unroll
            for (int o = JOIN_LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(top, M);
            const float base = top == -INFINITY ? 0.0f : top, keep = ex2(M - base);
            w = ex2(w - base);
            float sum = pl * w;
#pragma unroll
            for (int o = JOIN_LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = fmaf(l, keep, sum);
            M = top;
            if (c0 > first) {
#pragma unroll
                for (int e = 0; e < N; ++e) a.v[e] *= keep;
            }
            for (int j0 = 0; j0 < n; j0 += JOIN_AHEAD) {
                if (j0 > 0) fetch(j0);
#pragma unroll
                for (int u = 0; u < JOIN_AHEAD; ++u)
                    if (j0 + u < n) {
                        const float f = __shfl_sync(0xffffffffu, w, j0 + u, JOIN_LANES);
#pragma unroll
                        for (int e = 0; e < N; ++e) a.v[e] = fmaf(x[u].v[e], f, a.v[e]);
                    }
            }
        }
        if (r0 + side >= rows) continue;
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int r = s.t.row0 + row, tok = attn_token(p, r);
        const int64_t out = (s.t.q0 + tok) * p.Hq + s.head * p.G + (r - tok * p.G);
#pragma unroll
        for (int e = 0; e < N; ++e) a.v[e] *= inv;
        a.store(static_cast<TA*>(p.o) + out * p.Dh, sub * N, p.Dh);
        if (sub == 0 && p.lse != nullptr) p.lse[out] = attn_lse(M, l);
    }
}

template <typename TA>
cudaError_t launch_tree_join(const AttnParams& p, cudaStream_t s) {
    if (p.plan.ncta < 2) return cudaSuccess;
    const int most = (p.plan.slot_rows + JOIN_WARPS * JOIN_ROWS - 1) / (JOIN_WARPS * JOIN_ROWS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.plan.ncta - 1), static_cast<unsigned>(most < JOIN_SPLIT ? most : JOIN_SPLIT));
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.Dh <= 64) return cudaLaunchKernelEx(&cfg, tree_join_kernel<TA, 64>, p);
    if (p.Dh <= 128) return cudaLaunchKernelEx(&cfg, tree_join_kernel<TA, 128>, p);
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<TA, 256>, p);
}

}  // namespace attn

cudaError_t launch_tree_attn(bool bf16, const AttnParams& p, cudaStream_t s) {
    cudaError_t e;
    if (attn_tc_supports(bf16, p.Hq, p.Hk, p.Dh, p.page_size)) {
        e = launch_tree_attn_tc(p, s);
        if (p.force_timeout != 0u) return e;   // a forced timeout leaves no shares to join
    } else {   // (nothing waits here: the hook has nothing to run out)
        g_error_word.may_be_set();
        e = bf16 ? attn::launch_cc_dp<__nv_bfloat16, true>(p, s) : attn::launch_cc_dp<float, true>(p, s);
    }
    if (e != cudaSuccess) return e;
    return bf16 ? attn::launch_tree_join<__nv_bfloat16>(p, s) : attn::launch_tree_join<float>(p, s);
}

}  // namespace mhc
