// paged_attn_tree.cu -- attention of trees of drafted tokens over a paged cache:
// the choice of kernel, and the CUDA-core kernel with TREE on.
//
// A sequence's new tokens are the nodes of a tree (or of a forest; any mask is
// taken), in any order.  Node i sees every cached token before the new ones, and
// of the new ones those whose bits its row of the mask has:
//   z_ij = scale <q_i, k_j> over those keys,  o_i = sum_j softmax(z_i)_j v_j.
// All nodes read the same context, so the tiles and the kernels are those of a
// causal chunk (with each CTA finding its own share: tree_share); only the blocks with drafted tokens differ: there a
// row's bits take the place of the diagonal, 32 keys to a word, and values that no
// row of a tile sees are zeroed like those past a sequence's end.
//
// Tiles of trees have many rows, and a tile that is split over CTAs leaves a part
// of every row with each of them. The last CTA joining them by itself, a warp for
// 32 rows, takes longer than all of the rest when contexts are short (one sequence
// of 13 tokens and 777 keys: 22 of 35 us), so the joins are a kernel of their own,
// a warp for each row.
#include "paged_attn_cc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tree_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_error, word); }

namespace attn {

// Rows that a warp has on their way together, parts of each, blocks of a tile.  Of
// 1 and 2 rows with 4, 8 and 16 parts and 4 to 32 blocks these are within 3 % of the
// best for 11 batches of all kinds; 8 parts or more cost registers, and with them
// blocks of an SM (2 rows, 8 parts: 104 -> 111 us for 32 sequences of up to 8192),
// 4 blocks of a tile leave too little in flight (37 -> 87 us in the worst case).
constexpr int JOIN_THREADS = 128, JOIN_WARPS = JOIN_THREADS / 32, JOIN_ROWS = 2, JOIN_AHEAD = 4, JOIN_SPLIT = 16;

// N consecutive floats of a part.
template <int N> struct Floats {
    float v[N];
    __device__ __forceinline__ void load(const float* p) {
        if constexpr (N == 2) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
            v[0] = x.x;
            v[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p + i));
                v[i] = x.x;
                v[i + 1] = x.y;
                v[i + 2] = x.z;
                v[i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void store(float* p) const {
        if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
        else
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        uint32_t u[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = u[0];
        else if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
        else *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// Block (c, y): of the tile and head whose first part is CTA c's (a CTA has at
// most one such, its last piece), a share of the rows, JOIN_ROWS at a time for a
// warp.  Lane j takes the maximum and the sum of the j-th part, so that all weights
// come from one round of loads; then the lanes have DP/32 values of each row and
// the parts are added in their order, JOIN_AHEAD of them on their way together.
template <typename TA, int DP>
__global__ void __launch_bounds__(JOIN_THREADS, DP <= 128 ? 8 : 4)
tree_join_kernel(const AttnParams p) {
    constexpr int N = DP / 32, R = JOIN_ROWS;
    ptx::griddep_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AttnStart& s = attn_starts(p)[c + 1];   // where this CTA's share ends
    if (s.begin >= s.end || s.unit <= p.plan.lead) return;   // no tile goes on there
    const int64_t per = attn_head(p)->per_cta;
    const int64_t u0 = s.t.start + static_cast<int64_t>(s.head) * (s.t.nblk + p.plan.lead) + p.plan.lead;
    const int first = tree_divide(u0, per), last = tree_divide(u0 + s.t.nblk - 1, per);
    if (first != c || last == first) return;
    const int rows = min(p.plan.tile_rows, s.t.qlen * p.G - s.t.row0), sr = p.plan.slot_rows;
    auto part = [&](int j) { return attn_slot(p, 2 * j + (j == first ? 1 : 0)); };
    for (int r0 = (blockIdx.y * JOIN_WARPS + warp) * R; r0 < rows; r0 += gridDim.y * JOIN_WARPS * R) {
        float M[R], l[R];
        Floats<N> a[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            M[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) a[i].v[e] = 0.0f;
        }
        for (int c0 = first; c0 <= last; c0 += 32) {
            const int n = min(32, last - c0 + 1);
            const float* stat = part(c0 + min(lane, n - 1)) + static_cast<int64_t>(sr) * DP;
            float w[R], pl[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = min(r0 + i, rows - 1);
                w[i] = lane < n ? __ldcg(stat + row) : -INFINITY;
                pl[i] = lane < n ? __ldcg(stat + sr + row) : 0.0f;
            }
            Floats<N> x[JOIN_AHEAD][R];
            auto fetch = [&](int j0) {
#pragma unroll
                for (int u = 0; u < JOIN_AHEAD; ++u) {
                    const float* base = part(c0 + min(j0 + u, n - 1)) + lane * N;
#pragma unroll
                    for (int i = 0; i < R; ++i) x[u][i].load(base + static_cast<int64_t>(min(r0 + i, rows - 1)) * DP);
                }
            };
            fetch(0);   // on their way with the weights
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float top = w[i];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = fmaxf(top, M[i]);
                const float base = top == -INFINITY ? 0.0f : top, keep = ex2(M[i] - base);
                w[i] = ex2(w[i] - base);
                l[i] = fmaf(l[i], keep, warp_sum(pl[i] * w[i]));
                M[i] = top;
#pragma unroll
                for (int e = 0; e < N; ++e) a[i].v[e] *= keep;
            }
            for (int j0 = 0; j0 < n; j0 += JOIN_AHEAD) {
                if (j0 > 0) fetch(j0);
#pragma unroll
                for (int u = 0; u < JOIN_AHEAD; ++u)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float f = __shfl_sync(0xffffffffu, w[i], min(j0 + u, 31));
                        if (j0 + u < n)
#pragma unroll
                            for (int e = 0; e < N; ++e) a[i].v[e] = fmaf(x[u][i].v[e], f, a[i].v[e]);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (r0 + i >= rows) break;
            const float inv = l[i] != 0.0f ? 1.0f / l[i] : 0.0f;
            const int r = s.t.row0 + r0 + i, tok = attn_token(p, r);
            const int64_t out = (s.t.q0 + tok) * p.Hq + s.head * p.G + (r - tok * p.G);
#pragma unroll
            for (int e = 0; e < N; ++e) a[i].v[e] *= inv;
            if (lane * N < p.Dh) a[i].store(static_cast<TA*>(p.o) + out * p.Dh + lane * N);   // heads are multiples of 8
            if (lane == 0 && p.lse != nullptr) p.lse[out] = attn_lse(M[i], l[i]);
        }
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
    } else {
        g_error_word.may_be_set();
        e = bf16 ? attn::launch_cc_dp<__nv_bfloat16, true>(p, s) : attn::launch_cc_dp<float, true>(p, s);
    }
    // (a forced timeout leaves no shares to join)
    if (e != cudaSuccess || p.force_timeout != 0u) return e;
    return bf16 ? attn::launch_tree_join<__nv_bfloat16>(p, s) : attn::launch_tree_join<float>(p, s);
}

}  // namespace mhc
