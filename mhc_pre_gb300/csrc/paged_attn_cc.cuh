// paged_attn_cc.cuh -- attention over a paged cache on the CUDA cores, for causal
// rows (paged_attn.cu) and for trees of drafted tokens (TREE, paged_attn_tree.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace mhc {

// Each translation unit has its own word: ATTN_ERR_* bits.
static __device__ unsigned g_attn_error;

namespace attn {

// ------------------------------------------------------------ CUDA cores ---
//
// TY x 16 threads: thread (ty, tx) has the rows ty, ty + TY, ... of the tile and
// keys tx, tx + 16, ... of a block for the scores, and the columns
// 4 tx + 64 c of the values for the sums; a row's maximum and sum live in the
// 16 lanes that share the row.  Those are every other lane of a warp, which has
// two rows at a time: 16-byte reads of shared memory take 2 cycles a warp where
// neighbouring lanes share an address, and 4 where only lanes 16 apart do (a
// chunk of 1024 tokens on 4096 keys in float32: 896 us, 960 with rows in half
// warps).  Products go through packed pairs of float32
// (pairs along d for the scores, of columns for the sums): a register tile of
// 4 x 4 then has more arithmetic than shared-memory reads.  Keys and values
// come by asynchronous copies, each while the other is being multiplied.
// Bound by float32 arithmetic and the reads of the register tile from shared
// memory, which take about as long as each other: that chunk, of 20 + 4 heads of
// 128, takes 883 us, 42.6 TFLOP/s of the products that the mask leaves; 6
// sequences of up to 300 new tokens and 2000 keys 216 us; one new token for each
// of 64 sequences of up to 8192 keys (20 + 4 heads) 320 us, 2.4 TB/s.
constexpr int CC_KEYS = 64, CC_KPT = CC_KEYS / 16;

template <typename TA>
__device__ __forceinline__ float4 ld4(const TA* p) {
    if (sizeof(TA) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    }
    return *reinterpret_cast<const float4*>(p);
}

// Elements of a row of keys or values: 16 bytes more than its values, so that
// the rows of 8 neighbouring threads lie in different banks.
template <typename TA> __host__ __device__ constexpr int cc_pitch(int dp) { return dp + 16 / static_cast<int>(sizeof(TA)); }
constexpr int CC_PP = CC_KEYS + 4;   // floats of a row of exponentials
template <typename TA>
constexpr size_t cc_smem(int dp, int rows) {
    return sizeof(float) * static_cast<size_t>(rows) * (dp + 4 + CC_PP) + sizeof(TA) * 2u * CC_KEYS * cc_pitch<TA>(dp);
}

// Starts the copy of one block of keys or values; what lies outside [lo, hi)
// becomes zeros, whatever the pages hold there, and so do a tree's tokens that no
// row of the tile sees (`drafted`: those that some row does).
template <typename TA, int DP, int TY, bool TREE>
__device__ __forceinline__ void cc_copy(const AttnParams& p, const AttnPiece& pc, const uint32_t* drafted, TA* dst,
                                        const void* cache, int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                                        int k0, int tid) {
    constexpr int PER = 16 / static_cast<int>(sizeof(TA)), CPR = DP / PER;   // values of a copy, copies of a row
    constexpr int ROWS = TY * 16 / CPR, PASSES = CC_KEYS / ROWS;
    static_assert(ROWS * PASSES == CC_KEYS, "the threads copy whole rows");
    const int d = (tid % CPR) * PER;
    int page[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int key = k0 + i * ROWS + tid / CPR;
        page[i] = -1;
        bool seen = key >= pc.lo && key < pc.hi && d < p.Dh;
        if (TREE) {
            const int node = key - (pc.kvlen - pc.qlen);
            if (seen && node >= 0) seen = drafted[node >> 5] >> (node & 31) & 1u;
        }
        if (seen) {
            const int pg = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
            page[i] = p.page_table[pc.seq * p.table_stride + pg];
            if (page[i] < 0 || page[i] >= p.num_pages) {
                atomicOr(&g_attn_error, ATTN_ERR_RANGE);
                page[i] = -1;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = i * ROWS + tid / CPR, key = k0 + row;
        const int in = p.page_shift >= 0 ? key & (p.page_size - 1) : key % p.page_size;
        const TA* src = static_cast<const TA*>(cache);
        if (page[i] >= 0) src += page[i] * page_stride + in * slot_stride + pc.head * head_stride + d;
        ptx::cp_async16(ptx::smem_u32(dst + row * cc_pitch<TA>(DP) + d), src, page[i] >= 0 ? 16u : 0u);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// One piece of a tile of at most TY RPT rows.
template <typename TA, int DP, int TY, int RPT, bool TREE>
__device__ __forceinline__ void cc_piece(const AttnParams& p, const AttnPiece& pc, float* Qs, float* Ps, TA* Ks, TA* Vs,
                                         int* s_last, uint32_t* drafted) {
    constexpr int QP = DP + 4, PITCH = cc_pitch<TA>(DP), NC = DP / 64, PP = CC_PP;
    const int tid = threadIdx.x, tx = (tid >> 1) & 15, ty = (tid >> 5) * 2 + (tid & 1);
    const float zscale = p.scale * LOG2E;
    const float cap_in = p.softcap > 0.0f ? p.scale / p.softcap : 0.0f;
    const int nrows = pc.qlen * p.G;
    auto copy_k = [&](int b) {
        cc_copy<TA, DP, TY, TREE>(p, pc, drafted, Ks, p.k_cache, p.k_page_stride, p.k_slot_stride, p.k_head_stride,
                        (pc.blk + b) * CC_KEYS, tid);
    };
    auto copy_v = [&](int b) {
        cc_copy<TA, DP, TY, TREE>(p, pc, drafted, Vs, p.v_cache, p.v_page_stride, p.v_slot_stride, p.v_head_stride,
                        (pc.blk + b) * CC_KEYS, tid);
    };
    if (TREE) {
        // the tokens of the tree that some row of the tile sees
        const int words = (pc.qlen + 31) / 32, tok0 = attn_token(p, pc.row0);
        const int tok1 = attn_token(p, min(pc.row0 + TY * RPT, nrows) - 1);
        for (int w = tid >> 5; w < words; w += TY / 2) {
            uint32_t bits = 0u;
            for (int t = tok0 + (tid & 31); t <= tok1; t += 32) {
                AttnNode n;
                n.words = p.tree + (pc.q0 + t) * p.tree_stride;
                n.nodes = pc.qlen;
                bits |= n.word(w);
            }
            bits = __reduce_or_sync(0xffffffffu, bits);
            if ((tid & 31) == 0) drafted[w] = bits;
        }
        __syncthreads();
    }
    copy_k(0);
    copy_v(0);
    // the tile's queries
    for (int i = tid; i < TY * RPT * (DP / 4); i += TY * 16) {
        const int row = i / (DP / 4), d = (i - row * (DP / 4)) * 4, r = pc.row0 + row;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nrows && d < p.Dh) {
            const int tok = attn_token(p, r);
            v = ld4(static_cast<const TA*>(p.q) + (pc.q0 + tok) * p.q_stride +
                    static_cast<int64_t>(pc.head * p.G + r - tok * p.G) * p.Dh + d);
        }
        *reinterpret_cast<float4*>(Qs + row * QP + d) = v;
    }
    int lo[RPT], hi[RPT];   // of a tree: the keys that the row sees are those and some from hi on
    float m[RPT], l[RPT];
    float2 acc[RPT][NC][2];
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
        const int r = pc.row0 + ty + TY * a;
        lo[a] = hi[a] = 0;
        if (r < nrows && !TREE) attn_token_keys(pc, attn_token(p, r), p.window, lo[a], hi[a]);
        if (r < nrows && TREE) {
            AttnNode n;
            n.init(p, pc, attn_token(p, r));
            lo[a] = n.lo;
            hi[a] = max(0, n.ctx);
        }
        m[a] = -INFINITY;
        l[a] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[a][c][0] = acc[a][c][1] = make_float2(0.0f, 0.0f);
    }
    for (int b = 0; b < pc.nb; ++b) {
        const int k0 = (pc.blk + b) * CC_KEYS;
        const bool more = b + 1 < pc.nb;
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys; the values may still come
        __syncthreads();
        float2 s2[RPT][CC_KPT];
#pragma unroll
        for (int a = 0; a < RPT; ++a)
#pragma unroll
            for (int j = 0; j < CC_KPT; ++j) s2[a][j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int d = 0; d < DP; d += 4) {
            float4 kv[CC_KPT];
#pragma unroll
            for (int j = 0; j < CC_KPT; ++j) kv[j] = ld4(Ks + (tx + 16 * j) * PITCH + d);
#pragma unroll
            for (int a = 0; a < RPT; ++a) {
                const float4 qv = *reinterpret_cast<const float4*>(Qs + (ty + TY * a) * QP + d);
#pragma unroll
                for (int j = 0; j < CC_KPT; ++j) {
                    s2[a][j] = __ffma2_rn(make_float2(qv.x, qv.y), make_float2(kv[j].x, kv[j].y), s2[a][j]);
                    s2[a][j] = __ffma2_rn(make_float2(qv.z, qv.w), make_float2(kv[j].z, kv[j].w), s2[a][j]);
                }
            }
        }
        __syncthreads();
        if (more) copy_k(b + 1);
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
            float s[CC_KPT], mx = m[a];
            uint32_t node[2] = {0u, 0u};   // which of the block's keys the row sees as drafted tokens
            if (TREE && k0 + CC_KEYS > hi[a] && pc.row0 + ty + TY * a < nrows) {
                AttnNode n;
                n.words = p.tree + (pc.q0 + attn_token(p, pc.row0 + ty + TY * a)) * p.tree_stride;
                n.ctx = pc.kvlen - pc.qlen;
                n.nodes = n.ctx >= 0 ? pc.qlen : 0;
                n.drafted(k0, node);
            }
#pragma unroll
            for (int j = 0; j < CC_KPT; ++j) {
                const int key = k0 + tx + 16 * j;
                const float x = s2[a][j].x + s2[a][j].y;
                const float z = p.softcap > 0.0f ? p.softcap * LOG2E * tanhf(x * cap_in) : x * zscale;
                bool seen = key >= lo[a] && key < hi[a];
                if (TREE) seen = seen || (node[j >> 1] >> (tx + 16 * (j & 1)) & 1u);
                s[j] = seen ? z : -INFINITY;
                mx = fmaxf(mx, s[j]);
            }
#pragma unroll
            for (int o = 16; o > 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float base = mx > -INFINITY ? mx : 0.0f;
            const float keep = exp2f(m[a] - base);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < CC_KPT; ++j) {
                const float e = exp2f(s[j] - base);
                sum += e;
                Ps[(ty + TY * a) * PP + tx + 16 * j] = e;
            }
#pragma unroll
            for (int o = 16; o > 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[a] = fmaf(l[a], keep, sum);
            m[a] = mx;
            const float2 keep2 = make_float2(keep, keep);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                acc[a][c][0] = __fmul2_rn(acc[a][c][0], keep2);
                acc[a][c][1] = __fmul2_rn(acc[a][c][1], keep2);
            }
        }
        if (more) asm volatile("cp.async.wait_group 1;" ::: "memory");   // the values; the next keys may still come
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < CC_KEYS; k += 4) {
            float4 pr[RPT];
#pragma unroll
            for (int a = 0; a < RPT; ++a) pr[a] = *reinterpret_cast<const float4*>(Ps + (ty + TY * a) * PP + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 v = ld4(Vs + (k + kk) * PITCH + tx * 4 + 64 * c);
#pragma unroll
                    for (int a = 0; a < RPT; ++a) {
                        const float w = kk == 0 ? pr[a].x : kk == 1 ? pr[a].y : kk == 2 ? pr[a].z : pr[a].w;
                        acc[a][c][0] = __ffma2_rn(make_float2(w, w), make_float2(v.x, v.y), acc[a][c][0]);
                        acc[a][c][1] = __ffma2_rn(make_float2(w, w), make_float2(v.z, v.w), acc[a][c][1]);
                    }
                }
            }
        }
        __syncthreads();
        if (more) copy_v(b + 1);
    }
    if (pc.whole) {
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
            const int r = pc.row0 + ty + TY * a;
            if (r >= nrows) continue;
            const float inv = l[a] != 0.0f ? 1.0f / l[a] : 0.0f;
            const int tok = attn_token(p, r);
            const int64_t out = (pc.q0 + tok) * p.Hq + pc.head * p.G + (r - tok * p.G);
            TA* o = static_cast<TA*>(p.o) + out * p.Dh;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = tx * 4 + 64 * c;
                if (d >= p.Dh) continue;
                if (sizeof(TA) == 2) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[a][c][0].x * inv, acc[a][c][0].y * inv);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[a][c][1].x * inv, acc[a][c][1].y * inv);
                    *reinterpret_cast<uint2*>(o + d) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                                                  *reinterpret_cast<const uint32_t*>(&y));
                } else {
                    *reinterpret_cast<float4*>(o + d) = make_float4(acc[a][c][0].x * inv, acc[a][c][0].y * inv,
                                                                    acc[a][c][1].x * inv, acc[a][c][1].y * inv);
                }
            }
            if (tx == 0 && p.lse != nullptr) p.lse[out] = attn_lse(m[a], l[a]);
        }
    } else {
        float* s = attn_slot(p, pc.slot);
        const int sr = p.plan.slot_rows;
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
            const int row = ty + TY * a;
            if (pc.row0 + row >= nrows) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<float4*>(s + static_cast<int64_t>(row) * DP + tx * 4 + 64 * c) =
                    make_float4(acc[a][c][0].x, acc[a][c][0].y, acc[a][c][1].x, acc[a][c][1].y);
            if (tx == 0) {
                s[static_cast<int64_t>(sr) * DP + row] = m[a];
                s[static_cast<int64_t>(sr) * (DP + 1) + row] = l[a];
            }
        }
        if constexpr (TREE) return;   // joined by a kernel of their own (paged_attn_tree.cu)
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            const int n = atomicAdd(attn_counts(p) + pc.cnt, 1);
            *s_last = n == pc.last_cta - pc.first_cta;
            // the counter is back at zero for the next call with this plan
            if (*s_last) attn_counts(p)[pc.cnt] = 0;
            __threadfence();
        }
        __syncthreads();
        if (*s_last) {
            const int rows = min(p.plan.tile_rows, nrows - pc.row0), each = (rows + TY / 2 - 1) / (TY / 2), begin = (tid >> 5) * each;
            attn_join<TA, DP, 4, 2>(p, pc, begin, min(rows, begin + each), tid & 31);
        }
    }
}

// Tiles of up to TY RPT rows; one of at most TY (a sequence that decodes, in a
// batch with chunks) takes the code that has no other rows.
template <typename TA, int DP, int TY, int RPT, bool TREE>
__global__ void __launch_bounds__(TY * 16)
attn_cc_kernel(const AttnParams p) {
    extern __shared__ __align__(16) float smem_f[];
    float* Qs = smem_f;
    float* Ps = Qs + TY * RPT * (DP + 4);
    TA* Ks = reinterpret_cast<TA*>(Ps + TY * RPT * CC_PP);
    TA* Vs = Ks + CC_KEYS * cc_pitch<TA>(DP);
    __shared__ int s_last;
    __shared__ uint32_t s_drafted[TREE ? TREE_MOST / 32 : 1];
    const int cta = blockIdx.x;
    if (TREE) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    AttnWalk walk;
    if constexpr (TREE) {
        __shared__ TreeShare share;
        // a block of 64 keys takes longer than the joins, and about as long with fewer rows
        tree_share<TY * 16>(p, cta, {1, 0, 1, 1}, share, &g_attn_error);
        if (!walk.begin(share.start)) return;
    } else {
        if (!attn_plan_agrees(p)) {
            if (threadIdx.x == 0) atomicOr(&g_attn_error, ATTN_ERR_RANGE);
            return;
        }
        if (!walk.begin(p, cta)) return;
    }
    AttnPiece pc;
    while (walk.next<TREE>(p, cta, pc)) {
        const int rows = pc.qlen * p.G - pc.row0;
        if (RPT > 1 && rows <= TY) cc_piece<TA, DP, TY, 1, TREE>(p, pc, Qs, Ps, Ks, Vs, &s_last, s_drafted);
        else if (TREE && RPT > 2 && rows <= 2 * TY) cc_piece<TA, DP, TY, 2, TREE>(p, pc, Qs, Ps, Ks, Vs, &s_last, s_drafted);
        else if (TREE && RPT > 3 && rows <= 3 * TY) cc_piece<TA, DP, TY, 3, TREE>(p, pc, Qs, Ps, Ks, Vs, &s_last, s_drafted);
        else cc_piece<TA, DP, TY, RPT, TREE>(p, pc, Qs, Ps, Ks, Vs, &s_last, s_drafted);
        __syncthreads();
    }
}

// cudaFuncSetAttribute once per device and kernel (idempotent, so a race is harmless).
inline cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

template <typename TA, int DP, int TY, int RPT, bool TREE>
cudaError_t launch_cc(const AttnParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = cc_smem<TA>(DP, TY * RPT);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_cc_kernel<TA, DP, TY, RPT, TREE>), done, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.plan.ncta));
    cfg.blockDim = dim3(TY * 16);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_cc_kernel<TA, DP, TY, RPT, TREE>, p);
}

template <typename TA, bool TREE>
cudaError_t launch_cc_dp(const AttnParams& p, cudaStream_t s) {
    const bool small = p.plan.tile_rows == 16;
    if (p.Dh <= 64) return small ? launch_cc<TA, 64, 16, 1, TREE>(p, s) : launch_cc<TA, 64, 32, 4, TREE>(p, s);
    if (p.Dh <= 128) return small ? launch_cc<TA, 128, 16, 1, TREE>(p, s) : launch_cc<TA, 128, 32, 4, TREE>(p, s);
    return small ? launch_cc<TA, 256, 16, 1, TREE>(p, s) : launch_cc<TA, 256, 32, 2, TREE>(p, s);
}

}  // namespace attn
}  // namespace mhc
