// paged_attn.cu -- attention of a chunk of new tokens over a paged cache: the
// plan kernel, the CUDA-core kernel, and the choice of kernel.
//
//   z[i, j] = scale <q_i, k_j>,  z = softcap tanh(z / softcap) when capped,
//   keys j <= kvlen - qlen + i, and j > kvlen - qlen + i - window,
//   o_i = sum_j exp(z_ij - lse_i) v_j,  lse_i = log sum_j exp(z_ij);
// a row that sees no key gives o = 0 and lse = -inf.
//
// bf16 heads of at most 128 over pages that divide (or are a multiple of) 128
// keys run on the tensor cores (paged_attn_tc.cu).  Everything else (float32,
// wider heads, other page sizes) runs in attn_cc_kernel below, which keeps a
// tile's scores and sums in registers and walks the keys once.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace mhc {

__device__ unsigned g_attn_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_error, word); }

namespace attn {

constexpr int PLAN_THREADS = 512;   // also at least PLAN_CTAS
constexpr int PLAN_NEAR = 256;      // whole tiles kept there for the borders (12 KB)
constexpr int SMALL_TILE = 8;       // tiles below 1/8 of a CTA's share are not split
constexpr int PLAN_CTAS = 512;      // most CTAs of a launch
constexpr int PLAN_TILES = 2048;    // tile starts kept in shared memory for the CTAs' search

struct PlanParams {
    const int32_t *cu_q, *kv_lens;
    unsigned char* ws;
    int64_t T;
    int64_t max_kv;
    int B, Hq, Hk, G, window, max_q;
    AttnPlan plan;
};

// Exclusive sum over the block; `total` is the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < PLAN_THREADS / 32; ++i) {
        const int64_t s = warp_sums[i];
        if (i < w) before += s;
        all += s;
    }
    total = all;
    return before + x - v;
}

// One block: tiles of every sequence, their first units, and each CTA's start.
// A chain of reads, scans and writes: 4.4 us for one sequence, 5.0 for 64, 6.4
// for 5 prompts of 269 tiles.  The first tiles stay in shared memory too, so that
// a CTA's border costs no read of what has just been written.
__global__ void __launch_bounds__(PLAN_THREADS)
attn_plan_kernel(const PlanParams p) {
    __shared__ int64_t sums[PLAN_THREADS / 32];
    __shared__ int tile_base[PLAN_THREADS];
    __shared__ int s_q0[PLAN_THREADS], s_qlen[PLAN_THREADS], s_kvlen[PLAN_THREADS];
    __shared__ int64_t s_start[PLAN_TILES];
    __shared__ AttnTile s_tile[PLAN_NEAR];   // the first tiles again, for the borders
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x;
    AttnTile* tiles = reinterpret_cast<AttnTile*>(p.ws + p.plan.tile_off);
    int* counts = reinterpret_cast<int*>(p.ws + p.plan.count_off);
    const int TR = p.plan.tile_rows, BN = p.plan.block_keys;
    int64_t units = 0;
    int ntiles = 0;
    for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        int q0 = 0, qlen = 0, kvlen = 0;
        if (b < p.B) {
            q0 = p.cu_q[b];
            qlen = p.cu_q[b + 1] - q0;
            kvlen = p.kv_lens[b];
            // a sequence whose numbers do not fit the call is left out
            if (q0 < 0 || qlen < 0 || qlen > p.max_q || q0 + static_cast<int64_t>(qlen) > p.T || kvlen < 0 ||
                kvlen > p.max_kv) {
                atomicOr(&g_attn_error, ATTN_ERR_RANGE);
                qlen = 0;
                kvlen = 0;
            }
        }
        const int nt = (qlen * p.G + TR - 1) / TR;
        int64_t all = 0;
        const int64_t base = block_scan(nt, sums, all);
        // sequences of a call have at most max_tiles tiles unless their rows overlap
        const int64_t room = p.plan.max_tiles - ntiles;
        if (all > room) {
            if (tid == 0) atomicOr(&g_attn_error, ATTN_ERR_RANGE);
            all = room;
        }
        tile_base[tid] = static_cast<int>(min(base, room));
        s_q0[tid] = q0;
        s_qlen[tid] = qlen;
        s_kvlen[tid] = kvlen;
        __syncthreads();
        for (int t0 = 0; t0 < all; t0 += PLAN_THREADS) {
            const int i = t0 + tid;
            const bool on = i < all;
            AttnTile t = {};
            if (on) {
                // the sequence of tile i: the last one whose base is at most i
                int lo = 0, hi = PLAN_THREADS - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (tile_base[mid] <= i) lo = mid;
                    else hi = mid - 1;
                }
                t.seq = b0 + lo;
                t.q0 = s_q0[lo];
                t.qlen = s_qlen[lo];
                t.kvlen = s_kvlen[lo];
                t.row0 = (i - tile_base[lo]) * TR;
                const int last = min(t.row0 + TR, t.qlen * p.G) - 1;
                int lo_k, hi_k, unused;
                attn_token_keys(t, t.row0 / p.G, p.window, lo_k, unused);
                attn_token_keys(t, last / p.G, p.window, unused, hi_k);
                // rows that see nothing still get their zeros written: one masked block
                t.blk0 = hi_k > lo_k ? lo_k / BN : 0;
                t.nblk = hi_k > lo_k ? (hi_k + BN - 1) / BN - t.blk0 : 1;
                t.cnt = (ntiles + i) * p.Hk;
            }
            int64_t sum = 0;
            t.start = units + block_scan(on ? static_cast<int64_t>(t.nblk + p.plan.lead) * p.Hk : 0, sums, sum);
            units += sum;
            if (on) {
                tiles[ntiles + i] = t;
                if (ntiles + i < PLAN_TILES) s_start[ntiles + i] = t.start;
                if (ntiles + i < PLAN_NEAR) s_tile[ntiles + i] = t;
            }
        }
        ntiles += static_cast<int>(all);
        __syncthreads();
    }
    for (int64_t i = tid; i < static_cast<int64_t>(ntiles) * p.Hk * (JOINS / 4); i += PLAN_THREADS)
        reinterpret_cast<int4*>(counts)[i] = make_int4(0, 0, 0, 0);
    int64_t per = (units + p.plan.ncta - 1) / p.plan.ncta;
    if (per < 1) per = 1;
    if (tid == 0) {
        AttnHead* h = reinterpret_cast<AttnHead*>(p.ws);
        h->per_cta = per;
        h->T = p.T;
        h->max_q = p.max_q;
        h->max_kv = p.max_kv;
        h->ntiles = ntiles;
        h->ncta = p.plan.ncta;
        h->Hq = p.Hq;
        h->Hk = p.Hk;
        h->B = p.B;
        h->tile_rows = TR;
        h->block_keys = BN;
        h->window = p.window;
        h->lead = p.plan.lead;
        h->spent = 0;
    }
    AttnStart* starts = reinterpret_cast<AttnStart*>(p.ws + p.plan.start_off);
    // The border at unit u: moved to the nearer end of a small tile (of one key
    // head), and where it lies.
    auto border = [&](int64_t u, AttnStart& s) {
        if (u >= units) return units;
        int lo = 0, hi = ntiles - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            const int64_t st = mid < PLAN_TILES ? s_start[mid] : tiles[mid].start;
            if (st <= u) lo = mid;
            else hi = mid - 1;
        }
        s.t = lo < PLAN_NEAR ? s_tile[lo] : tiles[lo];
        const int cost = s.t.nblk + p.plan.lead;
        const int64_t in = u - s.t.start;
        s.tile = lo;
        s.head = static_cast<int>(in / cost);
        s.unit = static_cast<int>(in - static_cast<int64_t>(s.head) * cost);
        if (s.unit > 0 && cost * SMALL_TILE <= per) {
            if (2 * s.unit < cost) {
                u -= s.unit;
            } else {
                u += cost - s.unit;
                if (++s.head == p.Hk && u < units) {
                    s.head = 0;
                    ++s.tile;
                    s.t = s.tile < PLAN_NEAR ? s_tile[s.tile] : tiles[s.tile];
                }
            }
            s.unit = 0;
        }
        return u;
    };
    __shared__ int64_t s_begin[PLAN_CTAS + 1];
    AttnStart s = {};
    if (tid < p.plan.ncta) s_begin[tid] = s.begin = border(tid * per, s);
    if (tid == 0) s_begin[p.plan.ncta] = units;
    __syncthreads();
    if (tid < p.plan.ncta) {
        s.end = s_begin[tid + 1];
        starts[tid] = s;
    }
}

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
// becomes zeros, whatever the pages hold there.
template <typename TA, int DP, int TY>
__device__ __forceinline__ void cc_copy(const AttnParams& p, const AttnPiece& pc, TA* dst, const void* cache,
                                        int64_t page_stride, int64_t slot_stride, int64_t head_stride, int k0, int tid) {
    constexpr int PER = 16 / static_cast<int>(sizeof(TA)), CPR = DP / PER;   // values of a copy, copies of a row
    constexpr int ROWS = TY * 16 / CPR, PASSES = CC_KEYS / ROWS;
    static_assert(ROWS * PASSES == CC_KEYS, "the threads copy whole rows");
    const int d = (tid % CPR) * PER;
    int page[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int key = k0 + i * ROWS + tid / CPR;
        page[i] = -1;
        if (key >= pc.lo && key < pc.hi && d < p.Dh) {
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
template <typename TA, int DP, int TY, int RPT>
__device__ __forceinline__ void cc_piece(const AttnParams& p, const AttnPiece& pc, float* Qs, float* Ps, TA* Ks, TA* Vs,
                                         int* s_last) {
    constexpr int QP = DP + 4, PITCH = cc_pitch<TA>(DP), NC = DP / 64, PP = CC_PP;
    const int tid = threadIdx.x, tx = (tid >> 1) & 15, ty = (tid >> 5) * 2 + (tid & 1);
    const float zscale = p.scale * LOG2E;
    const float cap_in = p.softcap > 0.0f ? p.scale / p.softcap : 0.0f;
    const int nrows = pc.qlen * p.G;
    auto copy_k = [&](int b) {
        cc_copy<TA, DP, TY>(p, pc, Ks, p.k_cache, p.k_page_stride, p.k_slot_stride, p.k_head_stride,
                        (pc.blk + b) * CC_KEYS, tid);
    };
    auto copy_v = [&](int b) {
        cc_copy<TA, DP, TY>(p, pc, Vs, p.v_cache, p.v_page_stride, p.v_slot_stride, p.v_head_stride,
                        (pc.blk + b) * CC_KEYS, tid);
    };
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
    int lo[RPT], hi[RPT];
    float m[RPT], l[RPT];
    float2 acc[RPT][NC][2];
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
        const int r = pc.row0 + ty + TY * a;
        lo[a] = hi[a] = 0;
        if (r < nrows) attn_token_keys(pc, attn_token(p, r), p.window, lo[a], hi[a]);
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
#pragma unroll
            for (int j = 0; j < CC_KPT; ++j) {
                const int key = k0 + tx + 16 * j;
                const float x = s2[a][j].x + s2[a][j].y;
                const float z = p.softcap > 0.0f ? p.softcap * LOG2E * tanhf(x * cap_in) : x * zscale;
                s[j] = key >= lo[a] && key < hi[a] ? z : -INFINITY;
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
template <typename TA, int DP, int TY, int RPT>
__global__ void __launch_bounds__(TY * 16)
attn_cc_kernel(const AttnParams p) {
    extern __shared__ __align__(16) float smem_f[];
    float* Qs = smem_f;
    float* Ps = Qs + TY * RPT * (DP + 4);
    TA* Ks = reinterpret_cast<TA*>(Ps + TY * RPT * CC_PP);
    TA* Vs = Ks + CC_KEYS * cc_pitch<TA>(DP);
    __shared__ int s_last;
    const int cta = blockIdx.x;
    ptx::griddep_wait();
    if (!attn_plan_agrees(p)) {
        if (threadIdx.x == 0) atomicOr(&g_attn_error, ATTN_ERR_RANGE);
        return;
    }
    AttnWalk walk;
    if (!walk.begin(p, cta)) return;
    AttnPiece pc;
    while (walk.next(p, cta, pc)) {
        if (RPT > 1 && pc.qlen * p.G - pc.row0 <= TY) cc_piece<TA, DP, TY, 1>(p, pc, Qs, Ps, Ks, Vs, &s_last);
        else cc_piece<TA, DP, TY, RPT>(p, pc, Qs, Ps, Ks, Vs, &s_last);
        __syncthreads();
    }
}

// cudaFuncSetAttribute once per device and kernel (idempotent, so a race is harmless).
cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

template <typename TA, int DP, int TY, int RPT>
cudaError_t launch_cc(const AttnParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = cc_smem<TA>(DP, TY * RPT);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_cc_kernel<TA, DP, TY, RPT>), done, smem);
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
    return cudaLaunchKernelEx(&cfg, attn_cc_kernel<TA, DP, TY, RPT>, p);
}

template <typename TA>
cudaError_t launch_cc_dp(const AttnParams& p, cudaStream_t s) {
    const bool small = p.plan.tile_rows == 16;
    if (p.Dh <= 64) return small ? launch_cc<TA, 64, 16, 1>(p, s) : launch_cc<TA, 64, 32, 4>(p, s);
    if (p.Dh <= 128) return small ? launch_cc<TA, 128, 16, 1>(p, s) : launch_cc<TA, 128, 32, 4>(p, s);
    return small ? launch_cc<TA, 256, 16, 1>(p, s) : launch_cc<TA, 256, 32, 2>(p, s);
}

size_t up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace attn

AttnPlan attn_plan_sizes(bool bf16, int64_t T, int B, int Hq, int Hk, int Dh, int page_size, int64_t max_q) {
    AttnPlan a = {};
    const int64_t G = Hq / Hk;
    const int dp = Dh <= 64 ? 64 : Dh <= 128 ? 128 : 256;
    if (attn_tc_supports(bf16, Hq, Hk, Dh, page_size)) {
        a.lane_rows = static_cast<int>(128 / G * G);
        a.tile_rows = (max_q * G <= a.lane_rows ? 1 : 2) * a.lane_rows;
        a.block_keys = 128;
        a.ncta = sm_count();
    } else {
        // up to 16 rows a sequence and key head: the 16-row tile, which wastes
        // no arithmetic on rows that are not there
        a.tile_rows = max_q * G <= 16 ? 16 : dp == 256 ? 64 : 128;
        a.block_keys = attn::CC_KEYS;
        // CTAs of an SM by their shared memory: two of the 16-row tile
        a.ncta = (a.tile_rows == 16 && dp < 256 ? 2 : 1) * sm_count();
    }
    if (a.ncta > attn::PLAN_CTAS) a.ncta = attn::PLAN_CTAS;
    a.lead = 2;   // 1, 2 and 3 take 191, 157 and 163 us for 4096 new tokens, 132, 131 and 132 us for 64 sequences decoding
    const int64_t rows = max_q * G < a.tile_rows ? max_q * G : a.tile_rows;
    a.slot_rows = static_cast<int>((rows + 3) & ~int64_t(3));
    a.max_tiles = T * G / a.tile_rows + B;
    a.start_off = 256;
    a.tile_off = a.start_off + attn::up(static_cast<size_t>(a.ncta) * sizeof(AttnStart));
    a.count_off = a.tile_off + attn::up(static_cast<size_t>(a.max_tiles) * sizeof(AttnTile));
    a.part_off = a.count_off + attn::up(static_cast<size_t>(a.max_tiles) * Hk * JOINS * sizeof(int));
    a.part_slot_bytes = attn::up(static_cast<size_t>(a.slot_rows) * (dp + 2) * sizeof(float));
    a.total = a.part_off + 2u * static_cast<size_t>(a.ncta) * a.part_slot_bytes;
    return a;
}

cudaError_t launch_attn_plan(const AttnPlan& plan, const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int B,
                             int Hq, int Hk, int window, int64_t max_q, int64_t max_kv, void* ws, cudaStream_t s) {
    g_error_word.may_be_set();
    attn::PlanParams p;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.ws = static_cast<unsigned char*>(ws);
    p.T = T;
    p.max_kv = max_kv;
    p.B = B;
    p.Hq = Hq;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.window = window;
    p.max_q = static_cast<int>(max_q);
    p.plan = plan;
    attn::attn_plan_kernel<<<1, attn::PLAN_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_attn(bool bf16, const AttnParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    if (attn_tc_supports(bf16, p.Hq, p.Hk, p.Dh, p.page_size)) return launch_paged_attn_tc(p, s);
    return bf16 ? attn::launch_cc_dp<__nv_bfloat16>(p, s) : attn::launch_cc_dp<float>(p, s);
}

}  // namespace mhc
