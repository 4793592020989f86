// paged_attn.cu -- attention of a chunk of new tokens over a paged cache: the
// plan kernel, and the choice of kernel.
//
//   z[i, j] = scale <q_i, k_j>,  z = softcap tanh(z / softcap) when capped,
//   keys j <= kvlen - qlen + i, and j > kvlen - qlen + i - window,
//   o_i = sum_j exp(z_ij - lse_i) v_j,  lse_i = log sum_j exp(z_ij);
// a row that sees no key gives o = 0 and lse = -inf.
//
// bf16 heads of at most 128 over pages that divide (or are a multiple of) 128
// keys run on the tensor cores (paged_attn_tc.cu).  Everything else (float32,
// wider heads, other page sizes) runs in attn_cc_kernel (paged_attn_cc.cuh), which keeps a
// tile's scores and sums in registers and walks the keys once.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_attn_cc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_error, word); }

namespace attn {

constexpr int PLAN_THREADS = 512;   // also at least PLAN_CTAS
constexpr int PLAN_NEAR = 256;      // whole tiles kept there for the borders (12 KB)
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
        if (s.unit > 0 && cost * ATTN_SMALL_TILE <= per) {
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
    return bf16 ? attn::launch_cc_dp<__nv_bfloat16, false>(p, s) : attn::launch_cc_dp<float, false>(p, s);
}

}  // namespace mhc
