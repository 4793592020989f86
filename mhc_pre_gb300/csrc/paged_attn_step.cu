// paged_attn_step.cu -- the integer tables of a step's new tokens, made on the
// GPU from the lengths of its sequences: who gets which pages, where each token
// goes in the cache, its position, and what it sees as a node of a tree.
//
// For sequence b with m = lens[b] cached and n = new_lens[b] new tokens that
// holds h = held[b] pages:
//   row start     cu[b] = sum of the new tokens before it
//   missing pages need[b] = max(0, ceil((m + n) / page) - h)
//   page k of all that are missing, counted over the sequences in order, is the
//   k-th from the top of the free list (on which the pages of sequences that end
//   have been put back); b gets its pages if the sum up to and with it is there
//   token i       place m + i, slot = page number * page + place in the page
//   node i        sees itself and what its parent sees
// The sums are three prefix sums over the sequences. One cluster of up to 16
// CTAs runs it: each CTA makes the sums in its own shared memory (a round of
// loads and a scan, cheaper than handing them over), then tokens and pages are
// spread over all threads and find their sequence by bisection.  New pages are
// computed from the free list, not read back from the table, and what others
// still read (held, the list's length) is written behind the cluster's barrier,
// so nothing waits on anything else.
// Bound by latency: the chain of loads, scan, bisection and two dependent loads.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "mhc_common.cuh"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace mhc {

static __device__ unsigned g_step_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_step_error(unsigned* word) { return g_error_word.read_and_clear(g_step_error, word); }

namespace step {

constexpr int THREADS = 1024, WARPS = THREADS / 32;

// Inclusive sums over the block of three values each; `carry` is added to and
// becomes the sums so far.
__device__ __forceinline__ void scan3(int64_t (&v)[3], int64_t (&carry)[3], int64_t (*warp_sums)[3]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += y;
        }
    __syncthreads();   // the sums of the round before have been read
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 3; ++i) warp_sums[w][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        int64_t s = warp_sums[lane][i];   // WARPS is 32
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const int64_t before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
        v[i] += carry[i] + (w > 0 ? before : 0);
        carry[i] += __shfl_sync(0xffffffffu, s, 31);
    }
}
static_assert(WARPS == 32, "scan3");

// The last of entries [0, n) that is at most x; entry 0 is.
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (a[lo + half] <= x) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

// What a sequence asks for, from its own numbers alone.
struct Ask {
    int64_t rows, need;   // tokens of the step, pages that it has not got
    int back;             // pages that it gives back
    bool over, good;      // it ends; its numbers fit
};
__device__ __forceinline__ Ask ask_of(const StepParams& p, int b) {
    const int n = p.new_lens[b], m = p.lens[b], h = p.held[b];
    Ask a;
    a.over = n == -1;
    a.good = h >= 0 && h <= p.width;
    if (!a.over)
        a.good = a.good && n >= 0 && m >= 0 && static_cast<int64_t>(h) * p.page >= m &&
                 static_cast<int64_t>(m) + n <= p.width * p.page && static_cast<int64_t>(m) + n <= p.max_len;
    a.rows = n > 0 ? min(static_cast<int64_t>(n), p.T + 1) : 0;
    a.need = a.good && !a.over ? max(int64_t(0), (static_cast<int64_t>(m) + n + p.page - 1) / p.page - h) : 0;
    a.back = a.good && a.over ? h : 0;
    return a;
}

__global__ void __launch_bounds__(THREADS)
step_kernel(const StepParams p) {
    extern __shared__ int smem[];
    int* cu = smem;                    // [B + 1] first rows (more than T: does not fit the call)
    int* upto = cu + p.B + 1;          // [B + 1] missing pages of the sequences before
    int* back = upto + p.B + 1;        // [B + 1] pages given back by the sequences before
    __shared__ int64_t warp_sums[WARPS][3];
    __shared__ int s_rows, s_take;
    const int tid = threadIdx.x, rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    if (tid == 0) {
        cu[0] = upto[0] = back[0] = 0;
        s_rows = s_take = 0;
    }
    const int raw = *p.free_count;
    int64_t carry[3] = {0, 0, 0};
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + tid;
        int64_t v[3] = {0, 0, 0};
        if (b < p.B) {
            const Ask a = ask_of(p, b);
            if (!a.good && rank == 0) atomicOr(&g_step_error, ATTN_ERR_RANGE);
            v[0] = a.rows;
            v[1] = a.need;
            v[2] = a.back;
        }
        scan3(v, carry, warp_sums);
        if (b < p.B) {
            cu[b + 1] = static_cast<int>(min(v[0], p.T + 1));
            upto[b + 1] = static_cast<int>(v[1]);
            back[b + 1] = static_cast<int>(v[2]);
            if (v[0] <= p.T) atomicMax(&s_rows, static_cast<int>(v[0]));
            else if (rank == 0) atomicOr(&g_step_error, ATTN_ERR_RANGE);
        }
    }
    __syncthreads();
    const int count = max(0, min(raw, p.cap));
    const int avail = static_cast<int>(min(static_cast<int64_t>(count) + back[p.B], static_cast<int64_t>(p.cap)));
    if (rank == 0 && tid == 0 && (raw != count || static_cast<int64_t>(count) + back[p.B] > p.cap))
        atomicOr(&g_step_error, ATTN_ERR_RANGE);
    // Sequences whose rows fit and whose pages are there; of those that miss pages they are the first.
    auto served = [&](int b) { return cu[b + 1] <= p.T && (upto[b + 1] == upto[b] || upto[b + 1] <= avail); };
    for (int b = tid; b < p.B; b += THREADS)
        if (upto[b + 1] > upto[b] && served(b)) atomicMax(&s_take, upto[b + 1]);
    __syncthreads();
    const int rows = s_rows, take = s_take;
    // the i-th page that came back, the k-th from the top of the list with those on it
    auto returned = [&](int i) {
        const int b = last_at_most(back, p.B + 1, i);
        return p.table[b * p.table_stride + (i - back[b])];
    };
    auto page_from_top = [&](int k) {
        const int at = avail - 1 - k;
        return at >= count ? returned(at - count) : p.free_pages[at];
    };
    const int64_t me = static_cast<int64_t>(rank) * THREADS + tid, all = static_cast<int64_t>(ctas) * THREADS;

    for (int64_t t = me; t < p.T; t += all) {
        int64_t slot = -1;
        int pos = 0, path = 0;
        int32_t* words = p.tree != nullptr ? p.tree + t * p.words : nullptr;
        int w = p.words - 1;
        uint32_t bits = 0u;
        if (t < rows) {
            const int b = last_at_most(cu, p.B + 1, static_cast<int>(t));
            const int i = static_cast<int>(t) - cu[b], m = p.lens[b], h = p.held[b];
            const bool good = ask_of(p, b).good;
            pos = good ? m + i : 0;
            if (good && served(b)) {
                const int at = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page;
                const int page = at < h ? p.table[b * p.table_stride + at] : page_from_top(upto[b] + at - h);
                if (page >= 0) slot = static_cast<int64_t>(page) * p.page + (pos - at * p.page);
                else atomicOr(&g_step_error, ATTN_ERR_RANGE);
            }
            if (words != nullptr) {
                // up the tree: numbers fall, so the words are finished from the last to the first
                const int32_t* parents = p.parents + cu[b];
                for (int node = i; node >= 0; ++path) {
                    if (node < 32 * p.words) {
                        for (; w > node >> 5; --w) {
                            words[w] = static_cast<int32_t>(bits);
                            bits = 0u;
                        }
                        bits |= 1u << (node & 31);
                    } else {
                        atomicOr(&g_step_error, ATTN_ERR_RANGE);
                    }
                    int up = __ldg(parents + node);
                    if (up < -1 || up >= node) {
                        atomicOr(&g_step_error, ATTN_ERR_RANGE);
                        up = -1;
                    }
                    node = up;
                }
                pos = good ? m + path - 1 : 0;
            }
        }
        if (words != nullptr)
            for (; w >= 0; --w) {
                words[w] = static_cast<int32_t>(bits);
                bits = 0u;
            }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
    // the missing pages into the table; those that came back and stay, onto the list
    for (int64_t k = me; k < take; k += all) {
        const int b = last_at_most(upto, p.B + 1, static_cast<int>(k));
        p.table[b * p.table_stride + p.held[b] + (k - upto[b])] = page_from_top(static_cast<int>(k));
    }
    for (int64_t i = me; i < avail - take - count; i += all) p.free_pages[count + i] = returned(static_cast<int>(i));
    for (int64_t b = me; b < p.B; b += all) {
        const Ask a = ask_of(p, static_cast<int>(b));
        p.cu_q[b + 1] = cu[b + 1] <= p.T ? cu[b + 1] : rows;
        p.kv_lens[b] = a.over || !a.good ? 0 : p.lens[b] + (served(static_cast<int>(b)) ? p.new_lens[b] : 0);
        if (b == 0) p.cu_q[0] = 0;
    }
    if (p.B == 0 && me == 0) p.cu_q[0] = 0;
    // every CTA has read held and the list's length
    __syncwarp();
    ptx::cluster_sync();
    if (rank == 0) {
        for (int b = tid; b < p.B; b += THREADS) {
            const Ask a = ask_of(p, b);
            if (a.back > 0) p.held[b] = 0;
            else if (upto[b + 1] > upto[b] && served(b)) p.held[b] += upto[b + 1] - upto[b];
        }
        if (tid == 0) *p.free_count = avail - take;
    }
}

}  // namespace step

cudaError_t launch_paged_step(const StepParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    static std::atomic<uint64_t> done{0};   // devices whose kernel has its shared memory and clusters allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit == 0 || !(done.load() & bit)) {
        e = cudaFuncSetAttribute(step::step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 3 * (STEP_SEQUENCES + 1) * static_cast<int>(sizeof(int)));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(step::step_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    unsigned ctas = 1;
    while (ctas < 16 && static_cast<int64_t>(ctas) * step::THREADS < p.T) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(step::THREADS);
    cfg.dynamicSmemBytes = 3u * static_cast<size_t>(p.B + 1) * sizeof(int);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, step::step_kernel, p);
}

}  // namespace mhc
