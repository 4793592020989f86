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
// Bound by latency, the chain of loads, scan, bisection and two dependent loads: 64
// sequences that decode take 3.9 us, 1024 6.8, 512 with trees of up to 64 tokens and
// fifty that end with 1000 pages each 15.4.  One CTA of 256 threads for small steps
// took 6.8 -> 4.2 us, with atomics for what fits replaced by bisection of the sums.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace mhc {

static __device__ unsigned g_step_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_step_error(unsigned* word) { return g_error_word.read_and_clear(g_step_error, word); }

namespace step {

// Inclusive sums over the block of three values each; `carry` is added to and
// becomes the sums so far.
template <int WARPS>
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
        int64_t s = lane < WARPS ? warp_sums[lane][i] : 0;
#pragma unroll
        for (int o = 1; o < WARPS; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const int64_t before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
        v[i] += carry[i] + (w > 0 ? before : 0);
        carry[i] += __shfl_sync(0xffffffffu, s, WARPS - 1);
    }
}

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

// Five numbers of each sequence in shared memory.
constexpr int NUMBERS = 5;
constexpr int BAD = -1, OVER = -2;   // in place of its cached tokens: its numbers do not fit, it ends

template <int THREADS>
__global__ void __launch_bounds__(THREADS)
step_kernel(const StepParams p) {
    extern __shared__ int smem[];
    int* cu = smem;                    // [B + 1] first rows (more than T: does not fit the call)
    int* upto = cu + p.B + 1;          // [B + 1] missing pages of the sequences before
    int* back = upto + p.B + 1;        // [B + 1] pages given back by the sequences before
    int* cached = back + p.B + 1;      // [B] tokens, BAD or OVER
    int* holds = cached + p.B + 1;     // [B] pages
    __shared__ int64_t warp_sums[THREADS / 32][3];
    const int tid = threadIdx.x, rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    const int raw = *p.free_count;
    if (tid == 0) cu[0] = upto[0] = back[0] = 0;
    int64_t carry[3] = {0, 0, 0};
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + tid;
        int64_t v[3] = {0, 0, 0};      // rows, missing pages, pages given back
        if (b < p.B) {
            const int n = p.new_lens[b], m = p.lens[b], h = p.held[b];
            const bool over = n == -1;
            bool good = h >= 0 && h <= p.width;
            if (!over) {
                const int64_t all = static_cast<int64_t>(m) + n;
                good = good && n >= 0 && m >= 0 && static_cast<int64_t>(h) * p.page >= m && all <= p.width * p.page &&
                       all <= p.max_len;
            }
            if (!good && rank == 0) atomicOr(&g_step_error, ATTN_ERR_RANGE);
            v[0] = n > 0 ? min(static_cast<int64_t>(n), p.T + 1) : 0;
            if (good && !over) {       // m + n is below 2^31 - 256
                const uint32_t last = static_cast<uint32_t>(m + n) + static_cast<uint32_t>(p.page - 1);
                const int pages = static_cast<int>(p.page_shift >= 0 ? last >> p.page_shift : last / static_cast<uint32_t>(p.page));
                v[1] = max(0, pages - h);
            }
            v[2] = good && over ? h : 0;
            cached[b] = !good ? BAD : over ? OVER : m;
            holds[b] = h;
        }
        scan3<THREADS / 32>(v, carry, warp_sums);
        if (b < p.B) {
            cu[b + 1] = static_cast<int>(min(v[0], p.T + 1));
            upto[b + 1] = static_cast<int>(v[1]);
            back[b + 1] = static_cast<int>(v[2]);
        }
    }
    __syncthreads();
    // All three sums rise, so what fits is found by bisection: sequences whose rows
    // fit, their rows, the pages that those of them take which get what they miss.
    const int count = max(0, min(raw, p.cap));
    const int avail = static_cast<int>(min(static_cast<int64_t>(count) + back[p.B], static_cast<int64_t>(p.cap)));
    const int fit = cu[p.B] <= p.T ? p.B : last_at_most(cu, p.B + 1, static_cast<int>(p.T));
    const int rows = cu[fit];
    const int take = upto[fit] <= avail ? upto[fit] : upto[last_at_most(upto, fit + 1, avail)];
    if (rank == 0 && tid == 0 && (raw != count || static_cast<int64_t>(count) + back[p.B] > p.cap || fit < p.B))
        atomicOr(&g_step_error, ATTN_ERR_RANGE);
    auto served = [&](int b) { return b < fit && (upto[b + 1] == upto[b] || upto[b + 1] <= avail); };
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
            const int i = static_cast<int>(t) - cu[b], m = cached[b], h = holds[b];
            const bool good = m >= 0;   // (one that ends has no rows)
            pos = good ? m + i : 0;
            int page = 0, in = 0;
            const bool room = good && served(b);
            if (room) {   // on its way while the tree is climbed
                const int at = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page;
                in = pos - at * p.page;
                page = at < h ? p.table[b * p.table_stride + at] : page_from_top(upto[b] + at - h);
            }
            if (words != nullptr) {
                // numbers fall on the way up, so the words are finished from the last to the first
                const int32_t* parents = p.parents + cu[b];
                // (a path of more than 1024 is of a node past the words, and is cut off: the
                // climbs of a chain of all rows would take minutes)
                for (int node = i; node >= 0 && path < TREE_MOST; ++path) {
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
            if (room) {
                if (page >= 0) slot = static_cast<int64_t>(page) * p.page + in;
                else atomicOr(&g_step_error, ATTN_ERR_RANGE);
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
        p.table[b * p.table_stride + holds[b] + (k - upto[b])] = page_from_top(static_cast<int>(k));
    }
    for (int64_t i = me; i < avail - take - count; i += all) p.free_pages[count + i] = returned(static_cast<int>(i));
    for (int64_t i = me; i < p.B; i += all) {
        const int b = static_cast<int>(i), m = cached[b];
        p.cu_q[b + 1] = b < fit ? cu[b + 1] : rows;
        // a sequence without room has no new tokens; one with room its rows (of numbers that fit)
        p.kv_lens[b] = m < 0 ? 0 : m + (served(b) ? cu[b + 1] - cu[b] : 0);
    }
    if (me == 0) p.cu_q[0] = 0;
    // every CTA has read held and the list's length
    if (ctas > 1) {
        __syncwarp();
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    if (rank == 0) {
        for (int b = tid; b < p.B; b += THREADS) {
            if (back[b + 1] > back[b]) p.held[b] = 0;
            else if (upto[b + 1] > upto[b] && served(b)) p.held[b] = holds[b] + upto[b + 1] - upto[b];
        }
        if (tid == 0) *p.free_count = avail - take;
    }
}

template <int THREADS>
cudaError_t launch(const StepParams& p, unsigned ctas, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};   // devices whose kernel has its shared memory and clusters allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit == 0 || !(done.load() & bit)) {
        e = cudaFuncSetAttribute(step_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 NUMBERS * (STEP_SEQUENCES + 1) * static_cast<int>(sizeof(int)));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(step_kernel<THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(NUMBERS) * static_cast<size_t>(p.B + 1) * sizeof(int);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, step_kernel<THREADS>, p);
}

}  // namespace step

// One CTA of 256 threads where that is a thread for each token and sequence, else
// 1024 threads in as many CTAs as the tokens fill, up to 16.
cudaError_t launch_paged_step(const StepParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    if (p.T <= 256 && p.B <= 256) return step::launch<256>(p, 1, s);
    unsigned ctas = 1;
    while (ctas < 16 && static_cast<int64_t>(ctas) * 1024 < p.T) ctas *= 2;
    return step::launch<1024>(p, ctas, s);
}

}  // namespace mhc
