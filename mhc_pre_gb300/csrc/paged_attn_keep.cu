// paged_attn_keep.cu -- after the verification of a drafted tree: the keys and
// values of the accepted path move to the places behind the context, in every
// layer's caches.
//
// For sequence b with context c = m - n and accepted nodes path[0] < path[1] <
// ...: token c + path[d] -> place c + d.  path[d] >= d, so a row moves to a lower
// place or stays, and a row that is read for d is never the goal of an earlier
// one.  A block (one sequence in one cache, or in up to four, one after the other)
// therefore takes as many 16-byte pieces as its threads hold in registers, in the
// order of d: all are read, then all are written, and the next ones need no more
// than that.
// Bound by memory behind two dependent reads (the path, the page number): 7 of 32
// tokens of 48 sequences in 16 layers, 44 MB read and written, take 10.9 us (4.1
// TB/s), one sequence in one layer 3.7.  Rows looked up together in shared memory:
// 13.4 -> 10.9 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "paged_attn.cuh"

namespace mhc {

static __device__ unsigned g_keep_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_keep_error(unsigned* word) { return g_error_word.read_and_clear(g_keep_error, word); }

namespace keep {

constexpr int THREADS = 128, HELD = 8;   // 16-byte pieces of a thread: 16 KB of a block in flight
constexpr int ROWS = THREADS;            // of a path, looked up together
constexpr int BLOCKS = 8192;             // a block has two caches from twice as many sequences and caches on, ...

__global__ void __launch_bounds__(THREADS)
keep_kernel(const __grid_constant__ KeepParams p) {
    __shared__ int64_t from[ROWS], to[ROWS];   // byte offsets in the cache, -1: a page outside it
    const int b = static_cast<int>(blockIdx.x), tid = threadIdx.x;
    const bool reports = blockIdx.y == 0 && tid == 0;
    const int32_t* path = p.path + b * p.path_stride;
    // the path's first entries are on their way before its length is known
    int mine = tid < p.max_keep ? path[tid] : 0, before = tid > 0 && tid < p.max_keep ? path[tid - 1] : -1;
    const int n = p.cu_q[b + 1] - p.cu_q[b], m = p.kv_lens[b], c = p.keep[b];
    if (c == 0) return;   // nothing moves, its length stays
    bool bad = c < 0 || c > p.max_keep || n < 0 || m < n || m > p.max_kv || c > n;
    if (!bad)
        for (int d = tid; d < c; d += THREADS) {
            const int at = d == tid ? mine : path[d], prev = d == tid ? before : path[d - 1];
            bad = bad || at <= prev || at >= n;
        }
    if (__syncthreads_or(bad)) {
        if (reports) atomicOr(&g_keep_error, ATTN_ERR_RANGE);
        return;
    }
    const int ctx = m - n;
    if (p.lens != nullptr && reports) p.lens[b] = ctx + c;
    // once an entry has moved all later ones have: the first ones stay
    int first = 0;
    for (int d0 = 0; d0 < c; d0 += THREADS) first += __syncthreads_count(d0 + tid < c && (d0 == 0 ? mine : path[d0 + tid]) == d0 + tid);
    const int32_t* table = p.table + b * p.table_stride;
    const uint32_t per = static_cast<uint32_t>(p.row_pieces), head = static_cast<uint32_t>(p.head_pieces);
    for (int cache = blockIdx.y; cache < 2 * p.layers; cache += gridDim.y) {
        const bool values = cache >= p.layers;
        char* base = static_cast<char*>(values ? p.v[cache - p.layers] : p.k[cache]);
        const int64_t page_bytes = values ? p.v_page : p.k_page, slot_bytes = values ? p.v_slot : p.k_slot;
        const int64_t head_bytes = values ? p.v_head : p.k_head;
        auto place = [&](int token) -> int64_t {
            const int pg = p.page_shift >= 0 ? token >> p.page_shift : token / p.page;
            const int page = __ldg(table + pg);
            if (page < 0 || page >= p.num_pages) {
                atomicOr(&g_keep_error, ATTN_ERR_RANGE);
                return -1;
            }
            return page * page_bytes + (token - pg * p.page) * slot_bytes;
        };
        for (int d0 = first; d0 < c; d0 += ROWS) {
            const int rows = min(ROWS, c - d0);
            if (tid < rows) {
                const int64_t f = place(ctx + path[d0 + tid]), t = place(ctx + d0 + tid);
                from[tid] = t >= 0 ? f : -1;
                to[tid] = t;
            }
            __syncthreads();
            const uint32_t total = static_cast<uint32_t>(rows) * per;
            for (uint32_t i0 = 0; i0 < total; i0 += THREADS * HELD) {
                uint4 held[HELD];
                char* goal[HELD];
#pragma unroll
                for (int u = 0; u < HELD; ++u) {
                    const uint32_t i = i0 + u * THREADS + tid;
                    goal[u] = nullptr;
                    if (i < total) {
                        const uint32_t d = i / per, piece = i - d * per, h = piece / head;
                        const int64_t f = from[d], in = h * head_bytes + (piece - h * head) * 16u;
                        if (f >= 0) {
                            held[u] = *reinterpret_cast<const uint4*>(base + f + in);
                            goal[u] = base + to[d] + in;
                        }
                    }
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < HELD; ++u)
                    if (goal[u] != nullptr) *reinterpret_cast<uint4*>(goal[u]) = held[u];
            }
        }
    }
}

}  // namespace keep

// A block for each sequence and cache; where those are many, most of them may find
// only that nothing moves, at 0.5 ns each, and a block has up to 4 caches one after the
// other: two from 16384 sequences and caches on, 4 from 32768. 48 sequences that keep rows among 512, 2048 and 8192, in 16 layers: 14.5, 22
// and 45 us, with a block each 16, 38 and 136 (up to 8 caches: 14.5, 28 and 39).  256 that
// all do in 32 layers: 82, with a block each 86.
cudaError_t launch_cache_keep(const KeepParams& p, int B, cudaStream_t s) {
    g_error_word.may_be_set();
    const int64_t each = static_cast<int64_t>(B) * 2 * p.layers / keep::BLOCKS, caches = each < 1 ? 1 : each > 4 ? 4 : each;
    const unsigned split = static_cast<unsigned>((2 * p.layers + caches - 1) / caches);
    keep::keep_kernel<<<dim3(static_cast<unsigned>(B), split), keep::THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mhc
