// paged_attn_keep.cu -- after the verification of a drafted tree: the keys and
// values of the accepted path move to the places behind the context, in every
// layer's caches.
//
// For sequence b with context c = m - n and accepted nodes path[0] < path[1] <
// ...: token c + path[d] -> place c + d.  path[d] >= d, so a row moves to a lower
// place or stays, and a row that is read for d is never the goal of an earlier
// one.  A block (one sequence in one cache) therefore takes as many 16-byte
// pieces as its threads hold in registers, in the order of d: all are read, then
// all are written, and the next ones need no more than that.
// Bound by memory: two dependent reads (the path, the page number), then the rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "mhc_common.cuh"
#include "paged_attn.cuh"

namespace mhc {

static __device__ unsigned g_keep_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_keep_error(unsigned* word) { return g_error_word.read_and_clear(g_keep_error, word); }

namespace keep {

constexpr int THREADS = 128, HELD = 8;   // 16-byte pieces of a thread: 16 KB of a block in flight

__global__ void __launch_bounds__(THREADS)
keep_kernel(const __grid_constant__ KeepParams p) {
    const int b = static_cast<int>(blockIdx.x), cache = static_cast<int>(blockIdx.y), tid = threadIdx.x;
    const bool values = cache >= p.layers;
    const int n = p.cu_q[b + 1] - p.cu_q[b], m = p.kv_lens[b], c = p.keep[b];
    if (c == 0) return;   // nothing moves, its length stays
    const int32_t* path = p.path + b * p.path_stride;
    bool bad = c < 0 || c > p.max_keep || n < 0 || m < n || m > p.max_kv || c > n;
    int moved = 0;        // path entries of this thread that do not stay
    if (!bad)
        for (int d = tid; d < c; d += THREADS) {
            const int at = path[d], before = d > 0 ? path[d - 1] : -1;
            bad = bad || at <= before || at >= n;
            moved += at != d;
        }
    __shared__ int s_moved;
    if (tid == 0) s_moved = 0;
    if (__syncthreads_or(bad)) {
        if (tid == 0 && cache == 0) atomicOr(&g_keep_error, ATTN_ERR_RANGE);
        return;
    }
    if (moved > 0) atomicAdd(&s_moved, moved);
    __syncthreads();
    // once an entry has moved all later ones have
    const int first = c - s_moved, ctx = m - n;
    if (p.lens != nullptr && cache == 0 && tid == 0) p.lens[b] = ctx + c;
    char* base = static_cast<char*>(values ? p.v[cache - p.layers] : p.k[cache]);
    const int64_t page_bytes = values ? p.v_page : p.k_page, slot_bytes = values ? p.v_slot : p.k_slot;
    const int64_t head_bytes = values ? p.v_head : p.k_head;
    const int32_t* table = p.table + b * p.table_stride;
    // a token's row in the cache, null for a page number outside it
    auto row = [&](int token) -> char* {
        const int pg = p.page_shift >= 0 ? token >> p.page_shift : token / p.page;
        const int page = __ldg(table + pg);
        if (page < 0 || page >= p.num_pages) return nullptr;
        return base + page * page_bytes + (token - pg * p.page) * slot_bytes;
    };
    const int per = p.row_pieces;   // pieces of a token
    const int64_t total = static_cast<int64_t>(c - first) * per;
    for (int64_t i0 = 0; i0 < total; i0 += THREADS * HELD) {
        uint4 held[HELD];
        char* to[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int64_t i = i0 + u * THREADS + tid;
            to[u] = nullptr;
            if (i < total) {
                const int d = first + static_cast<int>(i / per), piece = static_cast<int>(i % per);
                const char* from = row(ctx + path[d]);
                char* goal = row(ctx + d);
                const int64_t in = (piece / p.head_pieces) * head_bytes + (piece % p.head_pieces) * 16;
                if (from != nullptr && goal != nullptr) {
                    held[u] = *reinterpret_cast<const uint4*>(from + in);
                    to[u] = goal + in;
                } else {
                    atomicOr(&g_keep_error, ATTN_ERR_RANGE);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < HELD; ++u)
            if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = held[u];
    }
}

}  // namespace keep

cudaError_t launch_cache_keep(const KeepParams& p, int B, cudaStream_t s) {
    g_error_word.may_be_set();
    keep::keep_kernel<<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(2 * p.layers)), keep::THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mhc
