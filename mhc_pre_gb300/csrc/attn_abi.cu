// attn_abi.cu -- the extern "C" entry points of the attention sublayer:
// validation and dispatch only (the qk_norm_rope and paged_attn files compute).
// Nothing here allocates memory or synchronises the host.
#include <math.h>

#include "../../include/mhc.h"
#include "launch.h"
#include "paged_attn.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
mhc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA; }

// Largest sizes taken: inside what the kernels' index arithmetic holds.
constexpr int64_t MAX_T = int64_t(1) << 30, MAX_STRIDE = int64_t(1) << 36, MAX_KV = (int64_t(1) << 31) - 256;
constexpr int MAX_HEADS = 1024;

mhc_status check_heads(mhc_dtype dt, int64_t T, int Hq, int Hk, int Dh) {
    if (dt != MHC_F32 && dt != MHC_BF16) return MHC_ERR_INVALID_ARG;
    if (T < 0 || Hq <= 0 || Hk <= 0 || Dh <= 0) return MHC_ERR_INVALID_ARG;
    if (Hq % Hk != 0 || Hq > MAX_HEADS || Dh % 8 != 0 || Dh > 256 || T > MAX_T) return MHC_ERR_UNSUPPORTED;
    return MHC_OK;
}

// Integers and row statistics are read and written one by one: their own size.
mhc_status check_plain(const void* p, unsigned bytes) {
    if (p == nullptr) return MHC_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 ? MHC_OK : MHC_ERR_MISALIGNED;
}

// Numbers that may be null where there are none.
mhc_status check_counted(const void* p, unsigned bytes, int64_t entries) {
    return entries == 0 && p == nullptr ? MHC_OK : check_plain(p, bytes);
}

mhc_status check_ptrs(const void* const* ptrs, int n) {
    for (int i = 0; i < n; ++i) {
        if (ptrs[i] == nullptr) return MHC_ERR_INVALID_ARG;
        if (!aligned16(ptrs[i])) return MHC_ERR_MISALIGNED;
    }
    return MHC_OK;
}

// The distance between the tokens of a tensor of H heads.
mhc_status check_stride(mhc_dtype dt, int64_t stride, int H, int Dh) {
    const int64_t vec = dt == MHC_BF16 ? 8 : 4;
    if (stride < static_cast<int64_t>(H) * Dh) return MHC_ERR_INVALID_ARG;
    if (stride > MAX_STRIDE) return MHC_ERR_UNSUPPORTED;
    return stride % vec == 0 ? MHC_OK : MHC_ERR_MISALIGNED;
}

mhc_status check_rope(int Dh, int rot, int flags, float eps, int64_t max_pos, const int32_t* positions,
                      const float* cos_sin) {
    if (rot < 0 || rot > Dh || (flags & ~MHC_ROPE_ADJACENT) != 0) return MHC_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return MHC_ERR_INVALID_ARG;
    if (rot % 16 != 0) return MHC_ERR_UNSUPPORTED;
    if (rot == 0) return MHC_OK;
    if (cos_sin == nullptr || max_pos <= 0) return MHC_ERR_INVALID_ARG;
    if (max_pos > MAX_T) return MHC_ERR_UNSUPPORTED;
    if (!aligned16(cos_sin)) return MHC_ERR_MISALIGNED;
    return check_plain(positions, 4);
}

mhc_status check_cache(mhc_dtype dt, int64_t num_pages, int page_size, int Hk, int Dh, int64_t page_stride,
                       int64_t slot_stride, int64_t head_stride) {
    const int64_t vec = dt == MHC_BF16 ? 8 : 4;
    if (num_pages <= 0 || page_size <= 0) return MHC_ERR_INVALID_ARG;
    if (num_pages > (int64_t(1) << 31) - 1 || page_size > (1 << 20)) return MHC_ERR_UNSUPPORTED;
    if (slot_stride < Dh || (Hk > 1 && head_stride < Dh) || head_stride < 0 || page_stride < Dh)
        return MHC_ERR_INVALID_ARG;
    if (page_stride > MAX_STRIDE || slot_stride > MAX_STRIDE || head_stride > MAX_STRIDE) return MHC_ERR_UNSUPPORTED;
    if (page_stride % vec != 0 || slot_stride % vec != 0 || head_stride % vec != 0) return MHC_ERR_MISALIGNED;
    return MHC_OK;
}

mhc_status check_attn(mhc_dtype dt, int64_t T, int B, int Hq, int Hk, int Dh, int page_size, int64_t max_q,
                      int64_t max_kv, int window) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (B < 0 || page_size <= 0 || max_q < 0 || max_kv < 0 || window < 0) return MHC_ERR_INVALID_ARG;
    // rows of a sequence and keys are 32-bit numbers in the kernels, and a
    // tile's key range plus one block must not pass them
    if (B > (1 << 24) || max_q > MAX_T / Hq || max_kv > MAX_KV || T > MAX_T / Hq) return MHC_ERR_UNSUPPORTED;
    return MHC_OK;
}

// 32-bit numbers in memory: rows of `width`, `stride` apart.
struct Numbers {
    const void* p;
    int64_t rows, width, stride;
};
// Whether rows and a run (one row) have any in common; what lies between rows is theirs only.
bool meet(const Numbers& a, const Numbers& run) {
    if (a.p == nullptr || run.p == nullptr || a.rows == 0 || a.width == 0 || run.width == 0) return false;
    const int64_t from = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(run.p)) -
                          static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p))) / 4, to = from + run.width;
    int64_t r = a.rows > 1 && from > 0 ? from / a.stride : 0;   // the last row that begins at `from` or before
    if (r >= a.rows) r = a.rows - 1;
    if (from < r * a.stride + a.width && r * a.stride < to) return true;
    return r + 1 < a.rows && (r + 1) * a.stride < to;
}

// The page size as a shift, -1 where it is none.
int shift_of(int page_size) {
    for (int i = 0; i < 21; ++i)
        if (page_size == (1 << i)) return i;
    return -1;
}

// A tile's join counters are numbered in 32 bits.
bool counters_fit(const mhc::AttnPlan& plan, int Hk) {
    return plan.max_tiles * Hk < (int64_t(1) << 31) / mhc::JOINS;
}

}  // namespace

extern "C" {

mhc_status mhc_qk_norm_rope(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const float* w_q, const float* w_k, const int32_t* positions, const float* cos_sin,
                            int64_t max_pos, int64_t T, int Hq, int Hk, int Dh, int rot, int flags, float eps,
                            void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            cudaStream_t stream) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (T == 0) return MHC_OK;
    const void* ptrs[] = {q, k, w_q, w_k, q_out, k_out};
    if ((st = check_ptrs(ptrs, 6)) != MHC_OK) return st;
    if ((st = check_rope(Dh, rot, flags, eps, max_pos, positions, cos_sin)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_out_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_out_stride, Hk, Dh)) != MHC_OK) return st;
    mhc::QkParams p = {};
    p.q = q;
    p.k = k;
    p.w_q = w_q;
    p.w_k = w_k;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.T = T;
    p.page_size = 1;
    p.Hq = Hq;
    p.Hk = Hk;
    p.Dh = Dh;
    p.rot = rot;
    p.max_pos = static_cast<int>(rot > 0 ? max_pos : 0);
    p.eps = eps;
    p.q_out = q_out;
    p.k_out = k_out;
    return from_cuda(mhc::launch_qk_norm_rope(dt == MHC_BF16, (flags & MHC_ROPE_ADJACENT) != 0, false, p, stream));
}

size_t mhc_qk_norm_rope_bwd_workspace_bytes(int64_t T, int Dh) {
    if (T <= 0 || Dh <= 0) return 0;
    return static_cast<size_t>(mhc::qk_bwd_blocks(T)) * 2u * static_cast<size_t>(Dh) * sizeof(float);
}

mhc_status mhc_qk_norm_rope_bwd(mhc_dtype dt, const void* g_q, int64_t gq_stride, const void* g_k, int64_t gk_stride,
                                const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* w_q,
                                const float* w_k, const int32_t* positions, const float* cos_sin, int64_t max_pos,
                                int64_t T, int Hq, int Hk, int Dh, int rot, int flags, float eps, void* dq,
                                int64_t dq_stride, void* dk, int64_t dk_stride, float* dw_q, float* dw_k,
                                void* workspace, size_t ws_bytes, cudaStream_t stream) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (T == 0) {   // sums over no tokens
        const void* outs[] = {dw_q, dw_k};
        if ((st = check_ptrs(outs, 2)) != MHC_OK) return st;
        const size_t n = static_cast<size_t>(Dh) * sizeof(float);
        cudaError_t e = cudaMemsetAsync(dw_q, 0, n, stream);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_k, 0, n, stream);
        return from_cuda(e);
    }
    const void* ptrs[] = {g_q, g_k, q, k, w_q, w_k, dq, dk, dw_q, dw_k, workspace};
    if ((st = check_ptrs(ptrs, 11)) != MHC_OK) return st;
    if ((st = check_rope(Dh, rot, flags, eps, max_pos, positions, cos_sin)) != MHC_OK) return st;
    const int64_t strides_q[] = {gq_stride, q_stride, dq_stride}, strides_k[] = {gk_stride, k_stride, dk_stride};
    for (int i = 0; i < 3; ++i) {
        if ((st = check_stride(dt, strides_q[i], Hq, Dh)) != MHC_OK) return st;
        if ((st = check_stride(dt, strides_k[i], Hk, Dh)) != MHC_OK) return st;
    }
    if (ws_bytes < mhc_qk_norm_rope_bwd_workspace_bytes(T, Dh)) return MHC_ERR_INVALID_ARG;
    mhc::QkBwdParams p = {};
    p.g_q = g_q;
    p.g_k = g_k;
    p.q = q;
    p.k = k;
    p.w_q = w_q;
    p.w_k = w_k;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.gq_stride = gq_stride;
    p.gk_stride = gk_stride;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.dq_stride = dq_stride;
    p.dk_stride = dk_stride;
    p.T = T;
    p.Hq = Hq;
    p.Hk = Hk;
    p.Dh = Dh;
    p.rot = rot;
    p.max_pos = static_cast<int>(rot > 0 ? max_pos : 0);
    p.eps = eps;
    p.dq = dq;
    p.dk = dk;
    p.partial = static_cast<float*>(workspace);
    return from_cuda(mhc::launch_qk_norm_rope_bwd(dt == MHC_BF16, (flags & MHC_ROPE_ADJACENT) != 0, p, dw_q, dw_k,
                                                  stream));
}

mhc_status mhc_qk_norm_rope_append(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                   const void* v, int64_t v_stride, const float* w_q, const float* w_k,
                                   const int32_t* positions, const float* cos_sin, int64_t max_pos,
                                   const int64_t* slots, int64_t T, int Hq, int Hk, int Dh, int rot, int flags,
                                   float eps, void* q_out, int64_t q_out_stride, void* k_cache, int64_t k_page_stride,
                                   int64_t k_slot_stride, int64_t k_head_stride, void* v_cache,
                                   int64_t v_page_stride, int64_t v_slot_stride, int64_t v_head_stride,
                                   int64_t num_pages, int page_size, cudaStream_t stream) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (T == 0) return MHC_OK;
    const void* ptrs[] = {q, k, v, w_q, w_k, q_out, k_cache, v_cache};
    if ((st = check_ptrs(ptrs, 8)) != MHC_OK) return st;
    if ((st = check_plain(slots, 8)) != MHC_OK) return st;
    if ((st = check_rope(Dh, rot, flags, eps, max_pos, positions, cos_sin)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, v_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_out_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, k_page_stride, k_slot_stride, k_head_stride)) != MHC_OK)
        return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, v_page_stride, v_slot_stride, v_head_stride)) != MHC_OK)
        return st;
    mhc::QkParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.w_q = w_q;
    p.w_k = w_k;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.slots = slots;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.k_page_stride = k_page_stride;
    p.k_slot_stride = k_slot_stride;
    p.k_head_stride = k_head_stride;
    p.v_page_stride = v_page_stride;
    p.v_slot_stride = v_slot_stride;
    p.v_head_stride = v_head_stride;
    p.num_slots = num_pages * page_size;
    p.T = T;
    p.page_size = page_size;
    p.Hq = Hq;
    p.Hk = Hk;
    p.Dh = Dh;
    p.rot = rot;
    p.max_pos = static_cast<int>(rot > 0 ? max_pos : 0);
    p.eps = eps;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    return from_cuda(mhc::launch_qk_norm_rope(dt == MHC_BF16, (flags & MHC_ROPE_ADJACENT) != 0, true, p, stream));
}

static mhc_status rope_call(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk,
                            int Dh, int rot, int flags, bool back, void* q_out, int64_t q_out_stride, void* k_out,
                            int64_t k_out_stride, cudaStream_t stream) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (T == 0) return MHC_OK;
    const void* ptrs[] = {q, k, q_out, k_out};
    if ((st = check_ptrs(ptrs, 4)) != MHC_OK) return st;
    if (rot == 0) return MHC_ERR_INVALID_ARG;   // nothing to turn
    if ((st = check_rope(Dh, rot, flags, 0.0f, max_pos, positions, cos_sin)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_out_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_out_stride, Hk, Dh)) != MHC_OK) return st;
    mhc::QkParams p = {};
    p.q = q;
    p.k = k;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.T = T;
    p.page_size = 1;
    p.Hq = Hq;
    p.Hk = Hk;
    p.Dh = Dh;
    p.rot = rot;
    p.max_pos = static_cast<int>(max_pos);
    p.sine_sign = back ? -1.0f : 1.0f;
    p.q_out = q_out;
    p.k_out = k_out;
    return from_cuda(mhc::launch_rope(dt == MHC_BF16, (flags & MHC_ROPE_ADJACENT) != 0, false, p, stream));
}

mhc_status mhc_rope(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk, int Dh,
                    int rot, int flags, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                    cudaStream_t stream) {
    return rope_call(dt, q, q_stride, k, k_stride, positions, cos_sin, max_pos, T, Hq, Hk, Dh, rot, flags, false, q_out,
                     q_out_stride, k_out, k_out_stride, stream);
}

mhc_status mhc_rope_bwd(mhc_dtype dt, const void* g_q, int64_t gq_stride, const void* g_k, int64_t gk_stride,
                        const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk,
                        int Dh, int rot, int flags, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                        cudaStream_t stream) {
    return rope_call(dt, g_q, gq_stride, g_k, gk_stride, positions, cos_sin, max_pos, T, Hq, Hk, Dh, rot, flags, true, dq,
                     dq_stride, dk, dk_stride, stream);
}

mhc_status mhc_rope_append(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                           int64_t max_pos, const int64_t* slots, int64_t T, int Hq, int Hk, int Dh, int rot, int flags,
                           void* q_out, int64_t q_out_stride, void* k_cache, int64_t k_page_stride,
                           int64_t k_slot_stride, int64_t k_head_stride, void* v_cache, int64_t v_page_stride,
                           int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                           cudaStream_t stream) {
    mhc_status st = check_heads(dt, T, Hq, Hk, Dh);
    if (st != MHC_OK) return st;
    if (T == 0) return MHC_OK;
    const void* ptrs[] = {q, k, v, q_out, k_cache, v_cache};
    if ((st = check_ptrs(ptrs, 6)) != MHC_OK) return st;
    if ((st = check_plain(slots, 8)) != MHC_OK) return st;
    if (rot == 0) return MHC_ERR_INVALID_ARG;
    if ((st = check_rope(Dh, rot, flags, 0.0f, max_pos, positions, cos_sin)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, k_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, v_stride, Hk, Dh)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_out_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, k_page_stride, k_slot_stride, k_head_stride)) != MHC_OK)
        return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, v_page_stride, v_slot_stride, v_head_stride)) != MHC_OK)
        return st;
    mhc::QkParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.slots = slots;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.k_page_stride = k_page_stride;
    p.k_slot_stride = k_slot_stride;
    p.k_head_stride = k_head_stride;
    p.v_page_stride = v_page_stride;
    p.v_slot_stride = v_slot_stride;
    p.v_head_stride = v_head_stride;
    p.num_slots = num_pages * page_size;
    p.T = T;
    p.page_size = page_size;
    p.Hq = Hq;
    p.Hk = Hk;
    p.Dh = Dh;
    p.rot = rot;
    p.max_pos = static_cast<int>(max_pos);
    p.sine_sign = 1.0f;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    return from_cuda(mhc::launch_rope(dt == MHC_BF16, (flags & MHC_ROPE_ADJACENT) != 0, true, p, stream));
}

mhc_status mhc_rope_table(int64_t n, int rot, double base, double factor, double original, double low, double high,
                          float amplitude, float* cos_sin, cudaStream_t stream) {
    if (n < 0 || rot <= 0 || !(base >= 1.0) || !isfinite(base) || !(factor > 0.0) || !isfinite(factor) ||
        !isfinite(1.0 / factor) || !(original >= 0.0) || !isfinite(original) || !isfinite(low) || !isfinite(high) ||
        !(low < high) || !isfinite(amplitude))
        return MHC_ERR_INVALID_ARG;
    if (rot % 16 != 0 || rot > 256 || n > MAX_T) return MHC_ERR_UNSUPPORTED;
    if (n == 0) return MHC_OK;
    const void* ptrs[] = {cos_sin};
    mhc_status st = check_ptrs(ptrs, 1);
    if (st != MHC_OK) return st;
    return from_cuda(mhc::launch_rope_table(n, rot, base, factor, original, low, high, amplitude, cos_sin, stream));
}

size_t mhc_paged_attn_workspace_bytes(mhc_dtype dt, int64_t T, int B, int Hq, int Hk, int Dh, int page_size,
                                      int64_t max_q) {
    if (check_attn(dt, T, B, Hq, Hk, Dh, page_size, max_q, 0, 0) != MHC_OK || T == 0 || B == 0) return 0;
    const mhc::AttnPlan plan = mhc::attn_plan_sizes(dt == MHC_BF16, T, B, Hq, Hk, Dh, page_size, max_q);
    return counters_fit(plan, Hk) ? plan.total : 0;
}

// What trees of drafted tokens ask for beside the causal call's checks.
static mhc_status check_tree(int64_t max_q, const int32_t* tree, int64_t tree_stride) {
    if (max_q > mhc::TREE_MOST) return MHC_ERR_UNSUPPORTED;
    if (tree_stride < (max_q + 31) / 32) return MHC_ERR_INVALID_ARG;
    if (tree_stride > MAX_STRIDE) return MHC_ERR_UNSUPPORTED;
    return check_plain(tree, 4);
}

mhc_status mhc_paged_attn_plan(mhc_dtype dt, const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int B, int Hq,
                               int Hk, int Dh, int page_size, int64_t max_q, int64_t max_kv, int window,
                               void* workspace, size_t ws_bytes, cudaStream_t stream) {
    mhc_status st = check_attn(dt, T, B, Hq, Hk, Dh, page_size, max_q, max_kv, window);
    if (st != MHC_OK) return st;
    if (T == 0 || B == 0) return MHC_OK;
    const void* ptrs[] = {workspace};
    if ((st = check_ptrs(ptrs, 1)) != MHC_OK) return st;
    if ((st = check_plain(cu_q, 4)) != MHC_OK || (st = check_plain(kv_lens, 4)) != MHC_OK) return st;
    const mhc::AttnPlan plan = mhc::attn_plan_sizes(dt == MHC_BF16, T, B, Hq, Hk, Dh, page_size, max_q);
    if (!counters_fit(plan, Hk)) return MHC_ERR_UNSUPPORTED;
    if (ws_bytes < plan.total) return MHC_ERR_INVALID_ARG;
    return from_cuda(mhc::launch_attn_plan(plan, cu_q, kv_lens, T, B, Hq, Hk, window, max_q, max_kv, workspace, stream));
}

static mhc_status attn_call(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache, int64_t k_page_stride,
                            int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                            int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                            const int32_t* page_table, int64_t table_stride, bool trees, const int32_t* tree,
                            int64_t tree_stride, const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int B, int Hq,
                            int Hk, int Dh, int64_t max_q, int64_t max_kv, int window, float scale, float softcap,
                            void* o, float* lse, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    mhc_status st = check_attn(dt, T, B, Hq, Hk, Dh, page_size, max_q, max_kv, window);
    if (st != MHC_OK) return st;
    if (!(scale > 0.0f) || !isfinite(scale) || !(softcap >= 0.0f) || !isfinite(softcap)) return MHC_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return MHC_OK;
    if ((cu_q == nullptr) != (kv_lens == nullptr)) return MHC_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k_cache, v_cache, o, workspace};
    if ((st = check_ptrs(ptrs, 5)) != MHC_OK) return st;
    if ((st = check_plain(page_table, 4)) != MHC_OK) return st;
    if (lse != nullptr && (st = check_plain(lse, 4)) != MHC_OK) return st;
    if ((st = check_stride(dt, q_stride, Hq, Dh)) != MHC_OK) return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, k_page_stride, k_slot_stride, k_head_stride)) != MHC_OK)
        return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, v_page_stride, v_slot_stride, v_head_stride)) != MHC_OK)
        return st;
    if (table_stride < (max_kv + page_size - 1) / page_size) return MHC_ERR_INVALID_ARG;
    if (trees && (st = check_tree(max_q, tree, tree_stride)) != MHC_OK) return st;
    const mhc::AttnPlan plan = mhc::attn_plan_sizes(dt == MHC_BF16, T, B, Hq, Hk, Dh, page_size, max_q);
    if (!counters_fit(plan, Hk)) return MHC_ERR_UNSUPPORTED;
    if (ws_bytes < plan.total) return MHC_ERR_INVALID_ARG;
    if (trees) {
        if ((st = check_plain(cu_q, 4)) != MHC_OK || (st = check_plain(kv_lens, 4)) != MHC_OK) return st;
    } else if (cu_q != nullptr) {
        st = mhc_paged_attn_plan(dt, cu_q, kv_lens, T, B, Hq, Hk, Dh, page_size, max_q, max_kv, window, workspace,
                                 ws_bytes, stream);
        if (st != MHC_OK) return st;
    }
    mhc::AttnParams p = {};
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.o = o;
    p.lse = lse;
    p.page_table = page_table;
    p.tree = reinterpret_cast<const uint32_t*>(tree);
    p.tree_stride = tree_stride;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.ws = static_cast<unsigned char*>(workspace);
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.num_pages = num_pages;
    p.k_page_stride = k_page_stride;
    p.k_slot_stride = k_slot_stride;
    p.k_head_stride = k_head_stride;
    p.v_page_stride = v_page_stride;
    p.v_slot_stride = v_slot_stride;
    p.v_head_stride = v_head_stride;
    p.T = T;
    p.max_q = max_q;
    p.max_kv = max_kv;
    p.B = B;
    p.Hq = Hq;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.Dh = Dh;
    p.page_size = page_size;
    p.page_shift = shift_of(page_size);
    p.window = window;
    if (p.G > 1) {   // M = floor(2^(31+s) / G) + 1, 2^s >= G: exact below 2^31
        unsigned sh = 1;
        while ((1 << sh) < p.G) ++sh;
        p.g_mul = static_cast<unsigned>((uint64_t(1) << (31 + sh)) / static_cast<unsigned>(p.G)) + 1u;
        p.g_shift = sh - 1;
    }
    p.scale = scale;
    p.softcap = softcap;
    p.force_timeout = mhc::forced_timeout();
    p.plan = plan;
    if (trees) p.plan.lead = plan.block_keys == 128 ? mhc::TREE_LEAD : mhc::TREE_LEAD_CC;
    return from_cuda(trees ? mhc::launch_tree_attn(dt == MHC_BF16, p, stream)
                           : mhc::launch_paged_attn(dt == MHC_BF16, p, stream));
}

mhc_status mhc_paged_attn(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache, int64_t k_page_stride,
                          int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                          int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                          const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                          const int32_t* kv_lens, int64_t T, int B, int Hq, int Hk, int Dh, int64_t max_q,
                          int64_t max_kv, int window, float scale, float softcap, void* o, float* lse,
                          void* workspace, size_t ws_bytes, cudaStream_t stream) {
    return attn_call(dt, q, q_stride, k_cache, k_page_stride, k_slot_stride, k_head_stride, v_cache, v_page_stride,
                     v_slot_stride, v_head_stride, num_pages, page_size, page_table, table_stride, false, nullptr, 0, cu_q,
                     kv_lens, T, B, Hq, Hk, Dh, max_q, max_kv, window, scale, softcap, o, lse, workspace, ws_bytes, stream);
}

mhc_status mhc_tree_attn(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache, int64_t k_page_stride,
                         int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                         int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                         const int32_t* page_table, int64_t table_stride, const int32_t* tree, int64_t tree_stride,
                         const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int B, int Hq, int Hk, int Dh,
                         int64_t max_q, int64_t max_kv, int window, float scale, float softcap, void* o, float* lse,
                         void* workspace, size_t ws_bytes, cudaStream_t stream) {
    return attn_call(dt, q, q_stride, k_cache, k_page_stride, k_slot_stride, k_head_stride, v_cache, v_page_stride,
                     v_slot_stride, v_head_stride, num_pages, page_size, page_table, table_stride, true, tree, tree_stride,
                     cu_q, kv_lens, T, B, Hq, Hk, Dh, max_q, max_kv, window, scale, softcap, o, lse, workspace, ws_bytes,
                     stream);
}

mhc_status mhc_paged_step(const int32_t* new_lens, const int32_t* lens, int B, int32_t* page_table,
                          int64_t table_stride, int64_t table_width, int32_t* held, int32_t* free_pages,
                          int64_t free_capacity, int32_t* free_count, int page_size, int64_t T,
                          const int32_t* parents, int tree_words, int32_t* cu_q, int32_t* kv_lens,
                          int32_t* positions, int64_t* slots, int32_t* tree, cudaStream_t stream) {
    if (B < 0 || T < 0 || table_width < 0 || free_capacity < 0 || page_size <= 0) return MHC_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 30;
    if (B > mhc::STEP_SEQUENCES || T > MAX_T || free_capacity > most || page_size > (1 << 20) || table_width > most ||
        B * table_width > most || table_stride > MAX_STRIDE)
        return MHC_ERR_UNSUPPORTED;
    if (B > 1 && table_stride < table_width) return MHC_ERR_INVALID_ARG;
    mhc_status st;
    if ((st = check_counted(new_lens, 4, B)) != MHC_OK || (st = check_counted(lens, 4, B)) != MHC_OK ||
        (st = check_counted(held, 4, B)) != MHC_OK || (st = check_counted(kv_lens, 4, B)) != MHC_OK ||
        (st = check_counted(page_table, 4, B * table_width)) != MHC_OK ||
        (st = check_counted(free_pages, 4, free_capacity)) != MHC_OK || (st = check_plain(free_count, 4)) != MHC_OK ||
        (st = check_plain(cu_q, 4)) != MHC_OK || (st = check_counted(positions, 4, T)) != MHC_OK ||
        (st = check_counted(slots, 8, T)) != MHC_OK)
        return st;
    if (T > 0 && (parents == nullptr) != (tree == nullptr)) return MHC_ERR_INVALID_ARG;
    if (T > 0 && parents != nullptr) {
        if (tree_words <= 0) return MHC_ERR_INVALID_ARG;
        if (tree_words > mhc::TREE_MOST / 32) return MHC_ERR_UNSUPPORTED;
        if ((st = check_plain(parents, 4)) != MHC_OK || (st = check_plain(tree, 4)) != MHC_OK) return st;
    }
    // blocks read the inputs, and what is brought up to date, while outputs are written
    const int64_t words = T > 0 && tree != nullptr ? T * tree_words : 0;
    const Numbers table = {page_table, B, table_width, table_stride};
    const Numbers runs[] = {{held, 1, B, 0},     {free_pages, 1, free_capacity, 0}, {free_count, 1, 1, 0},
                            {cu_q, 1, B + 1, 0}, {kv_lens, 1, B, 0},                {positions, 1, T, 0},
                            {slots, 1, 2 * T, 0}, {tree, 1, words, 0},              {new_lens, 1, B, 0},
                            {lens, 1, B, 0},     {parents, 1, T, 0}};
    constexpr int WRITTEN = 8, RUNS = 11;   // the last ones are only read, and may be the same
    for (int i = 0; i < RUNS; ++i) {
        if (meet(table, runs[i])) return MHC_ERR_INVALID_ARG;
        for (int j = 0; j < i && j < WRITTEN; ++j)
            if (meet(runs[i], runs[j])) return MHC_ERR_INVALID_ARG;
    }
    mhc::StepParams p = {};
    p.new_lens = new_lens;
    p.lens = lens;
    p.parents = parents;
    p.table = page_table;
    p.held = held;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.positions = positions;
    p.tree = T > 0 ? tree : nullptr;
    p.slots = slots;
    p.table_stride = table_stride;
    p.width = table_width;
    p.T = T;
    p.max_len = MAX_KV;
    p.B = B;
    p.page = page_size;
    p.page_shift = shift_of(page_size);
    p.cap = static_cast<int>(free_capacity);
    p.words = tree_words;
    return from_cuda(mhc::launch_paged_step(p, stream));
}

mhc_status mhc_cache_keep(mhc_dtype dt, void* const* k_caches, int64_t k_page_stride, int64_t k_slot_stride,
                          int64_t k_head_stride, void* const* v_caches, int64_t v_page_stride, int64_t v_slot_stride,
                          int64_t v_head_stride, int layers, int64_t num_pages, int page_size,
                          const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                          const int32_t* kv_lens, int64_t max_kv, int B, int Hk, int Dh, const int32_t* path,
                          int64_t path_stride, int max_keep, const int32_t* keep, int32_t* lens, cudaStream_t stream) {
    mhc_status st = check_heads(dt, 0, Hk, Hk, Dh);
    if (st != MHC_OK) return st;
    if (B < 0 || layers < 0 || max_keep < 0 || max_kv < 0) return MHC_ERR_INVALID_ARG;
    if (B > (1 << 24) || max_kv > MAX_KV || path_stride > MAX_STRIDE || table_stride > MAX_STRIDE)
        return MHC_ERR_UNSUPPORTED;
    if (B == 0 || layers == 0 || max_keep == 0) return MHC_OK;
    if (k_caches == nullptr || v_caches == nullptr || path_stride < max_keep) return MHC_ERR_INVALID_ARG;
    if ((st = check_ptrs(k_caches, layers)) != MHC_OK || (st = check_ptrs(v_caches, layers)) != MHC_OK) return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, k_page_stride, k_slot_stride, k_head_stride)) != MHC_OK)
        return st;
    if ((st = check_cache(dt, num_pages, page_size, Hk, Dh, v_page_stride, v_slot_stride, v_head_stride)) != MHC_OK)
        return st;
    if (table_stride < (max_kv + page_size - 1) / page_size) return MHC_ERR_INVALID_ARG;
    const void* numbers[] = {page_table, cu_q, kv_lens, path, keep};
    for (const void* n : numbers)
        if ((st = check_plain(n, 4)) != MHC_OK) return st;
    if (lens != nullptr && (st = check_plain(lens, 4)) != MHC_OK) return st;
    const Numbers read[] = {{page_table, B, (max_kv + page_size - 1) / page_size, table_stride},
                            {cu_q, 1, int64_t(B) + 1, 0}, {kv_lens, 1, B, 0}, {path, B, max_keep, path_stride},
                            {keep, 1, B, 0}};
    for (const Numbers& r : read)   // blocks of other caches read them while `lens` is written
        if (meet(r, {lens, 1, B, 0})) return MHC_ERR_INVALID_ARG;
    const int64_t e = dt == MHC_BF16 ? 2 : 4;
    mhc::KeepParams p = {};
    p.table = page_table;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.path = path;
    p.keep = keep;
    p.k_page = k_page_stride * e;
    p.k_slot = k_slot_stride * e;
    p.k_head = k_head_stride * e;
    p.v_page = v_page_stride * e;
    p.v_slot = v_slot_stride * e;
    p.v_head = v_head_stride * e;
    p.table_stride = table_stride;
    p.path_stride = path_stride;
    p.num_pages = num_pages;
    p.max_kv = max_kv;
    p.page = page_size;
    p.page_shift = shift_of(page_size);
    p.max_keep = max_keep;
    p.head_pieces = static_cast<int>(Dh * e / 16);
    p.row_pieces = Hk * p.head_pieces;
    for (int l0 = 0; l0 < layers; l0 += mhc::KEEP_LAYERS) {
        p.layers = layers - l0 < mhc::KEEP_LAYERS ? layers - l0 : mhc::KEEP_LAYERS;
        for (int i = 0; i < p.layers; ++i) {
            p.k[i] = k_caches[l0 + i];
            p.v[i] = v_caches[l0 + i];
        }
        p.lens = l0 == 0 ? lens : nullptr;
        const cudaError_t err = mhc::launch_cache_keep(p, B, stream);
        if (err != cudaSuccess) return from_cuda(err);
    }
    return MHC_OK;
}

}  // extern "C"
