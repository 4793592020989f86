// attn_abi.cu -- the extern "C" entry points of the attention sublayer:
// validation and dispatch only (qk_norm_rope.cu and paged_attn.cu compute).
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

size_t mhc_paged_attn_workspace_bytes(mhc_dtype dt, int64_t T, int B, int Hq, int Hk, int Dh, int page_size,
                                      int64_t max_q) {
    if (check_attn(dt, T, B, Hq, Hk, Dh, page_size, max_q, 0, 0) != MHC_OK || T == 0 || B == 0) return 0;
    const mhc::AttnPlan plan = mhc::attn_plan_sizes(dt == MHC_BF16, T, B, Hq, Hk, Dh, page_size, max_q);
    return counters_fit(plan, Hk) ? plan.total : 0;
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

mhc_status mhc_paged_attn(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache, int64_t k_page_stride,
                          int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                          int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                          const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                          const int32_t* kv_lens, int64_t T, int B, int Hq, int Hk, int Dh, int64_t max_q,
                          int64_t max_kv, int window, float scale, float softcap, void* o, float* lse,
                          void* workspace, size_t ws_bytes, cudaStream_t stream) {
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
    const mhc::AttnPlan plan = mhc::attn_plan_sizes(dt == MHC_BF16, T, B, Hq, Hk, Dh, page_size, max_q);
    if (!counters_fit(plan, Hk)) return MHC_ERR_UNSUPPORTED;
    if (ws_bytes < plan.total) return MHC_ERR_INVALID_ARG;
    if (cu_q != nullptr) {
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
    p.page_shift = -1;
    for (int i = 0; i < 21; ++i)
        if (page_size == (1 << i)) p.page_shift = i;
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
    return from_cuda(mhc::launch_paged_attn(dt == MHC_BF16, p, stream));
}

}  // extern "C"
