// qk_norm_rope.cu -- per-head RMSNorm of queries and keys with the position
// rotation: the training forward, and the serving form that writes keys and
// values into a paged cache.  The mathematics and the shared parts are in
// qk_norm_rope.cuh.
// Bound by memory traffic: at T = 32768, 40 + 8 heads of 128, bf16, 138 us,
// 5.85 TB/s, 0.87 of the measured copy rate; 4096 tokens into the cache 25 us;
// one token 3.5 us, a round of loads and its reduction.
#include "qk_norm_rope_fwd.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_qk_error(unsigned* word) { return g_error_word.read_and_clear(g_qk_error, word); }

cudaError_t launch_qk_norm_rope(bool bf16, bool adjacent, bool append, const QkParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    using B = __nv_bfloat16;
    if (bf16) {
        if (append) return adjacent ? qk::launch_fwd<B, true, true, true>(p, s) : qk::launch_fwd<B, false, true, true>(p, s);
        return adjacent ? qk::launch_fwd<B, true, false, true>(p, s) : qk::launch_fwd<B, false, false, true>(p, s);
    }
    if (append) return adjacent ? qk::launch_fwd<float, true, true, true>(p, s) : qk::launch_fwd<float, false, true, true>(p, s);
    return adjacent ? qk::launch_fwd<float, true, false, true>(p, s) : qk::launch_fwd<float, false, false, true>(p, s);
}

}  // namespace mhc
