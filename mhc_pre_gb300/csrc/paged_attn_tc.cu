// paged_attn_tc.cu -- causal attention of new tokens over a paged cache on the
// tensor cores: the kernel of paged_attn_tc.cuh and the sizes that it takes.
#include "paged_attn_tc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tc_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_tc_error, word); }

// Boxes of 8 or more whole swizzle rows that tile a block of 128 keys, and a
// token's query heads of one key head within a lane's rows.
bool attn_tc_supports(bool bf16, int Hq, int Hk, int Dh, int page_size) {
    return bf16 && Hq / Hk <= 128 && Dh <= 128 && page_size >= 8 && (128 % page_size == 0 || page_size % 128 == 0);
}

cudaError_t launch_paged_attn_tc(const AttnParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    auto fn = tensor_map_encoder();
    return fn != nullptr ? attn_tc::launch_all<false>(p, fn, s) : cudaErrorNotSupported;
}

}  // namespace mhc
