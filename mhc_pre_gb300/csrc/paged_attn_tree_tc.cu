// paged_attn_tree_tc.cu -- attention of trees of drafted tokens over a paged
// cache on the tensor cores: the kernel of paged_attn_tc.cuh with TREE on.
#include "paged_attn_tc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tree_tc_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_tc_error, word); }

cudaError_t launch_tree_attn_tc(const AttnParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    auto fn = tensor_map_encoder();
    return fn != nullptr ? attn_tc::launch_all<true>(p, fn, s) : cudaErrorNotSupported;
}

}  // namespace mhc
