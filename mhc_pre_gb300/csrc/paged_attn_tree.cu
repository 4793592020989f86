// paged_attn_tree.cu -- attention of trees of drafted tokens over a paged cache:
// the choice of kernel, and the CUDA-core kernel with TREE on.
//
// A sequence's new tokens are the nodes of a tree (or of a forest; any mask is
// taken), in any order.  Node i sees every cached token before the new ones, and
// of the new ones those whose bits its row of the mask has:
//   z_ij = scale <q_i, k_j> over those keys,  o_i = sum_j softmax(z_i)_j v_j.
// All nodes read the same context, so the tiles, the plan and the kernels are
// those of a causal chunk; only the blocks with drafted tokens differ: there a
// row's bits take the place of the diagonal, 32 keys to a word, and values that no
// row of a tile sees are zeroed like those past a sequence's end.
#include "paged_attn_cc.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tree_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_error, word); }

cudaError_t launch_tree_attn(bool bf16, const AttnParams& p, cudaStream_t s) {
    if (attn_tc_supports(bf16, p.Hq, p.Hk, p.Dh, p.page_size)) return launch_tree_attn_tc(p, s);
    g_error_word.may_be_set();
    return bf16 ? attn::launch_cc_dp<__nv_bfloat16, true>(p, s) : attn::launch_cc_dp<float, true>(p, s);
}

}  // namespace mhc
