// tree_attention.cu -- attention of a tree of drafted tokens of each sequence over
// a paged cache: every node sees the tokens before the tree, and those nodes
// that its 64-bit word names.
//
//   out[t] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_t . k_j - m),
//   j < len - n, and j = len - n + i for every bit i of word t (n nodes)
//
// Bound by HBM as long as a kv head has few rows (nodes x query heads), by the
// products beyond some 280 (4 rows D flops for 4 D bytes). Up to 64 rows take the
// kernels of a line of tokens, with the word as their mask; more rows in bf16
// attn_wide_kernel, where boxes of a tensor map fit the pages (tokens of a page a
// multiple of 64, or 8, 16 or 32); what is left, and fp32, the warp-level kernel
// (attention.cuh, where all stand with what they measured).
#include "attention.cuh"

namespace gdn {

size_t tree_attn_workspace_size(const KvLayout &c, int n_seqs, int T, int H, int max_pages) {
  return workspace_size<true>(c, n_seqs, T, H, max_pages);
}

cudaError_t launch_tree_attention(const AttnArgs &a, cudaStream_t stream) {
  return launch_attention<true>(a, stream);
}

}  // namespace gdn
