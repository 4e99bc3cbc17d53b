// tree_attention.cu -- attention of a tree of drafted tokens of each sequence over
// a paged cache: every node sees the tokens before the tree, and those nodes
// that its 64-bit word names (attention.cuh).
#include "attention.cuh"

namespace gdn {

size_t tree_attn_workspace_size(const KvLayout &c, int n_seqs, int T, int H, int max_pages) {
  return workspace_size<true>(c, n_seqs, T, H, max_pages);
}

cudaError_t launch_tree_attention(const AttnArgs &a, cudaStream_t stream) {
  return launch_attention<true>(a, stream);
}

}  // namespace gdn
