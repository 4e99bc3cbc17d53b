// paged_attention.cu -- attention of the last T tokens of each sequence, a line
// of tokens, over a paged cache (attention.cuh).
#include "attention.cuh"

namespace gdn {

size_t attn_workspace_size(const KvLayout &c, int n_seqs, int T, int H, int max_pages) {
  return workspace_size<false>(c, n_seqs, T, H, max_pages);
}

cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t stream) {
  return launch_attention<false>(a, stream);
}

}  // namespace gdn
