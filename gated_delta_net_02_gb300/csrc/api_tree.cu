// api_tree.cu -- C entry points of the operators that verify a tree of drafts
// and take the tokens (declared in include/gdn.h): argument validation and
// dispatch to their kernels.
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "gdn.h"
#include "kernels.h"

using namespace gdn::api;

extern "C" {

gdn_status gdn_sample(const gdn_sample_shape *shape, const void *logits, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p,
                      const float *uniform, int32_t *tokens, float *probs, gdn_stream_t stream) {
  const char *fn = "gdn_sample";
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_sample_shape &s = *shape;
  if (s.rows < 0 || s.vocab < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: rows=%d vocab=%d", fn, s.rows, s.vocab);
  if (!dtype_ok(s.dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: dtype %d", fn, (int)s.dtype);
  const long long stride = s.row_stride == 0 ? s.vocab : s.row_stride;
  if (stride < s.vocab)
    return fail(GDN_ERR_INVALID_ARG, "%s: row_stride=%lld is below vocab=%d", fn, stride, s.vocab);
  if (s.vocab > (1 << 18) || s.rows > (1 << 24) || stride > (1LL << 32))
    return fail(GDN_ERR_UNSUPPORTED, "%s: rows=%d vocab=%d row_stride=%lld (at most 2^24, 2^18, 2^32)",
                fn, s.rows, s.vocab, stride);
  if (s.rows == 0) return GDN_OK;
  const size_t e = s.dtype == GDN_BF16 ? 2 : 4, n = (size_t)s.rows;
  const Buf in[] = {{"logits", logits, e * ((n - 1) * (size_t)stride + (size_t)s.vocab)},
                    {"uniform", uniform, 4 * n},
                    {"temperature", temperature, 4 * n},
                    {"top_k", top_k, 4 * n},
                    {"top_p", top_p, 4 * n},
                    {"min_p", min_p, 4 * n}};
  const Buf outs[] = {{"tokens", tokens, 4 * n}, {"probs", probs, 4 * n}};
  gdn_status st;
  for (const Buf &b : in) {
    if (!b.p && &b <= &in[1]) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, b.name);
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
  }
  if (!tokens) return fail(GDN_ERR_INVALID_ARG, "%s: tokens is NULL", fn);
  for (const Buf &o : outs) {
    if ((st = check_aligned(fn, o)) != GDN_OK) return st;
    for (const Buf &b : in)
      if ((st = check_apart(fn, o, b)) != GDN_OK) return st;
  }
  if ((st = check_apart(fn, outs[0], outs[1])) != GDN_OK) return st;
  gdn::SampleArgs a{};
  a.logits = logits; a.stride = stride;
  a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.uniform = uniform; a.tokens = tokens; a.probs = probs;
  a.rows = s.rows; a.vocab = s.vocab; a.bf16 = s.dtype == GDN_BF16;
  return check_launch(gdn::launch_sample(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_sample launch");
}

}  // extern "C"
