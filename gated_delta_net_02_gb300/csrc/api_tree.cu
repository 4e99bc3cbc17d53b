// api_tree.cu -- C entry points of the operators that verify a tree of drafts
// and take the tokens (declared in include/gdn.h): argument validation and
// dispatch to their kernels.
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "gdn.h"
#include "kernels.h"

using namespace gdn::api;

namespace {

constexpr int kMostNodes = 64;  // bits of a tree's word

// Checks the sizes of a tree call of the delta rule and fills them in; false
// in *work when there is nothing to do.
gdn_status tree_args(const char *fn, const gdn_shape *shape, gdn_mode mode, gdn::TreeDeltaArgs *a,
                     bool *work) {
  *work = false;
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_shape &s = *shape;
  if (s.n_seqs < 0 || s.T < 0 || s.H <= 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs=%d T=%d H=%d", fn, s.n_seqs, s.T, s.H);
  if (mode != GDN_MODE_GDA && mode != GDN_MODE_KDA)
    return fail(GDN_ERR_INVALID_ARG, "%s: mode %d", fn, (int)mode);
  if (!dtype_ok(s.in_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: in_dtype %d", fn, (int)s.in_dtype);
  if (s.D_k <= 0 || s.D_v <= 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: D_k=%d D_v=%d", fn, s.D_k, s.D_v);
  if (!head_size_ok(s.D_k) || !head_size_ok(s.D_v))
    return fail(GDN_ERR_UNSUPPORTED, "%s: head sizes D_k=%d D_v=%d (supported: 64, 128)", fn, s.D_k,
                s.D_v);
  if (!std::isfinite(s.scale)) return fail(GDN_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  int hq = 0;
  if (qk_heads(fn, s.H, s.H_qk, (int)s.qk_map, &hq) != GDN_OK) return GDN_ERR_INVALID_ARG;
  if (s.T > kMostNodes)
    return fail(GDN_ERR_UNSUPPORTED, "%s: T=%d nodes (at most %d)", fn, s.T, kMostNodes);
  if ((long long)s.n_seqs > (1LL << 24) / s.H)
    return fail(GDN_ERR_UNSUPPORTED, "%s: %d sequences x %d heads too large", fn, s.n_seqs, s.H);
  a->n_seqs = s.n_seqs; a->T = s.T; a->H = s.H; a->Hqk = hq; a->Dk = s.D_k; a->Dv = s.D_v;
  a->qk_grouped = s.qk_map == GDN_QK_GROUPED;
  a->kda = mode == GDN_MODE_KDA;
  a->bf16 = s.in_dtype == GDN_BF16;
  a->scale = s.scale != 0.f ? s.scale : 1.0f / std::sqrt((float)s.D_k);
  *work = s.n_seqs > 0 && s.T > 0;
  return GDN_OK;
}

// Every input given and aligned, every output too and apart from all.
template <int NI, int NO>
gdn_status check_bufs(const char *fn, const Buf (&in)[NI], const Buf (&outs)[NO]) {
  gdn_status st;
  for (const Buf &b : in) {
    if (!b.p) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, b.name);
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
  }
  for (int i = 0; i < NO; ++i) {
    if (!outs[i].p) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, outs[i].name);
    if ((st = check_aligned(fn, outs[i])) != GDN_OK) return st;
    for (const Buf &b : in)
      if ((st = check_apart(fn, outs[i], b)) != GDN_OK) return st;
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(fn, outs[i], outs[j])) != GDN_OK) return st;
  }
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_tree_forward(const gdn_shape *shape, const void *q, const void *k, const void *v,
                            const float *g, const float *beta, const float *const *state_in,
                            const int32_t *n_nodes, const uint64_t *tree, float *out,
                            float *updates, gdn_mode mode, gdn_stream_t stream) {
  const char *fn = "gdn_tree_forward";
  gdn::TreeDeltaArgs a{};
  bool work;
  gdn_status st = tree_args(fn, shape, mode, &a, &work);
  if (st != GDN_OK || !work) return st;
  const size_t e = a.bf16 ? 2 : 4, n = (size_t)a.n_seqs * a.T;
  const size_t rows = 4 * n * a.H * a.Dv;
  const Buf in[] = {{"q", q, e * n * a.Hqk * a.Dk},
                    {"k", k, e * n * a.Hqk * a.Dk},
                    {"v", v, e * n * a.H * a.Dv},
                    {"g", g, 4 * n * a.H * (a.kda ? a.Dk : 1)},
                    {"beta", beta, 4 * n * a.H},
                    {"state_in", state_in, 8 * (size_t)a.n_seqs},
                    {"tree", tree, 8 * n}};
  const Buf outs[] = {{"out", out, rows}, {"updates", updates, rows}};
  if ((st = check_bufs(fn, in, outs)) != GDN_OK) return st;
  const Buf nodes = {"n_nodes", n_nodes, 4 * (size_t)a.n_seqs};
  if ((st = check_aligned(fn, nodes)) != GDN_OK) return st;
  for (const Buf &o : outs)
    if ((st = check_apart(fn, o, nodes)) != GDN_OK) return st;
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state_in = state_in;
  a.n_nodes = n_nodes; a.tree = reinterpret_cast<const unsigned long long *>(tree);
  a.out = out; a.updates = updates;
  return check_launch(gdn::launch_tree_forward(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_tree_forward launch");
}

gdn_status gdn_tree_commit(const gdn_shape *shape, const void *k, const float *g,
                           const float *updates, const float *const *state_in,
                           const uint64_t *tree, const int32_t *leaf, float *state_out,
                           gdn_mode mode, gdn_stream_t stream) {
  const char *fn = "gdn_tree_commit";
  gdn::TreeDeltaArgs a{};
  bool work;
  gdn_status st = tree_args(fn, shape, mode, &a, &work);
  if (st != GDN_OK || !work) return st;
  const size_t e = a.bf16 ? 2 : 4, n = (size_t)a.n_seqs * a.T;
  const Buf in[] = {{"k", k, e * n * a.Hqk * a.Dk},
                    {"g", g, 4 * n * a.H * (a.kda ? a.Dk : 1)},
                    {"updates", updates, 4 * n * a.H * a.Dv},
                    {"state_in", state_in, 8 * (size_t)a.n_seqs},
                    {"tree", tree, 8 * n},
                    {"leaf", leaf, 4 * (size_t)a.n_seqs}};
  const Buf outs[] = {{"state_out", state_out, 4 * (size_t)a.n_seqs * a.H * a.Dk * a.Dv}};
  if ((st = check_bufs(fn, in, outs)) != GDN_OK) return st;
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  a.k = k; a.g = g; a.updates = const_cast<float *>(updates); a.state_in = state_in;
  a.tree = reinterpret_cast<const unsigned long long *>(tree); a.leaf = leaf;
  a.state_out = state_out;
  return check_launch(gdn::launch_tree_commit(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_tree_commit launch");
}

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
