// api_layer.cu -- C entry points of the attention layer's operators (declared
// in include/gdn.h): argument validation and dispatch to their kernels.
#include <cuda_runtime.h>

#include <limits.h>

#include <cmath>

#include "api_util.h"
#include "gdn.h"
#include "kernels.h"

using namespace gdn::api;

namespace {

// Checks a cache layout and resolves its strides; *bytes is the extent of
// each of its two buffers.
gdn_status kv_layout(const char *fn, const gdn_kv_cache *cache, gdn::KvLayout *l, size_t *bytes) {
  if (!cache) return fail(GDN_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  const gdn_kv_cache &c = *cache;
  if (c.n_pages < 0 || c.page_size < 1 || c.H_kv < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: n_pages=%d page_size=%d H_kv=%d", fn, c.n_pages,
                c.page_size, c.H_kv);
  if (!dtype_ok(c.dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: cache dtype %d", fn, (int)c.dtype);
  if (c.D != 64 && c.D != 128 && c.D != 256)
    return fail(c.D < 1 ? GDN_ERR_INVALID_ARG : GDN_ERR_UNSUPPORTED,
                "%s: head size D=%d (supported: 64, 128, 256)", fn, c.D);
  if (c.H_kv > (1 << 20))
    return fail(GDN_ERR_UNSUPPORTED, "%s: H_kv=%d is above 2^20", fn, c.H_kv);
  const long long most = 1LL << 60;
  long long ps = c.page_stride, ts = c.token_stride, hs = c.head_stride;
  if (!ps && !ts && !hs) {
    hs = c.D;
    ts = (long long)c.H_kv * c.D;
    ps = ts * c.page_size;
    if (c.n_pages && ps > most / c.n_pages)
      return fail(GDN_ERR_UNSUPPORTED, "%s: the cache is too large", fn);
  } else {
    const long long m = c.dtype == GDN_BF16 ? 8 : 4;
    if (ps <= 0 || ts <= 0 || hs <= 0 || ps % m || ts % m || hs % m)
      return fail(GDN_ERR_INVALID_ARG,
                  "%s: cache strides %lld, %lld, %lld (need positive multiples of 16 bytes)", fn,
                  ps, ts, hs);
    if (ps > most / (c.n_pages + 1LL) || ts > most / c.page_size || hs > most / c.H_kv)
      return fail(GDN_ERR_UNSUPPORTED, "%s: the cache is too large", fn);
    // each (page, token, head) has D elements of its own: true when, in the
    // order of their strides, each level steps over all of the level below
    struct { long long stride, n; } lv[3] = {{ps, c.n_pages}, {ts, c.page_size}, {hs, c.H_kv}};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (lv[j].stride > lv[j + 1].stride) {
          const auto t = lv[j];
          lv[j] = lv[j + 1];
          lv[j + 1] = t;
        }
    long long span = c.D;
    for (int i = 0; i < 3; ++i) {
      if (lv[i].n > 1 && lv[i].stride < span)
        return fail(GDN_ERR_INVALID_ARG, "%s: the cache's strides make its rows overlap", fn);
      if (lv[i].n > 1) span += (lv[i].n - 1) * lv[i].stride;
    }
  }
  *l = gdn::KvLayout{c.n_pages, c.page_size, c.H_kv, c.D, c.dtype == GDN_BF16, ps, ts, hs};
  const size_t e = c.dtype == GDN_BF16 ? 2 : 4;
  *bytes = c.n_pages == 0 ? 0
                          : e * (size_t)((c.n_pages - 1) * ps + (c.page_size - 1) * ts +
                                         (c.H_kv - 1) * hs + c.D);
  return GDN_OK;
}

// Whether rows of two buffers with the layout `l` share elements, the second
// `delta` elements behind the first: a difference of places
//   dp * page_stride + dt * token_stride + dh * head_stride
// comes within D of it. kv_layout has seen to it that each level steps over
// all of the level below, so at each level, largest stride first, only the two
// counts around what is left can come that near.
bool rows_collide(const gdn::KvLayout &l, long long delta) {
  struct { long long stride, n; } lv[3] = {
      {l.page_stride, l.n_pages}, {l.token_stride, l.page_size}, {l.head_stride, l.H_kv}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (lv[j].stride < lv[j + 1].stride) {
        const auto t = lv[j];
        lv[j] = lv[j + 1];
        lv[j + 1] = t;
      }
  for (int pick = 0; pick < 8; ++pick) {
    long long left = delta;
    for (int i = 0; i < 3; ++i) {
      if (lv[i].n <= 1) continue;
      long long c = left / lv[i].stride - (left % lv[i].stride < 0) + (pick >> i & 1);
      const long long most = lv[i].n - 1;
      c = c > most ? most : c < -most ? -most : c;
      left -= c * lv[i].stride;
    }
    if (left > -l.D && left < l.D) return true;
  }
  return false;
}

// Checks the sizes of an attention call; cache layout as kv_layout.
gdn_status attn_shape(const char *fn, const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                      gdn::KvLayout *l, size_t *cache_bytes) {
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_attn_shape &s = *shape;
  const gdn_status st = kv_layout(fn, cache, l, cache_bytes);
  if (st != GDN_OK) return st;
  if (s.n_seqs < 0 || s.T < 0 || s.H < 1 || s.max_pages < 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs=%d T=%d H=%d max_pages=%d", fn, s.n_seqs, s.T,
                s.H, s.max_pages);
  if (s.H % l->H_kv != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: H_kv=%d must divide H=%d", fn, l->H_kv, s.H);
  if (s.kv_map != GDN_QK_TILED && s.kv_map != GDN_QK_GROUPED)
    return fail(GDN_ERR_INVALID_ARG, "%s: kv_map %d", fn, (int)s.kv_map);
  if (!std::isfinite(s.scale)) return fail(GDN_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  if ((long long)s.n_seqs * s.T > (1LL << 30) / s.H)
    return fail(GDN_ERR_UNSUPPORTED, "%s: %d x %d tokens x %d heads too large", fn, s.n_seqs, s.T,
                s.H);
  return GDN_OK;
}

// Checks a call that rotates and appends, and fills its arguments (n_tokens = 0:
// nothing to do). The norm's weights may be NULL.
gdn_status rope_args(const char *fn, const gdn_rope_shape *shape, const gdn_kv_cache *cache,
                     const void *q, const void *k, const void *v, const void *q_weight,
                     const void *k_weight, const int32_t *positions, const float *inv_freq,
                     const int64_t *slots, void *q_out, void *k_cache, void *v_cache,
                     gdn::RopeArgs &a) {
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_rope_shape &s = *shape;
  size_t cache_bytes = 0;
  gdn_status st = kv_layout(fn, cache, &a.cache, &cache_bytes);
  if (st != GDN_OK) return st;
  const int D = a.cache.D, H_kv = a.cache.H_kv;
  if (s.n_tokens < 0 || s.H < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: n_tokens=%d H=%d", fn, s.n_tokens, s.H);
  if (s.H > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "%s: H=%d is above 2^20", fn, s.H);
  if (s.rot_dim < 0 || s.rot_dim > D || (s.rot_dim & 1))
    return fail(GDN_ERR_INVALID_ARG, "%s: rot_dim=%d (need even, 0 to D=%d)", fn, s.rot_dim, D);
  if (s.pairs != GDN_ROPE_HALVES && s.pairs != GDN_ROPE_NEIGHBOURS)
    return fail(GDN_ERR_INVALID_ARG, "%s: pairs %d", fn, (int)s.pairs);
  if (s.axes != GDN_ROPE_AXES_SECTIONED && s.axes != GDN_ROPE_AXES_INTERLEAVED)
    return fail(GDN_ERR_INVALID_ARG, "%s: axes %d", fn, (int)s.axes);
  if (s.n_axes < 1 || s.n_axes > 4)
    return fail(GDN_ERR_INVALID_ARG, "%s: n_axes=%d (need 1 to 4)", fn, s.n_axes);
  const int half = s.rot_dim / 2;
  int left = half;
  for (int i = 0; i < s.n_axes; ++i) {
    if (s.section[i] < 0 || s.section[i] > left)
      return fail(GDN_ERR_INVALID_ARG, "%s: the sections do not sum to rot_dim / 2 = %d", fn, half);
    // taking turns, axis i > 0 has the frequencies i, i + n_axes, ... below half
    if (s.axes == GDN_ROPE_AXES_INTERLEAVED && i > 0 &&
        s.section[i] > (half - i + s.n_axes - 1) / s.n_axes)
      return fail(GDN_ERR_INVALID_ARG, "%s: section[%d]=%d is more than the axis's turns", fn, i,
                  s.section[i]);
    left -= s.section[i];
  }
  if (left)
    return fail(GDN_ERR_INVALID_ARG, "%s: the sections do not sum to rot_dim / 2 = %d", fn, half);
  const long long m = a.cache.bf16 ? 8 : 4;
  const long long dense[3] = {(long long)s.H * D, (long long)H_kv * D, (long long)H_kv * D};
  long long stride[3] = {s.q_stride, s.k_stride, s.v_stride};
  const char *names[3] = {"q_stride", "k_stride", "v_stride"};
  for (int i = 0; i < 3; ++i) {
    if (stride[i] == 0) stride[i] = dense[i];
    if (stride[i] < dense[i] || stride[i] % m || stride[i] > (1LL << 28))
      return fail(GDN_ERR_INVALID_ARG,
                  "%s: %s=%lld (need a multiple of 16 bytes from %lld to 2^28)", fn, names[i],
                  stride[i], dense[i]);
  }
  a.n_tokens = s.n_tokens;
  if (s.n_tokens == 0) return GDN_OK;
  const size_t e = a.cache.bf16 ? 2 : 4, n = (size_t)s.n_tokens;
  const Buf in[] = {{"q", q, e * ((n - 1) * (size_t)stride[0] + (size_t)dense[0])},
                    {"k", k, e * ((n - 1) * (size_t)stride[1] + (size_t)dense[1])},
                    {"v", v, e * ((n - 1) * (size_t)stride[2] + (size_t)dense[2])},
                    {"positions", positions, 4 * n * s.n_axes},
                    {"slots", slots, 8 * n},
                    {"inv_freq", inv_freq, 4 * (size_t)half},
                    {"q_weight", q_weight, e * (size_t)D},
                    {"k_weight", k_weight, e * (size_t)D}};
  const Buf outs[] = {{"q_out", q_out, e * n * (size_t)dense[0]},
                      {"k_cache", k_cache, cache_bytes},
                      {"v_cache", v_cache, cache_bytes}};
  for (const Buf &b : in) {
    const bool optional = &b == &in[5] ? half == 0 : &b > &in[5];
    if (!b.p && !optional)
      return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, b.name);
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
  }
  for (int i = 0; i < 3; ++i) {
    if (!outs[i].p) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, outs[i].name);
    if ((st = check_aligned(fn, outs[i])) != GDN_OK) return st;
    for (const Buf &b : in)
      if ((st = check_apart(fn, outs[i], b)) != GDN_OK) return st;
  }
  // one buffer may hold both caches interleaved (strides twice as long), so
  // the two are compared row by row
  if (k_cache == v_cache)
    return fail(GDN_ERR_INVALID_ARG, "%s: k_cache and v_cache are the same", fn);
  if (ranges_overlap(k_cache, cache_bytes, v_cache, cache_bytes) &&
      rows_collide(a.cache, (static_cast<const char *>(v_cache) -
                             static_cast<const char *>(k_cache)) / (long long)e))
    return fail(GDN_ERR_INVALID_ARG, "%s: rows of k_cache and v_cache overlap", fn);
  for (int i = 1; i < 3; ++i)
    if ((st = check_apart(fn, outs[0], outs[i])) != GDN_OK) return st;
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  a.q = q; a.k = k; a.v = v;
  a.q_stride = stride[0]; a.k_stride = stride[1]; a.v_stride = stride[2];
  a.positions = positions; a.inv_freq = inv_freq; a.slots = slots;
  a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
  a.H = s.H; a.rot_dim = s.rot_dim; a.n_axes = s.n_axes;
  for (int i = 0; i < 4; ++i) a.section[i] = i < s.n_axes ? s.section[i] : 0;
  a.neighbours = s.pairs == GDN_ROPE_NEIGHBOURS;
  a.interleaved = s.axes == GDN_ROPE_AXES_INTERLEAVED;
  return GDN_OK;
}

// Checks an attention call and fills its arguments (n_seqs or T 0: nothing to
// do). `size` is its kernels' workspace.
gdn_status attn_args(const char *fn, const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                     const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *page_table, const int32_t *lens, void *out, void *workspace,
                     size_t workspace_bytes,
                     size_t (*size)(const gdn::KvLayout &, int, int, int, int), gdn::AttnArgs &a) {
  size_t cache_bytes = 0;
  gdn_status st = attn_shape(fn, shape, cache, &a.cache, &cache_bytes);
  if (st != GDN_OK) return st;
  const gdn_attn_shape &s = *shape;
  a.n_seqs = s.n_seqs; a.T = s.T;
  if (s.n_seqs == 0 || s.T == 0) return GDN_OK;
  const size_t e = a.cache.bf16 ? 2 : 4, rows = (size_t)s.n_seqs * s.T * s.H;
  const size_t need = size(a.cache, s.n_seqs, s.T, s.H, s.max_pages);
  const Buf in[] = {{"q", q, e * rows * a.cache.D},
                    {"k_cache", k_cache, cache_bytes},
                    {"v_cache", v_cache, cache_bytes},
                    {"page_table", page_table, 4 * (size_t)s.n_seqs * s.max_pages},
                    {"lens", lens, 4 * (size_t)s.n_seqs}};
  const Buf outs[] = {{"out", out, e * rows * a.cache.D}, {"workspace", workspace, need}};
  for (const Buf &b : in) {
    // no pages: every sequence is empty, and nothing of them is read
    if (!b.p && !(b.bytes == 0 && &b != &in[0]))
      return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, b.name);
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
  }
  for (const Buf &o : outs) {
    if (!o.p) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, o.name);
    if ((st = check_aligned(fn, o)) != GDN_OK) return st;
    for (const Buf &b : in)
      if ((st = check_apart(fn, o, b)) != GDN_OK) return st;
  }
  if ((st = check_apart(fn, outs[0], outs[1])) != GDN_OK) return st;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  if (workspace_bytes < need)
    return fail(GDN_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes,
                need);
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.table = page_table; a.lens = lens; a.out = out; a.workspace = workspace;
  a.H = s.H; a.max_pages = s.max_pages;
  a.grouped = s.kv_map == GDN_QK_GROUPED;
  a.scale = s.scale != 0.f ? s.scale : 1.0f / std::sqrt((float)a.cache.D);
  return GDN_OK;
}

constexpr int kMostNodes = 64;  // bits of a tree's word

gdn_status tree_shape(const char *fn, const gdn_attn_shape *shape) {
  if (shape->T > kMostNodes)
    return fail(GDN_ERR_UNSUPPORTED, "%s: T=%d nodes (at most %d)", fn, shape->T, kMostNodes);
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_rmsnorm_fp8(const gdn_norm_shape *shape, const void *x, const void *residual,
                           const void *weight, void *residual_out, void *out, void *out_fp8,
                           float *out_scale, gdn_stream_t stream) {
  const char *fn = "gdn_rmsnorm_fp8";
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_norm_shape &s = *shape;
  if (s.rows < 0 || s.cols < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: rows=%d cols=%d", fn, s.rows, s.cols);
  // column indexes step by up to 256 in 32 bits
  if (s.cols > INT_MAX - 1023)
    return fail(GDN_ERR_UNSUPPORTED, "%s: cols=%d is above 2^31 - 1024", fn, s.cols);
  if (!dtype_ok(s.dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: dtype %d", fn, (int)s.dtype);
  if (s.normalize != 0 && s.normalize != 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: normalize %d", fn, s.normalize);
  if (!std::isfinite(s.eps) || s.eps < 0.f)
    return fail(GDN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  if (!std::isfinite(s.weight_offset))
    return fail(GDN_ERR_INVALID_ARG, "%s: weight_offset is not finite", fn);
  if (!s.normalize && weight)
    return fail(GDN_ERR_INVALID_ARG, "%s: weight is given with normalize = 0", fn);
  if (s.rows == 0) return GDN_OK;
  if (!x) return fail(GDN_ERR_INVALID_ARG, "%s: x is NULL", fn);
  if (!out_fp8 != !out_scale)
    return fail(GDN_ERR_INVALID_ARG, "%s: out_fp8 and out_scale come together", fn);
  if (!out && !out_fp8)
    return fail(GDN_ERR_INVALID_ARG, "%s: out and out_fp8 are both NULL", fn);

  const size_t e = s.dtype == GDN_BF16 ? 2 : 4, n = (size_t)s.rows * s.cols;
  const Buf in[] = {{"x", x, n * e}, {"residual", residual, n * e},
                    {"weight", weight, (size_t)s.cols * e}};
  const Buf outs[] = {{"residual_out", residual_out, n * e},
                      {"out", out, n * e},
                      {"out_fp8", out_fp8, n},
                      {"out_scale", out_scale, 4 * (size_t)s.rows * ((s.cols + 127) / 128)}};
  gdn_status st;
  for (const Buf &b : in)
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
  for (int i = 0; i < 4; ++i) {
    if ((st = check_aligned(fn, outs[i])) != GDN_OK) return st;
    for (const Buf &b : in) {
      // each element is read before the same thread writes it, so the two
      // outputs of x's type may be x or residual itself
      const bool in_place = i < 2 && outs[i].p == b.p && b.p != weight;
      if (!in_place && (st = check_apart(fn, outs[i], b)) != GDN_OK) return st;
    }
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(fn, outs[i], outs[j])) != GDN_OK) return st;
  }

  gdn::NormArgs a{};
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  a.x = x; a.residual = residual; a.weight = weight;
  a.residual_out = residual_out; a.out = out;
  a.out_fp8 = static_cast<unsigned char *>(out_fp8); a.out_scale = out_scale;
  a.rows = s.rows; a.cols = s.cols;
  a.bf16 = s.dtype == GDN_BF16; a.normalize = s.normalize != 0;
  a.eps = s.eps; a.weight_offset = s.weight_offset;
  return check_launch(gdn::launch_norm_fp8(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_rmsnorm_fp8 launch");
}

gdn_status gdn_gemm_fp8(const gdn_gemm_shape *shape, const void *a, const float *a_scale,
                        const void *b, const float *b_scale, void *out, gdn_stream_t stream) {
  const char *fn = "gdn_gemm_fp8";
  if (!shape) return fail(GDN_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const gdn_gemm_shape &s = *shape;
  if (s.M < 0 || s.N < 0 || s.K < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: M=%d N=%d K=%d", fn, s.M, s.N, s.K);
  if (!dtype_ok(s.out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: out_dtype %d", fn, (int)s.out_dtype);
  if (s.K % 16)
    return fail(GDN_ERR_UNSUPPORTED, "%s: K=%d is no multiple of 16", fn, s.K);
  if (s.M > (1 << 21) || s.N > (1 << 21) || s.K > (1 << 21))
    return fail(GDN_ERR_UNSUPPORTED, "%s: M=%d N=%d K=%d above 2^21", fn, s.M, s.N, s.K);
  if (s.M == 0 || s.N == 0) return GDN_OK;
  const size_t M = (size_t)s.M, N = (size_t)s.N, K = (size_t)s.K, kb = (K + 127) / 128;
  const Buf in[] = {{"a", a, M * K},
                    {"a_scale", a_scale, 4 * M * kb},
                    {"b", b, N * K},
                    {"b_scale", b_scale, 4 * ((N + 127) / 128) * kb}};
  const Buf o = {"out", out, M * N * (s.out_dtype == GDN_BF16 ? 2 : 4)};
  gdn_status st;
  for (const Buf &x : in) {
    if (!x.p) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, x.name);
    if ((st = check_aligned(fn, x)) != GDN_OK) return st;
  }
  if (!o.p) return fail(GDN_ERR_INVALID_ARG, "%s: out is NULL", fn);
  if ((st = check_aligned(fn, o)) != GDN_OK) return st;
  for (const Buf &x : in)
    if ((st = check_apart(fn, o, x)) != GDN_OK) return st;
  gdn::GemmArgs g{};
  if ((st = device_err_ptr(&g.err)) != GDN_OK) return st;
  g.a = a; g.a_scale = a_scale; g.b = b; g.b_scale = b_scale; g.out = out;
  g.M = s.M; g.N = s.N; g.K = s.K; g.bf16_out = s.out_dtype == GDN_BF16;
  return check_launch(gdn::launch_gemm_fp8(g, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_gemm_fp8 launch");
}

gdn_status gdn_rope_append(const gdn_rope_shape *shape, const gdn_kv_cache *cache, const void *q,
                           const void *k, const void *v, const int32_t *positions,
                           const float *inv_freq, const int64_t *slots, void *q_out,
                           void *k_cache, void *v_cache, gdn_stream_t stream) {
  gdn::RopeArgs a{};
  const gdn_status st = rope_args("gdn_rope_append", shape, cache, q, k, v, nullptr, nullptr,
                                  positions, inv_freq, slots, q_out, k_cache, v_cache, a);
  if (st != GDN_OK || a.n_tokens == 0) return st;
  return check_launch(gdn::launch_rope_append(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_rope_append launch");
}

gdn_status gdn_qknorm_rope_append(const gdn_rope_shape *shape, const gdn_kv_cache *cache,
                                  const gdn_qk_norm *norm, const void *q, const void *k,
                                  const void *v, const void *q_weight, const void *k_weight,
                                  const int32_t *positions, const float *inv_freq,
                                  const int64_t *slots, void *q_out, void *k_cache,
                                  void *v_cache, gdn_stream_t stream) {
  const char *fn = "gdn_qknorm_rope_append";
  if (!norm) return fail(GDN_ERR_INVALID_ARG, "%s: norm is NULL", fn);
  if (!std::isfinite(norm->eps) || norm->eps < 0.f)
    return fail(GDN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  if (!std::isfinite(norm->weight_offset))
    return fail(GDN_ERR_INVALID_ARG, "%s: weight_offset is not finite", fn);
  gdn::QkNormArgs a{};
  const gdn_status st = rope_args(fn, shape, cache, q, k, v, q_weight, k_weight, positions,
                                  inv_freq, slots, q_out, k_cache, v_cache, a.rope);
  if (st != GDN_OK || a.rope.n_tokens == 0) return st;
  a.q_weight = q_weight; a.k_weight = k_weight;
  a.eps = norm->eps; a.weight_offset = norm->weight_offset;
  return check_launch(gdn::launch_qknorm_rope(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_qknorm_rope_append launch");
}

size_t gdn_paged_attention_workspace_size(const gdn_attn_shape *shape, const gdn_kv_cache *cache) {
  gdn::KvLayout l;
  size_t cache_bytes = 0;
  if (attn_shape("gdn_paged_attention_workspace_size", shape, cache, &l, &cache_bytes) != GDN_OK)
    return 0;
  if (shape->n_seqs == 0 || shape->T == 0) return 0;
  return gdn::attn_workspace_size(l, shape->n_seqs, shape->T, shape->H, shape->max_pages);
}

gdn_status gdn_paged_attention(const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                               const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *page_table, const int32_t *lens, void *out,
                               void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
  gdn::AttnArgs a{};
  gdn_status st =
      attn_args("gdn_paged_attention", shape, cache, q, k_cache, v_cache, page_table, lens, out,
                workspace, workspace_bytes, gdn::attn_workspace_size, a);
  if (st != GDN_OK || a.n_seqs == 0 || a.T == 0) return st;
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  return check_launch(gdn::launch_paged_attention(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_paged_attention launch");
}

size_t gdn_tree_attention_workspace_size(const gdn_attn_shape *shape, const gdn_kv_cache *cache) {
  const char *fn = "gdn_tree_attention_workspace_size";
  gdn::KvLayout l;
  size_t cache_bytes = 0;
  if (attn_shape(fn, shape, cache, &l, &cache_bytes) != GDN_OK) return 0;
  if (tree_shape(fn, shape) != GDN_OK || shape->n_seqs == 0 || shape->T == 0) return 0;
  return gdn::tree_attn_workspace_size(l, shape->n_seqs, shape->T, shape->H, shape->max_pages);
}

gdn_status gdn_tree_attention(const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                              const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *page_table, const int32_t *lens,
                              const int32_t *n_nodes, const uint64_t *tree, void *out,
                              void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
  const char *fn = "gdn_tree_attention";
  gdn::AttnArgs a{};
  gdn_status st;
  if (shape && (st = tree_shape(fn, shape)) != GDN_OK) return st;
  st = attn_args(fn, shape, cache, q, k_cache, v_cache, page_table, lens, out, workspace,
                 workspace_bytes, gdn::tree_attn_workspace_size, a);
  if (st != GDN_OK || a.n_seqs == 0 || a.T == 0) return st;
  const size_t n = (size_t)a.n_seqs, e = a.cache.bf16 ? 2 : 4;
  const Buf in[] = {{"tree", tree, 8 * n * a.T}, {"n_nodes", n_nodes, 4 * n}};
  const Buf outs[] = {{"out", out, e * n * a.T * a.H * a.cache.D},
                      {"workspace", workspace, workspace_bytes}};
  if (!tree) return fail(GDN_ERR_INVALID_ARG, "%s: tree is NULL", fn);
  for (const Buf &b : in) {
    if ((st = check_aligned(fn, b)) != GDN_OK) return st;
    for (const Buf &o : outs)
      if ((st = check_apart(fn, o, b)) != GDN_OK) return st;
  }
  if ((st = device_err_ptr(&a.err)) != GDN_OK) return st;
  a.tree = reinterpret_cast<const unsigned long long *>(tree);
  a.n_nodes = n_nodes;
  return check_launch(gdn::launch_tree_attention(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_tree_attention launch");
}

}  // extern "C"
