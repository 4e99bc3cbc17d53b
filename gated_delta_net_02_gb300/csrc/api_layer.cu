// api_layer.cu -- C entry points of the attention layer's operators (declared
// in include/gdn.h): argument validation and dispatch to their kernels.
#include <cuda_runtime.h>

#include <cmath>

#include "api_util.h"
#include "gdn.h"
#include "kernels.h"

using namespace gdn::api;

namespace {

struct Buf {
  const char *name;
  const void *p;
  size_t bytes;
};

gdn_status check_aligned(const char *fn, const Buf &b) {
  if (!aligned16(b.p))
    return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, b.name);
  return GDN_OK;
}

// GDN_ERR_INVALID_ARG if `out` shares bytes with `b` (either may be NULL).
gdn_status check_apart(const char *fn, const Buf &out, const Buf &b) {
  if (out.p && b.p && ranges_overlap(out.p, out.bytes, b.p, b.bytes))
    return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, b.name);
  return GDN_OK;
}

bool dtype_ok(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }

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
  a.x = x; a.residual = residual; a.weight = weight;
  a.residual_out = residual_out; a.out = out;
  a.out_fp8 = static_cast<unsigned char *>(out_fp8); a.out_scale = out_scale;
  a.rows = s.rows; a.cols = s.cols;
  a.bf16 = s.dtype == GDN_BF16; a.normalize = s.normalize != 0;
  a.eps = s.eps; a.weight_offset = s.weight_offset;
  return check_launch(gdn::launch_norm_fp8(a, reinterpret_cast<cudaStream_t>(stream)),
                      "gdn_rmsnorm_fp8 launch");
}

}  // extern "C"
