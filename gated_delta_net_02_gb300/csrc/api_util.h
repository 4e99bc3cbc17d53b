// api_util.h -- what the C entry points share (defined in api.cu): the
// calling thread's message, argument checks and the device error word.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {
namespace api {

// Records the message of gdn_last_error and returns `st`.
__attribute__((format(printf, 2, 3))) gdn_status fail(gdn_status st, const char *fmt, ...);

// Device address of the current device's error word (looked up once per device).
gdn_status device_err_ptr(int **out);

// GDN_OK, or GDN_ERR_CUDA with the launch's error as the message.
gdn_status check_launch(cudaError_t e, const char *what);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool ranges_overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

struct Buf {
  const char *name;
  const void *p;
  size_t bytes;
};

inline gdn_status check_aligned(const char *fn, const Buf &b) {
  if (!aligned16(b.p))
    return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, b.name);
  return GDN_OK;
}

// GDN_ERR_INVALID_ARG if `out` shares bytes with `b` (either may be NULL).
inline gdn_status check_apart(const char *fn, const Buf &out, const Buf &b) {
  if (out.p && b.p && ranges_overlap(out.p, out.bytes, b.p, b.bytes))
    return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, b.name);
  return GDN_OK;
}

inline bool head_size_ok(int d) { return d == 64 || d == 128; }

// Resolves the grouped-query fields: H_qk = 0 means H; H_qk must divide H.
inline gdn_status qk_heads(const char *fn, int H, int H_qk, int qk_map, int *hq) {
  *hq = H_qk == 0 ? H : H_qk;
  if (*hq <= 0 || *hq > H || H % *hq != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: H_qk=%d must divide H=%d", fn, H_qk, H);
  if (qk_map != GDN_QK_TILED && qk_map != GDN_QK_GROUPED)
    return fail(GDN_ERR_INVALID_ARG, "%s: qk_map %d", fn, qk_map);
  return GDN_OK;
}

inline bool dtype_ok(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }

}  // namespace api
}  // namespace gdn
