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

}  // namespace api
}  // namespace gdn
