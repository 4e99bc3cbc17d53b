// rope.cuh -- what the kernels that rotate q and k share (rope_append.cu,
// qknorm_rope.cu): the angles, the call's parameters, cache slots and copies of
// 16 bytes.
#pragma once

#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.cuh"

namespace gdn {
namespace {

constexpr int kSms = 152;

// Turns (cycles) of position x inverse frequency, reduced to about [-1/2, 1/2].
__device__ __forceinline__ float reduced_turns(int pos, float inv_freq) {
  // 1 / (2 pi) as the sum of two fp32 numbers
  const float c_hi = 0.15915494309189535f;
  const float c_lo = (float)(0.15915494309189535 - (double)0.15915494309189535f);
  const float f_hi = inv_freq * c_hi;
  const float f_lo = fmaf(inv_freq, c_hi, -f_hi) + inv_freq * c_lo;
  // the position in two parts that fp32 holds exactly
  const float part[2] = {(float)(pos & ~0xffff), (float)(pos & 0xffff)};
  float turns = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float t = part[i] * f_hi;
    turns += (t - rintf(t)) + (fmaf(part[i], f_hi, -t) + part[i] * f_lo);
  }
  return turns - rintf(turns);
}

// FastDiv for slot numbers, which pass 32 bits: 0 <= n < 2^62.
struct FastDiv64 {
  unsigned long long mul;
  uint32_t shift, d;
  FastDiv64() = default;
  explicit FastDiv64(uint32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < d) ++shift;
    mul = (unsigned long long)(((unsigned __int128)((1ull << shift) - d) << 64) / d + 1);
  }
  __device__ __forceinline__ long long div(long long n) const {
    return (long long)((__umul64hi(mul, (unsigned long long)n) + (unsigned long long)n) >> shift);
  }
};

struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  const int32_t *positions;
  const float *inv_freq;
  const int64_t *slots;
  long long q_stride, k_stride, v_stride, page_stride, token_stride, head_stride, n_slots;
  int n_tokens, H, H_kv, rot, n_axes, neighbours, interleaved;
  FastDiv64 page_size;
  int sec[4];
  int *err;
};

__device__ __forceinline__ int axis_of(const RopeParams &p, int i) {
  if (p.interleaved) {
    const int a = i % p.n_axes;
    return a > 0 && i / p.n_axes < p.sec[a] ? a : 0;
  }
  int a = 0;
  for (int left = i; a + 1 < p.n_axes && left >= p.sec[a]; ++a) left -= p.sec[a];
  return a;
}

__device__ __forceinline__ long long slot_offset(const RopeParams &p, long long slot) {
  const long long page = p.page_size.div(slot);
  return page * p.page_stride + (slot - page * p.page_size.d) * p.token_stride;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}

// Shared -> global copy of `bytes` (multiple of 16, aligned addresses), in
// this thread's current bulk group.
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src_smem)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_wait_read_but1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

template <typename T>
struct Vec16 {  // 16 bytes of T as fp32
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T *p) { unpack(*reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void unpack(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

inline RopeParams rope_params(const RopeArgs &a) {
  RopeParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.q_out = a.q_out; p.k_cache = a.k_cache; p.v_cache = a.v_cache;
  p.positions = a.positions; p.inv_freq = a.inv_freq; p.slots = a.slots;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
  p.page_stride = a.cache.page_stride; p.token_stride = a.cache.token_stride;
  p.head_stride = a.cache.head_stride;
  p.n_slots = (long long)a.cache.n_pages * a.cache.page_size;
  p.n_tokens = a.n_tokens; p.H = a.H; p.H_kv = a.cache.H_kv; p.rot = a.rot_dim;
  p.n_axes = a.n_axes; p.page_size = FastDiv64(a.cache.page_size);
  p.neighbours = a.neighbours; p.interleaved = a.interleaved;
  for (int i = 0; i < 4; ++i) p.sec[i] = a.section[i];
  p.err = a.err;
  return p;
}

}  // namespace
}  // namespace gdn
