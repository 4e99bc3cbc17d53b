// rope_append.cu -- rotary positions with several axes on q and k, and the
// append of the rotated k and of v to a paged cache, in one pass.
//
//   angle_i = positions[axis(i)][t] * inv_freq[i],
//   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Bound by HBM: each element is read once and written once. The angles are
// the only arithmetic worth counting, and they are the same for every head:
// a block takes whole tokens, computes each token's sines and cosines once
// into shared memory and reuses them for all its q and k heads.
//
// Precision: position * inv_freq in fp32 loses the angle itself once it
// passes some thousand radians (2^-24 of it). The product is formed in turns,
// as the fp32 product plus its exact error (fused multiply-add), so that the
// whole turns drop out exactly and what is left of the angle has an error of
// about 2^-24 turns at any position.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a block

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

struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  const int32_t *positions;
  const float *inv_freq;
  const int64_t *slots;
  long long q_stride, k_stride, v_stride, page_stride, token_stride, head_stride, n_slots;
  int n_tokens, H, H_kv, rot, n_axes, page_size, tpb, neighbours, interleaved;
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

template <typename T>
struct Vec16 {  // 16 bytes of T as fp32
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T *p) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
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

// A block takes p.tpb tokens; a thread one 16-byte vector of a head at a time.
// WHOLE: a vector's elements are all rotated with elements of one other
// vector (or of itself), or all pass; otherwise partners are read one by one.
template <typename T, int D, bool WHOLE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VE = 16 / (int)sizeof(T), NVEC = D / VE;
  __shared__ float cos_s[kMaxTokens][D / 2], sin_s[kMaxTokens][D / 2];
  __shared__ long long at_s[kMaxTokens];  // element offset of the slot, -1 = none
  const int tid = threadIdx.x, half = p.rot >> 1;
  const int t0 = blockIdx.x * p.tpb, nt = min(p.tpb, p.n_tokens - t0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int e = tid; e < nt * half; e += kThreads) {
    const int j = e / half, i = e - j * half;
    const int pos = p.positions[(long long)axis_of(p, i) * p.n_tokens + t0 + j];
    sincospif(2.f * reduced_turns(pos, p.inv_freq[i]), &sin_s[j][i], &cos_s[j][i]);
  }
  if (tid < nt) {
    const long long slot = p.slots[t0 + tid];
    long long at = -1;
    if (slot >= p.n_slots) set_error(p.err, kDevBadSlot);
    else if (slot >= 0)
      at = slot / p.page_size * p.page_stride + slot % p.page_size * p.token_stride;
    at_s[tid] = at;
  }
  __syncthreads();
  const int heads = p.H + 2 * p.H_kv;
  for (int e = tid; e < nt * heads * NVEC; e += kThreads) {
    const int row = e / NVEC, d0 = (e % NVEC) * VE;
    const int j = row / heads;
    int h = row - j * heads;
    const long long tok = t0 + j;
    const T *src;
    T *dst;
    bool turn = d0 < p.rot;
    if (h < p.H) {
      src = static_cast<const T *>(p.q) + tok * p.q_stride + (long long)h * D;
      dst = static_cast<T *>(p.q_out) + (tok * p.H + h) * D;
    } else {
      h -= p.H;
      const long long at = at_s[j];
      if (at < 0) continue;
      if (h < p.H_kv) {
        src = static_cast<const T *>(p.k) + tok * p.k_stride + (long long)h * D;
        dst = static_cast<T *>(p.k_cache) + at + h * p.head_stride;
      } else {
        h -= p.H_kv;
        src = static_cast<const T *>(p.v) + tok * p.v_stride + (long long)h * D;
        dst = static_cast<T *>(p.v_cache) + at + h * p.head_stride;
        turn = false;
      }
    }
    Vec16<T> x;
    x.load(src + d0);
    if (turn) {
      const float *cs = cos_s[j], *sn = sin_s[j];
      if (p.neighbours) {
        // rot is even, so a pair is never cut
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          const int f = (d0 + i) >> 1;
          if (!WHOLE && d0 + i >= p.rot) break;
          const float c = cs[f], s = sn[f], a = x.v[i], b = x.v[i + 1];
          x.v[i] = a * c - b * s;
          x.v[i + 1] = a * s + b * c;
        }
      } else if constexpr (WHOLE) {
        const bool first = d0 < half;
        const int f = first ? d0 : d0 - half;
        Vec16<T> y;
        y.load(src + (first ? d0 + half : f));
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float s = sn[f + i];
          x.v[i] = x.v[i] * cs[f + i] + y.v[i] * (first ? -s : s);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const int d = d0 + i;
          if (d >= p.rot) break;
          const bool first = d < half;
          const int f = first ? d : d - half;
          const float y = to_f32(src[first ? d + half : f]), s = sn[f];
          x.v[i] = x.v[i] * cs[f] + y * (first ? -s : s);
        }
      }
    }
    x.store(dst + d0);
  }
}

template <typename T, int D>
cudaError_t launch_d(RopeParams p, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const bool whole = p.neighbours ? p.rot % VE == 0 : (p.rot / 2) % VE == 0;
  p.tpb = 1;
  const dim3 grid((p.n_tokens + p.tpb - 1) / p.tpb), block(kThreads);
  return whole ? launch_pdl(rope_kernel<T, D, true>, grid, block, 0, stream, p)
               : launch_pdl(rope_kernel<T, D, false>, grid, block, 0, stream, p);
}

template <typename T>
cudaError_t launch_t(const RopeParams &p, int D, cudaStream_t stream) {
  if (D == 64) return launch_d<T, 64>(p, stream);
  if (D == 128) return launch_d<T, 128>(p, stream);
  return launch_d<T, 256>(p, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t stream) {
  RopeParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.q_out = a.q_out; p.k_cache = a.k_cache; p.v_cache = a.v_cache;
  p.positions = a.positions; p.inv_freq = a.inv_freq; p.slots = a.slots;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
  p.page_stride = a.cache.page_stride; p.token_stride = a.cache.token_stride;
  p.head_stride = a.cache.head_stride;
  p.n_slots = (long long)a.cache.n_pages * a.cache.page_size;
  p.n_tokens = a.n_tokens; p.H = a.H; p.H_kv = a.cache.H_kv; p.rot = a.rot_dim;
  p.n_axes = a.n_axes; p.page_size = a.cache.page_size;
  p.neighbours = a.neighbours; p.interleaved = a.interleaved;
  for (int i = 0; i < 4; ++i) p.sec[i] = a.section[i];
  p.err = a.err;
  return a.cache.bf16 ? launch_t<__nv_bfloat16>(p, a.cache.D, stream)
                      : launch_t<float>(p, a.cache.D, stream);
}

}  // namespace gdn
