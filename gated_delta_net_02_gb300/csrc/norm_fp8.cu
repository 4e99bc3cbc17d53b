// norm_fp8.cu -- RMS norm with the residual's addition and an e4m3 output with
// one fp32 scale for every 128 columns of a row.
//
//   h = x + r,  y = h * rsqrt(mean(h^2) + eps) * (w_off + w),
//   s_b = max(max |y| of block b / 448, 2^-100),  q = e4m3(y / s_b)
//
// Bound by HBM: an element is read once (x, r) and written once (h, q), with
// 2 flops each for the sum and a handful for the rounding. So a row's h stays
// in registers between the sum of squares and the output, as fp32 and not
// rounded: y is computed from the same h the sum was.
//  * 8 columns a thread and vector (one 16-byte load of bf16, two of fp32):
//    a block of 128 columns is then exactly the 16 lanes of a half warp, and
//    its maximum four xor-shuffles without shared memory.
//  * Rows of up to 32 vectors take one warp and no barrier; longer rows take
//    one barrier for the warps' partial sums. Sums run in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr float kFp8Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: no zero or subnormal scale

struct NormParams {
  const void *x, *residual, *weight;
  void *residual_out, *out;
  unsigned char *out_fp8;
  float *out_scale;
  int rows, cols, normalize;
  float eps, weight_offset;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0];
  const float4 b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float block_scale(float amax) {
  return fmaxf(amax * (1.f / kFp8Max), kScaleFloor);
}

// The sum of `v` over the `tr` threads of a row (tr a multiple of 32, rows
// are runs of tr threads of the block), in every one of them.
__device__ __forceinline__ float row_sum(float v, int tr, float *red) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (tr == 32) return v;
  const int warp = threadIdx.x >> 5, wr = tr >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / wr * wr;
  v = 0.f;
  for (int w = 0; w < wr; ++w) v += red[first + w];
  return v;
}

// Columns a multiple of 8. Thread t of a row holds the vectors t, t + tr, ...
template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_rows_kernel(const NormParams p, int tr) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[16];
  const int t = threadIdx.x % tr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tr) + threadIdx.x / tr;
  const bool live = row < p.rows;
  const int nvec = p.cols >> 3;
  const long long base = row * p.cols;
  const T *x = static_cast<const T *>(p.x), *r = static_cast<const T *>(p.residual);
  const T *w = static_cast<const T *>(p.weight);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float h[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tr;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    if (live && v < nvec) {
      load8(x + base + v * 8, h[i]);
      if (r) {
        float b[8];
        load8(r + base + v * 8, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += b[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
  }
  float rstd = 1.f;
  if (p.normalize) rstd = rsqrtf(row_sum(sum, tr, red) / (float)p.cols + p.eps);

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tr;
    const bool in = live && v < nvec;
    float y[8];
    if (in && p.residual_out) store8(static_cast<T *>(p.residual_out) + base + v * 8, h[i]);
    if (in && w) {
      float g[8];
      load8(w + v * 8, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rstd * (p.weight_offset + g[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rstd;
    }
    if (in && p.out) store8(static_cast<T *>(p.out) + base + v * 8, y);
    if (!p.out_fp8) continue;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
#pragma unroll
    for (int off = 8; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float scale = block_scale(amax), inv = 1.f / scale;
    if (!in) continue;
    uint32_t q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(y[4 * j] * inv, y[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(y[4 * j + 2] * inv, y[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      q[j] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    *reinterpret_cast<uint2 *>(p.out_fp8 + base + v * 8) = make_uint2(q[0], q[1]);
    if ((v & 15) == 0) p.out_scale[row * ((p.cols + 127) >> 7) + (v >> 4)] = scale;
  }
}

// Any number of columns (those that are no multiple of 8, and rows too long
// for the registers): one block a row, h computed again for the output.
template <typename T>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[16];
  const long long row = blockIdx.x, base = row * p.cols;
  const T *x = static_cast<const T *>(p.x), *r = static_cast<const T *>(p.residual);
  const T *w = static_cast<const T *>(p.weight);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float rstd = 1.f;
  if (p.normalize) {
    float sum = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 256) {
      const float h = to_f32(x[base + c]) + (r ? to_f32(r[base + c]) : 0.f);
      sum = fmaf(h, h, sum);
    }
    rstd = rsqrtf(row_sum(sum, 256, red) / (float)p.cols + p.eps);
  }
  // every thread has read the row's sum before anything is written in place:
  // row_sum's barrier stands between them
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nblk = (p.cols + 127) >> 7;
  for (int b = warp; b < nblk; b += 8) {
    float y[4];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = b * 128 + j * 32 + lane;
      y[j] = 0.f;
      if (c >= p.cols) continue;
      const float h = to_f32(x[base + c]) + (r ? to_f32(r[base + c]) : 0.f);
      y[j] = h * rstd * (w ? p.weight_offset + to_f32(w[c]) : 1.f);
      if (p.residual_out) static_cast<T *>(p.residual_out)[base + c] = from_f32<T>(h);
      if (p.out) static_cast<T *>(p.out)[base + c] = from_f32<T>(y[j]);
      amax = fmaxf(amax, fabsf(y[j]));
    }
    if (!p.out_fp8) continue;
#pragma unroll
    for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float scale = block_scale(amax), inv = 1.f / scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = b * 128 + j * 32 + lane;
      if (c < p.cols)
        p.out_fp8[base + c] = __nv_cvt_float_to_fp8(y[j] * inv, __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) p.out_scale[row * nblk + b] = scale;
  }
}

template <typename T>
cudaError_t launch_t(const NormParams &p, cudaStream_t stream) {
  const int nvec = p.cols >> 3;
  if ((p.cols & 7) || nvec > 512 * 8)
    return launch_pdl(norm_any_kernel<T>, dim3(p.rows), dim3(256), 0, stream, p);
  int nv = 1;
  while (nvec > 512 * nv) nv *= 2;
  const int tr = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  const int rpc = tr >= 256 ? 1 : 256 / tr;
  const dim3 grid((p.rows + rpc - 1) / rpc), block(tr * rpc);
  switch (nv) {
    case 1: return launch_pdl(norm_rows_kernel<T, 1>, grid, block, 0, stream, p, tr);
    case 2: return launch_pdl(norm_rows_kernel<T, 2>, grid, block, 0, stream, p, tr);
    case 4: return launch_pdl(norm_rows_kernel<T, 4>, grid, block, 0, stream, p, tr);
    default: return launch_pdl(norm_rows_kernel<T, 8>, grid, block, 0, stream, p, tr);
  }
}

}  // namespace

cudaError_t launch_norm_fp8(const NormArgs &a, cudaStream_t stream) {
  const NormParams p = {a.x, a.residual, a.weight, a.residual_out, a.out, a.out_fp8, a.out_scale,
                        a.rows, a.cols, a.normalize, a.eps, a.weight_offset};
  return a.bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace gdn
