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
//  * 8 (few rows) or 16 columns of a thread: a scale's 128 columns are then
//    16 or 8 neighbouring lanes, and their maximum a few xor-shuffles.
//  * Few rows: a row for each block or part of one, loaded straight into
//    registers. Many rows: persistent blocks fed by a ring of bulk copies.
//    Sums run in a fixed order in both.
// Measured on one GB300: 64 x 2048 bf16 with residual 1.9 us; 34739 x 4096
// 178 us (5.6 TB/s of its own bytes, of 6.8 copied).
// What is left there: 57 rows a block and their first loads after the
// previous kernel, and some 360 instructions a warp and row (half of the
// issue slots).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "layer.cuh"

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
  float eps, weight_offset, inv_cols;
  int *err;
};

constexpr int kSms = 152;
constexpr int kMaxStages = 4;
constexpr int kRingSmem = 216 * 1024;  // of an SM, for all its blocks

constexpr int kRingThreads = 256;
// blocks of an SM, which its registers and shared memory are shared out to
constexpr int ring_blocks(int nv) { return nv == 1 ? 4 : nv == 2 ? 2 : 1; }
// and the most that a block's ring may take of the latter
constexpr int ring_bytes(int nv) { return kRingSmem / ring_blocks(nv) - 1024; }

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

// The quotient's last step of Markstein (1990): q is a / b to within some units;
// its remainder a - q b is exact in one fused multiply-add, and q + remainder / b
// is the quotient rounded once, as an fp32 division rounds it.
__device__ __forceinline__ float block_scale(float amax) {
  const float inv = 1.f / kFp8Max, q = amax * inv;
  const float scale = fmaf(fmaf(-kFp8Max, q, amax), inv, q);
  return fmaxf(amax == INFINITY ? amax : scale, kScaleFloor);
}

// Two fp32 operations in one instruction; each half rounds as the scalar
// instruction does. The kernel is close to issue-bound without them.
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// x += a * b
__device__ __forceinline__ void fma2(float &x, float &y, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mov.b64 w, {%4, %5};\n\tfma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// s += a * a
__device__ __forceinline__ void square2(float &s, float &t, float a, float b) {
  fma2(s, t, a, b, a, b);
}
template <int N>
__device__ __forceinline__ void scale_by(float (&y)[N], float f) {
#pragma unroll
  for (int j = 0; j < N; j += 2) mul2(y[j], y[j + 1], f, f);
}

// y / scale, rounded once (as block_scale): a value half way between two e4m3
// numbers has to go to the even one, and a product with the reciprocal, which
// has roundings of its own, sends it either way. The two instructions more for
// every one or two columns take 34739 x 4096 from 174 to 178 us and 34314 x 2027
// (no residual, both outputs) from 121 to 128. An infinite scale has no
// remainder: finite y over it are 0, infinite ones NaN.
struct DivideBy {
  float inv, neg;
  __device__ __forceinline__ explicit DivideBy(float scale) {
    // to within a unit; the scale's floor keeps it finite
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    neg = scale == INFINITY ? 0.f : -scale;
  }
  __device__ __forceinline__ float operator()(float y) const {
    const float q = y * inv;
    return fmaf(fmaf(neg, q, y), inv, q);
  }
  template <int N>
  __device__ __forceinline__ void all(float (&y)[N]) const {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float q = y[j], t = y[j + 1], a = y[j], b = y[j + 1];
      mul2(q, t, inv, inv);
      fma2(a, b, q, t, neg, neg);
      fma2(q, t, a, b, inv, inv);
      y[j] = q;
      y[j + 1] = t;
    }
  }
};

// The sum of wr <= 16 numbers, in every lane, in one fixed order.
__device__ __forceinline__ float warps_sum(const float *red, int wr) {
  const int lane = threadIdx.x & 15;
  float v = lane < wr ? red[lane] : 0.f;
#pragma unroll
  for (int off = 8; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
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
  return warps_sum(red + warp / wr * wr, wr);
}

// One vector of 8 columns to its outputs: h, y, e4m3 and the block's scale.
// Called by whole warps; `in` says whether the thread's vector exists.
template <typename T>
__device__ __forceinline__ void put8(const NormParams &p, long long row, int v, bool in,
                                     const float (&h)[8], const float (&g)[8], float rstd) {
  const long long at = row * p.cols + v * 8;
  float y[8];
  if (in && p.residual_out) store8(static_cast<T *>(p.residual_out) + at, h);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = h[j];
  scale_by(y, rstd);
#pragma unroll
  for (int j = 0; j < 8; j += 2) mul2(y[j], y[j + 1], g[j], g[j + 1]);
  if (in && p.out) store8(static_cast<T *>(p.out) + at, y);
  if (!p.out_fp8) return;
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
#pragma unroll
  for (int off = 8; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const float scale = block_scale(amax);
  if (!in) return;
  DivideBy(scale).all(y);
  uint32_t q[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j], y[4 * j + 1]),
                                                             __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(y[4 * j + 2], y[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
    q[j] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  *reinterpret_cast<uint2 *>(p.out_fp8 + at) = make_uint2(q[0], q[1]);
  if ((v & 15) == 0) p.out_scale[row * ((p.cols + 127) >> 7) + (v >> 4)] = scale;
}

// The factors w_off + w of a vector's columns (1 without weights).
template <typename T>
__device__ __forceinline__ void weight8(const NormParams &p, int v, bool in, float (&g)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = 1.f;
  if (!in || !p.weight) return;
  load8(static_cast<const T *>(p.weight) + v * 8, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] += p.weight_offset;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float h[NV][8];
  float sum = 0.f, sum2 = 0.f;
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
        for (int j = 0; j < 8; j += 2) add2(h[i][j], h[i][j + 1], b[j], b[j + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) square2(sum, sum2, h[i][j], h[i][j + 1]);
  }
  float rstd = 1.f;
  if (p.normalize) rstd = rsqrtf(row_sum(sum + sum2, tr, red) * p.inv_cols + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tr;
    const bool in = live && v < nvec;
    float g[8];
    weight8<T>(p, v, in, g);
    put8<T>(p, row, v, in, h[i], g, rstd);
  }
}

// 16 columns of a thread in the ring kernel: loads, and stores of whole
// 32-byte sectors (`wide`: the rows start on 32 bytes).
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16]) {
  float a[8], b[8];
  load8(p, a);
  load8(p + 8, b);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = a[j];
    v[8 + j] = b[j];
  }
}
__device__ __forceinline__ void store32(void *p, const uint32_t *w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  store32(p, w, wide);
}
__device__ __forceinline__ void store16(float *p, const float (&v)[16], bool wide) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
  store32(p, w, wide);
  store32(p + 8, w + 8, wide);
}

// Many rows, columns a multiple of 16: persistent blocks, whose rows arrive
// in shared memory by bulk copies, `stages` groups of rows ahead (registers
// could not hold that many bytes under way). One barrier a group: it carries
// the rows' sums and says that the group has been read, so that its place can
// be loaded again. A thread has 16 columns at a time, which halves what 8
// cost in shuffles and addresses: with 8 the kernel was bound by instructions.
template <typename T, int NV>
__global__ void __launch_bounds__(kRingThreads, ring_blocks(NV))
    norm_ring_kernel(const NormParams p, int tr, int stages, uint32_t half, bool wide) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float red[2][16];
  const int rpc = blockDim.x / tr, t = threadIdx.x % tr, sub = threadIdx.x / tr;
  const int warp = threadIdx.x >> 5, wr = tr >> 5, nvec = p.cols >> 4, nblk = (p.cols + 127) >> 7;
  const int groups = (p.rows - 1) / rpc + 1;
  const T *x = static_cast<const T *>(p.x), *r = static_cast<const T *>(p.residual);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // a stage: the group's rows of x, then (at `half`) of the residual
  const uint32_t stage = r ? 2 * half : half;
  auto load = [&](int g, int s) {
    if (g >= groups) return;
    const long long row0 = (long long)g * rpc;
    const uint32_t bytes =
        (uint32_t)min((long long)rpc, p.rows - row0) * p.cols * (uint32_t)sizeof(T);
    unsigned char *st = smem + s * stage;
    mbar_arrive_expect_tx(&full[s], r ? 2 * bytes : bytes);
    bulk_g2s(st, x + row0 * p.cols, bytes, &full[s]);
    if (r) bulk_g2s(st + half, r + row0 * p.cols, bytes, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) load(blockIdx.x + s * gridDim.x, s);
  float w[NV][16];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tr;
#pragma unroll
    for (int j = 0; j < 16; ++j) w[i][j] = 1.f;
    if (p.weight && v < nvec) {
      load16(static_cast<const T *>(p.weight) + v * 16, w[i]);
#pragma unroll
      for (int j = 0; j < 16; ++j) w[i][j] += p.weight_offset;
    }
  }

  int s = 0, phase = 0, it = 0;
  for (int g = blockIdx.x; g < groups; g += gridDim.x, ++it) {
    const long long row = (long long)g * rpc + sub;
    const bool live = row < p.rows;
    const bool ok = mbar_wait(&full[s], phase, p.err, kSiteNormRow);
    const T *xs = reinterpret_cast<const T *>(smem + s * stage) + sub * p.cols;
    const T *rs = reinterpret_cast<const T *>(reinterpret_cast<const unsigned char *>(xs) + half);
    float h[NV][16];
    float sum = 0.f, sum2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tr;
#pragma unroll
      for (int j = 0; j < 16; ++j) h[i][j] = 0.f;
      if (live && v < nvec) {
        load16(xs + v * 16, h[i]);
        if (r) {
          float b[16];
          load16(rs + v * 16, b);
#pragma unroll
          for (int j = 0; j < 16; j += 2) add2(h[i][j], h[i][j + 1], b[j], b[j + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; j += 2) square2(sum, sum2, h[i][j], h[i][j + 1]);
    }
    sum += sum2;
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if ((threadIdx.x & 31) == 0) red[it & 1][warp] = sum;
    if (__syncthreads_or(!ok)) {
      if (threadIdx.x == 0)  // the stages loaded ahead
        for (int i = 0; i < stages && g < groups; ++i, g += gridDim.x) {
          mbar_drain(&full[s], phase);
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      break;
    }
    if (threadIdx.x == 0) load(g + stages * gridDim.x, s);
    float rstd = 1.f;
    if (p.normalize)
      rstd = rsqrtf(warps_sum(&red[it & 1][warp / wr * wr], wr) * p.inv_cols + p.eps);
    const long long at0 = row * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tr;
      const bool in = live && v < nvec;
      const long long at = at0 + v * 16;
      if (in && p.residual_out) store16(static_cast<T *>(p.residual_out) + at, h[i], wide);
      scale_by(h[i], rstd);
#pragma unroll
      for (int j = 0; j < 16; j += 2) mul2(h[i][j], h[i][j + 1], w[i][j], w[i][j + 1]);
      if (in && p.out) store16(static_cast<T *>(p.out) + at, h[i], wide);
      if (!p.out_fp8) continue;
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(h[i][j]));
#pragma unroll
      for (int off = 4; off; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      const float scale = block_scale(amax);
      DivideBy(scale).all(h[i]);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(h[i][4 * j], h[i][4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(h[i][4 * j + 2], h[i][4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
        q[j] = (uint32_t)lo | ((uint32_t)hi << 16);
      }
      if (in) *reinterpret_cast<uint4 *>(p.out_fp8 + at) = make_uint4(q[0], q[1], q[2], q[3]);
      if (in && (v & 7) == 0) p.out_scale[row * nblk + (v >> 3)] = scale;
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
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
    rstd = rsqrtf(row_sum(sum, 256, red) * p.inv_cols + p.eps);
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
    const float scale = block_scale(amax);
    const DivideBy quotient(scale);
    // value by value between the stores (all four before them: 147 us for 128)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = b * 128 + j * 32 + lane;
      if (c < p.cols)
        p.out_fp8[base + c] = __nv_cvt_float_to_fp8(quotient(y[j]), __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) p.out_scale[row * nblk + b] = scale;
  }
}

template <typename T>
cudaError_t launch_t(const NormParams &p, cudaStream_t stream) {
  const int nvec = p.cols >> 3;
  if ((p.cols & 7) || nvec > 512 * 8)
    return launch_pdl(norm_any_kernel<T>, dim3(p.rows), dim3(256), 0, stream, p);
  struct Split {  // vectors of a thread, threads of a row, rows of a block
    int nv, tr, rpc;
    Split(int nvec, int most_threads, int block) {
      nv = 1;
      while (nvec > most_threads * nv) nv *= 2;
      tr = ((nvec + nv - 1) / nv + 31) / 32 * 32;
      rpc = tr >= block ? 1 : block / tr;
    }
  };
  if (p.cols % 16 == 0) {
    const Split d(p.cols / 16, kRingThreads, kRingThreads);
    const int groups = (p.rows - 1) / d.rpc + 1;
    const uint32_t half = (uint32_t)d.rpc * p.cols * (uint32_t)sizeof(T);
    const uint32_t stage = half * (p.residual ? 2 : 1);
    const int grid = kSms * ring_blocks(d.nv);
    int stages = (int)(ring_bytes(d.nv) / stage);
    if (stages > kMaxStages) stages = kMaxStages;
    // below two rows a block the ring has nothing to run ahead for
    if (stages >= 2 && d.nv <= 4 && groups >= 2 * grid) {
      auto kernel = d.nv == 1   ? norm_ring_kernel<T, 1>
                    : d.nv == 2 ? norm_ring_kernel<T, 2>
                                : norm_ring_kernel<T, 4>;
      const size_t smem = (size_t)stages * stage;
      // The attribute is the process's: always the most that any call needs,
      // or another thread's call could lower it between here and the launch.
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           ring_bytes(d.nv));
      if (e != cudaSuccess) return e;
      const bool wide = ((reinterpret_cast<uintptr_t>(p.residual_out) |
                          reinterpret_cast<uintptr_t>(p.out)) & 31) == 0;
      return launch_pdl(kernel, dim3(grid), dim3(d.tr * d.rpc), smem, stream, p, d.tr, stages,
                        half, wide);
    }
  }
  const Split d(nvec, 512, 256);
  const int nv = d.nv, tr = d.tr, groups = (p.rows - 1) / d.rpc + 1;
  const dim3 block(d.tr * d.rpc);
  switch (nv) {
    case 1: return launch_pdl(norm_rows_kernel<T, 1>, dim3(groups), block, 0, stream, p, tr);
    case 2: return launch_pdl(norm_rows_kernel<T, 2>, dim3(groups), block, 0, stream, p, tr);
    case 4: return launch_pdl(norm_rows_kernel<T, 4>, dim3(groups), block, 0, stream, p, tr);
    default: return launch_pdl(norm_rows_kernel<T, 8>, dim3(groups), block, 0, stream, p, tr);
  }
}

}  // namespace

cudaError_t launch_norm_fp8(const NormArgs &a, cudaStream_t stream) {
  const NormParams p = {a.x, a.residual, a.weight, a.residual_out, a.out, a.out_fp8, a.out_scale,
                        a.rows, a.cols, a.normalize, a.eps, a.weight_offset, 1.f / (float)a.cols, a.err};
  return a.bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace gdn
