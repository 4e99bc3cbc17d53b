// qknorm_rope.cu -- RMS norm of every q and k head, rotary positions on the
// result, and the append of k and of v to a paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * (offset + weight)     over a head
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos)
//
// Bound by HBM: each element is read once and written once. The sum of a
// head's squares, the norm and the rotation are in fp32, with one rounding at
// the end.
#include "rope.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

struct NormParams {
  const void *qw, *kw;
  float eps, offset;
};

// One block a token, one warp a head; partners of a pair are read again.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qknorm_kernel(const RopeParams p, const NormParams n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float cs[D / 2], sn[D / 2];
  __shared__ long long at_s;  // element offset of the slot, -1 = none
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = p.rot >> 1;
  const long long tok = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = tid; i < half; i += kThreads) {
    const int pos = p.positions[(long long)axis_of(p, i) * p.n_tokens + tok];
    sincospif(2.f * reduced_turns(pos, p.inv_freq[i]), &sn[i], &cs[i]);
  }
  if (tid == 0) {
    const long long slot = p.slots[tok];
    at_s = -1;
    if (slot >= p.n_slots) set_error(p.err, kDevBadSlot);
    else if (slot >= 0) at_s = slot_offset(p, slot);
  }
  __syncthreads();
  const long long at = at_s;
  for (int r = warp; r < p.H + 2 * p.H_kv; r += kThreads / 32) {
    const bool is_q = r < p.H, is_v = r >= p.H + p.H_kv;
    const int h = is_q ? r : is_v ? r - p.H - p.H_kv : r - p.H;
    if (!is_q && at < 0) continue;
    const T *src;
    T *dst;
    if (is_q) {
      src = static_cast<const T *>(p.q) + tok * p.q_stride + (long long)h * D;
      dst = static_cast<T *>(p.q_out) + (tok * p.H + h) * D;
    } else {
      src = is_v ? static_cast<const T *>(p.v) + tok * p.v_stride + (long long)h * D
                 : static_cast<const T *>(p.k) + tok * p.k_stride + (long long)h * D;
      dst = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + at + h * p.head_stride;
    }
    if (is_v) {
      for (int d = lane; d < D; d += 32) dst[d] = src[d];
      continue;
    }
    float sum = 0.f;
    for (int d = lane; d < D; d += 32) {
      const float x = to_f32(src[d]);
      sum = fmaf(x, x, sum);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float inv = 1.f / sqrtf(sum / D + n.eps);
    const T *w = static_cast<const T *>(is_q ? n.qw : n.kw);
    auto normed = [&](int d) {
      const float y = to_f32(src[d]) * inv;
      return w ? y * (n.offset + to_f32(w[d])) : y;
    };
    for (int d = lane; d < D; d += 32) {
      float y = normed(d);
      if (d < p.rot) {
        const bool first = p.neighbours ? !(d & 1) : d < half;
        const int f = p.neighbours ? d >> 1 : first ? d : d - half;
        const float z = normed(p.neighbours ? d ^ 1 : first ? d + half : f);
        y = first ? y * cs[f] - z * sn[f] : z * sn[f] + y * cs[f];
      }
      dst[d] = from_f32<T>(y);
    }
  }
}

template <typename T>
cudaError_t launch_t(const RopeParams &p, const NormParams &n, int D, cudaStream_t stream) {
  const dim3 grid(p.n_tokens), block(kThreads);
  if (D == 64) return launch_pdl(qknorm_kernel<T, 64>, grid, block, 0, stream, p, n);
  if (D == 128) return launch_pdl(qknorm_kernel<T, 128>, grid, block, 0, stream, p, n);
  return launch_pdl(qknorm_kernel<T, 256>, grid, block, 0, stream, p, n);
}

}  // namespace

cudaError_t launch_qknorm_rope(const QkNormArgs &a, cudaStream_t stream) {
  const RopeParams p = rope_params(a.rope);
  const NormParams n{a.q_weight, a.k_weight, a.eps, a.weight_offset};
  return a.rope.cache.bf16 ? launch_t<__nv_bfloat16>(p, n, a.rope.cache.D, stream)
                           : launch_t<float>(p, n, a.rope.cache.D, stream);
}

}  // namespace gdn
