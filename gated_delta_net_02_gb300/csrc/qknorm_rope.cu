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

// Rows too long for the ring of qknorm_rows_kernel: one block a token, one warp a
// head; partners of a pair are read again.
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

// Persistent blocks; a token's rows pass through shared memory by bulk copies
// both ways, a ring of kStages groups of tpb tokens, as in rope_append.cu. A
// head's row is the work of D / (2 x 16 bytes) lanes, each with two vectors of 16
// bytes that lie half a rotation apart (so that partners meet in one lane), in
// registers from the sum of squares to the rotation.
constexpr int kStages = 3;
constexpr int kRowBlocks = 4;
constexpr int kStageBytes = 16 * 1024;
constexpr int kMostTokens = 8;
constexpr int kRowsSmem = 220 * 1024;

// How a rotation meets the vectors of a head: whole vectors of two halves, of
// neighbouring pairs, or pairs of two halves that cut a vector.
enum Meet { kHalves, kNeighbours, kCut };

template <typename T, int D, Meet MEET>
__global__ void __launch_bounds__(kThreads, kRowBlocks)
    qknorm_rows_kernel(const RopeParams p, const NormParams n, uint32_t q_bytes, uint32_t kv_bytes,
                       int tpb, FastDiv by_heads) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VE = 16 / (int)sizeof(T), LPR = D / VE / 2;  // lanes of a head's row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kStages];
  const int tid = threadIdx.x, half = p.rot >> 1;
  const uint32_t row = q_bytes + 2 * kv_bytes, stage = tpb * row;
  // sines and cosines of two groups of tokens, [tpb][half] each
  float *trig = reinterpret_cast<float *>(smem + kStages * stage);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int groups = (p.n_tokens + tpb - 1) / tpb, heads = p.H + p.H_kv;
  auto group_of = [&](int it) { return (long long)blockIdx.x + (long long)it * gridDim.x; };
  auto tokens_of = [&](long long g) {
    return g < groups ? min(tpb, p.n_tokens - (int)g * tpb) : 0;
  };
  // a lane of warp 0 for each token of a group
  auto load = [&](int it) {
    const long long g = group_of(it);
    const int nt = tokens_of(g), s = it % kStages;
    if (nt == 0) return;
    if (tid == 0) mbar_arrive_expect_tx(&full[s], nt * row);
    __syncwarp();
    if (tid < nt) {
      const long long tok = g * tpb + tid;
      unsigned char *st = smem + s * stage + tid * row;
      bulk_g2s(st, static_cast<const T *>(p.q) + tok * p.q_stride, q_bytes, &full[s]);
      bulk_g2s(st + q_bytes, static_cast<const T *>(p.k) + tok * p.k_stride, kv_bytes, &full[s]);
      bulk_g2s(st + q_bytes + kv_bytes, static_cast<const T *>(p.v) + tok * p.v_stride, kv_bytes,
               &full[s]);
    }
  };
  auto slot_of = [&](int it) -> long long {
    const long long g = group_of(it);
    return tid < tokens_of(g) ? p.slots[g * tpb + tid] : -1;
  };
  long long slot = -1;
  if (tid < 32) {
    for (int it = 0; it < kStages - 1; ++it) load(it);
    slot = slot_of(0);
  }
  // the lane's two vectors of a head, from these elements on
  const int l = tid % LPR;
  int at_a = 2 * l * VE, at_b = at_a + VE;
  if (MEET == kHalves) {
    const int turning = half / VE;
    at_a = l < turning ? l * VE : p.rot + 2 * (l - turning) * VE;
    at_b = l < turning ? at_a + half : at_a + VE;
  }
  // their weights, as they are stored
  uint4 wq[2], wk[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = i ? at_b : at_a;
    if (n.qw) wq[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(n.qw) + at);
    if (n.kw) wk[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(n.kw) + at);
  }
  // A thread has one pair of one token of each group (tpb * half threads do):
  // its axis and frequency stay, its position is read a group ahead.
  const int my_j = half > 0 ? tid / half : tpb, my_i = tid - my_j * half;
  const int32_t *my_pos = nullptr;
  float freq = 0.f;
  if (my_j < tpb) {
    my_pos = p.positions + (long long)axis_of(p, my_i) * p.n_tokens + my_j;
    freq = p.inv_freq[my_i];
  }
  auto position = [&](int it) -> int {
    const long long g = group_of(it);
    return my_j < tokens_of(g) ? my_pos[g * tpb] : 0;
  };
  int pos = position(0);
  auto angles = [&](int it) {
    float *cs = trig + (it & 1) * 2 * tpb * half, *sn = cs + tpb * half;
    const int next = position(it + 1);
    if (my_j < tpb) sincospif(2.f * reduced_turns(pos, freq), &sn[tid], &cs[tid]);
    pos = next;
  };
  int it = 0;
  for (long long g = blockIdx.x; g < groups; g += gridDim.x, ++it) {
    const int s = it % kStages, nt = tokens_of(g);
    const long long next_slot = slot_of(it + 1);
    angles(it);
    const bool ok = mbar_wait(&full[s], (it / kStages) & 1, p.err, kSiteRopeRow);
    if (__syncthreads_or(!ok)) {
      if (tid == 0)  // the stages loaded ahead
        for (int i = it; i < it + kStages - 1 && group_of(i) < groups; ++i)
          mbar_drain(&full[i % kStages], (i / kStages) & 1);
      break;
    }
    const float *cs0 = trig + (it & 1) * 2 * tpb * half, *sn0 = cs0 + tpb * half;
    unsigned char *st = smem + s * stage;
    const int rows = nt * heads;
    // a warp's lanes stay together: the sums pass between them
    for (int r0 = (tid & ~31) / LPR; r0 < rows; r0 += kThreads / LPR) {
      const int r = r0 + (tid & 31) / LPR;
      const bool live = r < rows;
      const int j = by_heads.div(live ? r : 0), h = (live ? r : 0) - j * heads;
      T *head = reinterpret_cast<T *>(st + j * row) + h * D;
      Vec16<T> a, b;
      a.load(head + at_a);
      b.load(head + at_b);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VE; ++i) sum = fmaf(a.v[i], a.v[i], fmaf(b.v[i], b.v[i], sum));
#pragma unroll
      for (int off = LPR / 2; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const float inv = 1.f / sqrtf(sum * (1.f / D) + n.eps);
      const bool is_q = h < p.H;
      if (is_q ? n.qw != nullptr : n.kw != nullptr) {
        Vec16<T> w;
        const float base = n.offset * inv;
        w.unpack(is_q ? wq[0] : wk[0]);
#pragma unroll
        for (int i = 0; i < VE; ++i) a.v[i] *= fmaf(w.v[i], inv, base);
        w.unpack(is_q ? wq[1] : wk[1]);
#pragma unroll
        for (int i = 0; i < VE; ++i) b.v[i] *= fmaf(w.v[i], inv, base);
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          a.v[i] *= inv;
          b.v[i] *= inv;
        }
      }
      const float *cs = cs0 + j * half, *sn = sn0 + j * half;
      if constexpr (MEET == kHalves) {
        if (at_a < half) {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const float c = cs[at_a + i], t = sn[at_a + i], x = a.v[i] * c - b.v[i] * t;
            b.v[i] = a.v[i] * t + b.v[i] * c;
            a.v[i] = x;
          }
        }
      } else if constexpr (MEET == kNeighbours) {
        auto turn = [&](Vec16<T> &x, int at) {
#pragma unroll
          for (int i = 0; i < VE; i += 2) {
            if (at + i >= p.rot) break;
            const float c = cs[(at + i) >> 1], t = sn[(at + i) >> 1];
            const float y = x.v[i] * c - x.v[i + 1] * t;
            x.v[i + 1] = x.v[i] * t + x.v[i + 1] * c;
            x.v[i] = y;
          }
        };
        turn(a, at_a);
        turn(b, at_b);
      }
      if constexpr (MEET != kCut) {
        if (live) {
          a.store(head + at_a);
          b.store(head + at_b);
        }
      } else {
        // the partners lie in other lanes' vectors: read again, once the row's
        // sum is known, and normed one by one
        auto normed = [&](int d) {
          const T *w = static_cast<const T *>(is_q ? n.qw : n.kw);
          const float y = to_f32(head[d]) * inv;
          return w ? y * (n.offset + to_f32(w[d])) : y;
        };
        __syncwarp();
        if (live) {
          for (int i = l; i < half; i += LPR) {
            const float x = normed(i), y = normed(i + half), c = cs[i], t = sn[i];
            head[i] = from_f32<T>(x * c - y * t);
            head[i + half] = from_f32<T>(x * t + y * c);
          }
          for (int d = p.rot + l; d < D; d += LPR) head[d] = from_f32<T>(normed(d));
        }
      }
    }
    fence_proxy_async();
    __syncthreads();
    if (tid < 32) {
      if (tid < nt) {
        const long long tok = g * tpb + tid;
        const unsigned char *src = st + tid * row;
        bulk_s2g(static_cast<T *>(p.q_out) + tok * p.H * D, src, q_bytes);
        if (slot >= p.n_slots) {
          set_error(p.err, kDevBadSlot);
        } else if (slot >= 0) {
          const long long at = slot_offset(p, slot);
          T *kd = static_cast<T *>(p.k_cache) + at, *vd = static_cast<T *>(p.v_cache) + at;
          // a slot's heads are one run of the cache unless its layout parts them
          const int runs = p.head_stride == D ? 1 : p.H_kv;
          const uint32_t bytes = kv_bytes / runs;
          for (int r = 0; r < runs; ++r) {
            bulk_s2g(kd + r * p.head_stride, src + q_bytes + r * bytes, bytes);
            bulk_s2g(vd + r * p.head_stride, src + q_bytes + kv_bytes + r * bytes, bytes);
          }
        }
      }
      bulk_commit();
      slot = next_slot;
      // the stage loaded next was stored from an iteration ago: all but the
      // stores just issued have read theirs
      bulk_wait_read_but1();
      __syncwarp();
      load(it + kStages - 1);
    }
  }
  if (tid < 32) bulk_wait_all();
}

template <typename T, int D>
cudaError_t launch_d(const RopeParams &p, const NormParams &n, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const long long row = (long long)(p.H + 2 * p.H_kv) * D * (int)sizeof(T);
  if (row * kStages + 4 * (p.rot / 2) * 4 > kRowsSmem)  // rows too long for the ring
    return launch_pdl(qknorm_kernel<T, D>, dim3(p.n_tokens), dim3(kThreads), 0, stream, p, n);
  // tokens of a stage: a block each while there are blocks for them, and no
  // more pairs in a group than threads
  int tpb = kStageBytes / row < kMostTokens ? (int)(kStageBytes / row) : kMostTokens;
  while (tpb > 1 && (p.n_tokens < kRowBlocks * kSms * tpb || tpb * (p.rot / 2) > kThreads)) --tpb;
  if (tpb < 1) tpb = 1;
  const int smem = (int)row * kStages * tpb + 4 * tpb * (p.rot / 2) * 4;
  auto kernel = p.neighbours             ? qknorm_rows_kernel<T, D, kNeighbours>
                : (p.rot / 2) % VE == 0 ? qknorm_rows_kernel<T, D, kHalves>
                                         : qknorm_rows_kernel<T, D, kCut>;
  // as in rope_append.cu: less needs no leave, and the attribute is the process's
  if (smem > 47 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    if (e != cudaSuccess) return e;
  }
  const int by_smem = kRowsSmem / (smem + 2048), per_sm = by_smem < kRowBlocks ? by_smem : kRowBlocks;
  const int most = kSms * (per_sm < 1 ? 1 : per_sm), groups = (p.n_tokens + tpb - 1) / tpb;
  return launch_pdl(kernel, dim3(groups < most ? groups : most), dim3(kThreads), smem, stream, p, n,
                    (uint32_t)(p.H * D * (int)sizeof(T)), (uint32_t)(p.H_kv * D * (int)sizeof(T)),
                    tpb, FastDiv(p.H + p.H_kv));
}

template <typename T>
cudaError_t launch_t(const RopeParams &p, const NormParams &n, int D, cudaStream_t stream) {
  if (D == 64) return launch_d<T, 64>(p, n, stream);
  if (D == 128) return launch_d<T, 128>(p, n, stream);
  return launch_d<T, 256>(p, n, stream);
}

}  // namespace

cudaError_t launch_qknorm_rope(const QkNormArgs &a, cudaStream_t stream) {
  const RopeParams p = rope_params(a.rope);
  const NormParams n{a.q_weight, a.k_weight, a.eps, a.weight_offset};
  return a.rope.cache.bf16 ? launch_t<__nv_bfloat16>(p, n, a.rope.cache.D, stream)
                           : launch_t<float>(p, n, a.rope.cache.D, stream);
}

}  // namespace gdn
