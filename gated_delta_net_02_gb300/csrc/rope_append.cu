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
// Measured on one GB300: 34739 tokens x 20 heads x 256 bf16, 64 of them
// turned, 108 us (6.6 TB/s of 6.8 copied); 64 tokens x 20 heads x 128 2.3 us.
//
// Precision: position * inv_freq in fp32 loses the angle itself once it
// passes some thousand radians (2^-24 of it). The product is formed in turns,
// as the fp32 product plus its exact error (fused multiply-add), so that the
// whole turns drop out exactly and what is left of the angle has an error of
// about 2^-24 turns for positions up to 2^24 and inverse frequencies up to 1;
// beyond, the rounding of position * (the frequency's low part) outgrows that,
// to some 2^-21 turns at 2^31.
#include <cuda_bf16.h>

#include "rope.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Rows too long for the ring of rope_rows_kernel: a block takes one token, a
// thread one 16-byte vector of a head at a time.
// WHOLE: a vector's elements are all rotated with elements of one other
// vector (or of itself), or all pass; otherwise partners are read one by one.
template <typename T, int D, bool WHOLE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VE = 16 / (int)sizeof(T), NVEC = D / VE;
  __shared__ float cs[D / 2], sn[D / 2];
  __shared__ long long at_s;  // element offset of the slot, -1 = none
  const int tid = threadIdx.x, half = p.rot >> 1;
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
  for (int e = tid; e < (p.H + 2 * p.H_kv) * NVEC; e += kThreads) {
    const int d0 = (e % NVEC) * VE;
    int h = e / NVEC;
    const T *src;
    T *dst;
    bool turn = d0 < p.rot;
    if (h < p.H) {
      src = static_cast<const T *>(p.q) + tok * p.q_stride + (long long)h * D;
      dst = static_cast<T *>(p.q_out) + (tok * p.H + h) * D;
    } else {
      h -= p.H;
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

// Persistent blocks; a token's rows pass through shared memory by bulk copies
// both ways. A ring of kStages groups of tpb tokens keeps the next
// groups' loads in flight, which registers could not hold (a thread would
// need them for every 16 bytes under way); only the elements that turn are
// touched by threads, in place, and v and the rest of each head are not.
// (One thread for each 16 bytes, as in rope_kernel, took 186 us on the batch
// above and 2.7 us on 64 tokens.)
// Three stages: two leave too little under way (141 us on that batch), four
// too little shared memory for the blocks (119 us).
constexpr int kStages = 3;
// Blocks on an SM. At four a thread may have 64 registers, which the turning
// of two vectors takes; five cost spills (113 us), and without the bound the
// compiler takes 80, three blocks (112 us).
constexpr int kRowBlocks = 4;
// Bytes of a stage: as many tokens as fit, so that all of a block's threads
// find pairs to turn where rows are short. 30000 tokens x 20 heads x 128 bf16
// (5 KB a token), all of them turned: 75 us with one token a stage, 52 with
// three; 6 heads x 64: 63 and 21 us.
constexpr int kStageBytes = 16 * 1024;
constexpr int kMostTokens = 8;
constexpr int kRowsSmem = 220 * 1024;

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads, kRowBlocks)
    rope_rows_kernel(const RopeParams p, int D, uint32_t q_bytes, uint32_t kv_bytes, int tpb,
                     FastDiv by_unit, FastDiv by_heads) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VE = 16 / (int)sizeof(T);
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
    if constexpr (WHOLE) {
      const int per = p.neighbours ? p.rot / VE : half / VE;
      for (int e = tid; e < nt * heads * per; e += kThreads) {
        const int r = by_unit.div(e), j = by_heads.div(r), h = r - j * heads;
        const int c = (e - r * per) * VE;
        T *a = reinterpret_cast<T *>(st + j * row) + h * D + c;
        const float *cs = cs0 + j * half, *sn = sn0 + j * half;
        Vec16<T> u, w;
        u.load(a);
        if (p.neighbours) {
#pragma unroll
          for (int i = 0; i < VE; i += 2) {
            const int f = (c + i) >> 1;
            const float v = u.v[i] * cs[f] - u.v[i + 1] * sn[f];
            u.v[i + 1] = u.v[i] * sn[f] + u.v[i + 1] * cs[f];
            u.v[i] = v;
          }
        } else {
          w.load(a + half);
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const float v = u.v[i] * cs[c + i] - w.v[i] * sn[c + i];
            w.v[i] = u.v[i] * sn[c + i] + w.v[i] * cs[c + i];
            u.v[i] = v;
          }
          w.store(a + half);
        }
        u.store(a);
      }
    } else {
      for (int e = tid; e < nt * heads * half; e += kThreads) {
        const int r = by_unit.div(e), j = by_heads.div(r), h = r - j * heads;
        const int i = e - r * half;
        T *a = reinterpret_cast<T *>(st + j * row) + h * D + (p.neighbours ? 2 * i : i);
        T *b = a + (p.neighbours ? 1 : half);
        const float u = to_f32(*a), w = to_f32(*b), c = cs0[j * half + i], n = sn0[j * half + i];
        *a = from_f32<T>(u * c - w * n);
        *b = from_f32<T>(u * n + w * c);
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
          const uint32_t n = kv_bytes / runs;
          for (int r = 0; r < runs; ++r) {
            bulk_s2g(kd + r * p.head_stride, src + q_bytes + r * n, n);
            bulk_s2g(vd + r * p.head_stride, src + q_bytes + kv_bytes + r * n, n);
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
cudaError_t launch_d(const RopeParams &p, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const bool whole = p.neighbours ? p.rot % VE == 0 : (p.rot / 2) % VE == 0;
  const long long row = (long long)(p.H + 2 * p.H_kv) * D * (int)sizeof(T);
  if (row * kStages + 4 * (p.rot / 2) * 4 > kRowsSmem) {
    const dim3 grid(p.n_tokens), block(kThreads);
    return whole ? launch_pdl(rope_kernel<T, D, true>, grid, block, 0, stream, p)
                 : launch_pdl(rope_kernel<T, D, false>, grid, block, 0, stream, p);
  }
  // tokens of a stage: a block each while there are blocks for them, and no
  // more pairs in a group than threads
  int tpb = kStageBytes / row < kMostTokens ? (int)(kStageBytes / row) : kMostTokens;
  while (tpb > 1 && (p.n_tokens < kRowBlocks * kSms * tpb || tpb * (p.rot / 2) > kThreads)) --tpb;
  if (tpb < 1) tpb = 1;
  const int smem = (int)row * kStages * tpb + 4 * tpb * (p.rot / 2) * 4;
  const int unit = !whole ? p.rot / 2 : p.neighbours ? p.rot / VE : p.rot / 2 / VE;
  auto kernel = whole ? rope_rows_kernel<T, true> : rope_rows_kernel<T, false>;
  // Less needs no leave, and the call costs the host time. The attribute is the
  // process's: always the most that any call needs, or another thread's call
  // could lower it between here and the launch.
  if (smem > 47 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    if (e != cudaSuccess) return e;
  }
  const int by_smem = kRowsSmem / (smem + 2048), per_sm = by_smem < kRowBlocks ? by_smem : kRowBlocks;
  const int most = kSms * (per_sm < 1 ? 1 : per_sm), groups = (p.n_tokens + tpb - 1) / tpb;
  return launch_pdl(kernel, dim3(groups < most ? groups : most), dim3(kThreads), smem, stream, p,
                    D, (uint32_t)(p.H * D * (int)sizeof(T)),
                    (uint32_t)(p.H_kv * D * (int)sizeof(T)), tpb, FastDiv(unit > 0 ? unit : 1),
                    FastDiv(p.H + p.H_kv));
}

template <typename T>
cudaError_t launch_t(const RopeParams &p, int D, cudaStream_t stream) {
  if (D == 64) return launch_d<T, 64>(p, stream);
  if (D == 128) return launch_d<T, 128>(p, stream);
  return launch_d<T, 256>(p, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t stream) {
  const RopeParams p = rope_params(a);
  return a.cache.bf16 ? launch_t<__nv_bfloat16>(p, a.cache.D, stream)
                      : launch_t<float>(p, a.cache.D, stream);
}

}  // namespace gdn
