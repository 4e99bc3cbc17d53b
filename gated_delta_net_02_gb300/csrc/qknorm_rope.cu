// qknorm_rope.cu -- RMS norm of every q and k head, rotary positions on the
// result, and the append of k and of v to a paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * (offset + weight)     over a head
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos)
//
// Bound by HBM: each element is read once and written once. The sum of a
// head's squares, the norm and the rotation are in fp32, with one rounding at
// the end. Measured on one GB300: 34739 tokens x (16 + 2 + 2) heads of 256, bf16, 64
// rotated, 117 us (104.9 by bytes, 6.1 TB/s); 64 tokens x 20 x 128 11.6 us, of which the
// host takes 9.
#include "rope.cuh"

namespace gdn {
namespace {

struct NormParams {
  const void *qw, *kw;
  float eps, offset;
};

// Persistent warps, each on its own: a warp's tokens pass through its ring of
// kStages units in shared memory, by bulk copies both ways; a unit is tpb tokens, or
// one of `parts` runs of a long row's heads (of q, k and v in turn). No warp waits
// for another (with a block on a token, as in rope_append.cu, its 18
// heads of 256 made two unequal rounds between two barriers: 217 us on 34739
// tokens). A head's row is the work of D / (2 x 16 bytes) lanes, each with two
// vectors of 16 bytes that lie half a rotation apart (so that partners meet in one
// lane), in registers from the sum of squares to the rotation.
constexpr int kStages = 3;
constexpr int kMostWarps = 16;
constexpr int kStageBytes = 4 * 1024;  // of a unit of short rows
constexpr int kPartBytes = 5 * 1024;   // of a part of a long one: 14 warps have room
constexpr int kMostTokens = 8;
constexpr int kMostAngles = 4;         // of a lane and group
constexpr int kRowsSmem = 220 * 1024;

// Two numbers to an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "mul.rn.f32x2 w, u, v;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 w, u, v, w;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// How a rotation meets the vectors of a head: whole vectors of two halves, of
// neighbouring pairs, or pairs of two halves that cut a vector.
enum Meet { kHalves, kNeighbours, kCut };

template <typename T, int D, Meet MEET>
__global__ void __launch_bounds__(32 * kMostWarps)
    qknorm_rows_kernel(const RopeParams p, const NormParams n, int tpb, int parts, int part_heads,
                       int warp_bytes, FastDiv64 by_parts, FastDiv by_q, FastDiv by_kv,
                       FastDiv by_half) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VE = 16 / (int)sizeof(T), LPR = D / VE / 2;  // lanes of a head's row
  extern __shared__ __align__(128) unsigned char smem_all[];
  __shared__ uint64_t full_all[kMostWarps][kStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = p.rot >> 1;
  uint64_t *const full = full_all[warp];
  unsigned char *const smem = smem_all + (size_t)warp * warp_bytes;
  constexpr uint32_t kHead = D * sizeof(T);
  const uint32_t row = part_heads * kHead, stage = tpb * row;
  // sines and cosines of a group of tokens, [tpb][half] each
  float *const cs0 = reinterpret_cast<float *>(smem + kStages * stage), *const sn0 = cs0 + tpb * half;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the grid's units, token by token, taken in turn by its warps
  const long long units = (long long)((p.n_tokens + tpb - 1) / tpb) * parts;
  const long long first = (long long)warp * gridDim.x + blockIdx.x,
                  step = (long long)gridDim.x * (blockDim.x >> 5);
  struct Unit {
    int tok, nt;  // first token, tokens (0: beyond the last unit)
    int h0;       // first of its heads, those of q, k and v counted on
  };
  auto unit_of = [&](int it) {
    const long long x = first + it * step;
    if (x >= units) return Unit{0, 0, 0};
    const int g = (int)(parts == 1 ? x : by_parts.div(x));
    return Unit{g * tpb, min(tpb, p.n_tokens - g * tpb), (int)(x - (long long)g * parts) * part_heads};
  };
  // a unit's heads of those that begin at `from` and are n: the first and how many
  auto heads_of = [&](const Unit &u, int from, int n) {
    const int h = max(u.h0 - from, 0);
    return make_int2(h, max(min(u.h0 + part_heads - from, n) - h, 0));
  };
  // a lane for each token of a unit
  auto load = [&](const Unit &u, int it) {
    const int s = it % kStages;
    if (u.nt == 0) return;
    const int2 q = heads_of(u, 0, p.H), k = heads_of(u, p.H, p.H_kv),
               v = heads_of(u, p.H + p.H_kv, p.H_kv);
    if (lane == 0) mbar_arrive_expect_tx(&full[s], u.nt * (q.y + k.y + v.y) * kHead);
    __syncwarp();
    if (lane < u.nt) {
      const long long tok = u.tok + lane;
      unsigned char *st = smem + s * stage + lane * row;
      if (q.y)
        bulk_g2s(st, static_cast<const T *>(p.q) + tok * p.q_stride + (long long)q.x * D,
                 q.y * kHead, &full[s]);
      if (k.y)
        bulk_g2s(st + q.y * kHead,
                 static_cast<const T *>(p.k) + tok * p.k_stride + (long long)k.x * D, k.y * kHead,
                 &full[s]);
      if (v.y)
        bulk_g2s(st + (q.y + k.y) * kHead,
                 static_cast<const T *>(p.v) + tok * p.v_stride + (long long)v.x * D, v.y * kHead,
                 &full[s]);
    }
  };
  auto slot_of = [&](const Unit &u) -> long long {
    return lane < u.nt ? p.slots[u.tok + lane] : -1;
  };
  static_assert(kStages == 3, "two units ahead of the current one");
  Unit u = unit_of(0), u1 = unit_of(1), u2 = unit_of(2);
  load(u, 0);
  load(u1, 1);
  long long slot = slot_of(u);
  // the lane's two vectors of a head, from these elements on
  const int l = lane % LPR;
  int at_a = 2 * l * VE, at_b = at_a + VE;
  if (MEET == kHalves) {
    const int turning = half / VE;
    at_a = l < turning ? l * VE : p.rot + 2 * (l - turning) * VE;
    at_b = l < turning ? at_a + half : at_a + VE;
  }
  // a vector's factors, as they are stored
  auto weights = [&](const void *w, int at) {
    return *reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + at);
  };
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 wq[2] = {n.qw ? weights(n.qw, at_a) : none, n.qw ? weights(n.qw, at_b) : none};
  const uint4 wk[2] = {n.kw ? weights(n.kw, at_a) : none, n.kw ? weights(n.kw, at_b) : none};
  // A lane has the same pairs of the same tokens of each group: their axes and
  // frequencies stay, their positions are read a group ahead.
  float freq[kMostAngles];
  int my_j[kMostAngles], my_axis[kMostAngles], pos[kMostAngles];
#pragma unroll
  for (int x = 0; x < kMostAngles; ++x) {
    const int e = lane + 32 * x;
    my_j[x] = tpb;
    if (e < tpb * half) {
      my_j[x] = by_half.div(e);
      const int i = e - my_j[x] * half;
      my_axis[x] = axis_of(p, i);
      freq[x] = p.inv_freq[i];
    }
  }
  auto positions = [&](const Unit &u) {
#pragma unroll
    for (int x = 0; x < kMostAngles; ++x)
      if (my_j[x] < u.nt)
        pos[x] = p.positions[(long long)my_axis[x] * p.n_tokens + u.tok + my_j[x]];
  };
  positions(u);
  for (int it = 0; u.nt > 0; ++it) {
    const int s = it % kStages, nt = u.nt;
    const long long next_slot = slot_of(u1);
#pragma unroll
    for (int x = 0; x < kMostAngles; ++x)
      if (my_j[x] < nt)
        sincospif(2.f * reduced_turns(pos[x], freq[x]), &sn0[lane + 32 * x], &cs0[lane + 32 * x]);
    positions(u1);
    const bool ok = mbar_wait(&full[s], (it / kStages) & 1, p.err, kSiteRopeRow);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0)  // the stages loaded ahead
        for (int i = it; i < it + kStages - 1 && (i == it || u1.nt > 0); ++i)
          mbar_drain(&full[i % kStages], (i / kStages) & 1);
      break;
    }
    __syncwarp();  // a vote orders no memory: other lanes read the sines stored above
    unsigned char *st = smem + s * stage;
    // H heads of each token of the unit, from its h0-th on.
    auto norm_rows = [&](int h0, int H, const FastDiv &by_H, const void *weight, const uint4 (&w)[2]) {
      // offset + weight, for the lane's two vectors; 1 without a weight
      float2 f[VE];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Vec16<T> v;
        v.unpack(w[x]);
        const float base = weight ? n.offset : 1.f;
#pragma unroll
        for (int i = 0; i < VE; i += 2)
          f[(x * VE + i) / 2] = make_float2(base + v.v[i], base + v.v[i + 1]);
      }
      const int rows = nt * H;
#pragma unroll 2
      for (int r0 = 0; r0 < rows; r0 += 32 / LPR) {
        const int r = r0 + lane / LPR;
        const bool live = r < rows;
        const int j = by_H.div(live ? r : 0), h = h0 + (live ? r : 0) - j * H;
        T *head = reinterpret_cast<T *>(st + j * row) + h * D;
        Vec16<T> a, b;
        a.load(head + at_a);
        b.load(head + at_b);
        float2 y[VE];  // the two vectors' pairs
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          y[i / 2] = make_float2(a.v[i], a.v[i + 1]);
          y[(VE + i) / 2] = make_float2(b.v[i], b.v[i + 1]);
        }
        float2 squares = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VE; ++i) squares = fma2(y[i], y[i], squares);
        float sum = squares.x + squares.y;
#pragma unroll
        for (int off = LPR / 2; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float inv = rsqrtf(fmaf(sum, 1.f / D, n.eps));
#pragma unroll
        for (int i = 0; i < VE; ++i) y[i] = mul2(y[i], mul2(f[i], make_float2(inv, inv)));
        const float *cs = cs0 + j * half, *sn = sn0 + j * half;
        if constexpr (MEET == kHalves) {
          if (at_a < half) {
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
              const float2 c = *reinterpret_cast<const float2 *>(cs + at_a + i);
              const float2 t = *reinterpret_cast<const float2 *>(sn + at_a + i);
              const float2 u = y[i / 2], v = y[(VE + i) / 2];
              y[i / 2] = fma2(make_float2(-v.x, -v.y), t, mul2(u, c));
              y[(VE + i) / 2] = fma2(u, t, mul2(v, c));
            }
          }
        } else if constexpr (MEET == kNeighbours) {
          // a vector's pairs stand side by side, at_b behind at_a
          const int pair0 = at_a >> 1;
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            if (pair0 + i >= half) break;
            const float c = cs[pair0 + i], t = sn[pair0 + i];
            y[i] = fma2(make_float2(-y[i].y, y[i].x), make_float2(t, t),
                        mul2(y[i], make_float2(c, c)));
          }
        }
        if constexpr (MEET != kCut) {
#pragma unroll
          for (int i = 0; i < VE; i += 2) {
            a.v[i] = y[i / 2].x;
            a.v[i + 1] = y[i / 2].y;
            b.v[i] = y[(VE + i) / 2].x;
            b.v[i + 1] = y[(VE + i) / 2].y;
          }
          if (live) {
            a.store(head + at_a);
            b.store(head + at_b);
          }
        } else {
          // the partners lie in other lanes' vectors: read again, once the row's
          // sum is known, and normed one by one
          auto normed = [&](int d) {
            const float x = to_f32(head[d]) * inv;
            return weight ? x * (n.offset + to_f32(static_cast<const T *>(weight)[d])) : x;
          };
          __syncwarp();
          if (live) {
            for (int i = l; i < half; i += LPR) {
              const float u = normed(i), v = normed(i + half), c = cs[i], t = sn[i];
              head[i] = from_f32<T>(u * c - v * t);
              head[i + half] = from_f32<T>(u * t + v * c);
            }
            for (int d = p.rot + l; d < D; d += LPR) head[d] = from_f32<T>(normed(d));
          }
        }
      }
    };
    // (a part of a row has one token: all of its rows are below by_H's divisor)
    const int2 qs = heads_of(u, 0, p.H), ks = heads_of(u, p.H, p.H_kv),
               vs = heads_of(u, p.H + p.H_kv, p.H_kv);
    norm_rows(0, qs.y, by_q, n.qw, wq);
    norm_rows(qs.y, ks.y, by_kv, n.kw, wk);
    fence_proxy_async();
    __syncwarp();
    if (lane < nt) {
      const long long tok = u.tok + lane;
      const unsigned char *src = st + lane * row;
      if (qs.y)
        bulk_s2g(static_cast<T *>(p.q_out) + (tok * p.H + qs.x) * D, src, qs.y * kHead);
      if (slot >= p.n_slots) {
        set_error(p.err, kDevBadSlot);
      } else if (slot >= 0) {
        // a slot's heads are one run of the cache unless its layout parts them
        const long long at = slot_offset(p, slot);
        auto append = [&](void *cache, int2 heads, const unsigned char *from) {
          T *to = static_cast<T *>(cache) + at + heads.x * p.head_stride;
          const bool one = p.head_stride == D;
          const int runs = one ? heads.y > 0 : heads.y;
          const uint32_t bytes = one ? heads.y * kHead : kHead;
          for (int r = 0; r < runs; ++r) bulk_s2g(to + r * p.head_stride, from + r * bytes, bytes);
        };
        append(p.k_cache, ks, src + qs.y * kHead);
        append(p.v_cache, vs, src + (qs.y + ks.y) * kHead);
      }
    }
    bulk_commit();
    slot = next_slot;
    // the stage loaded next was stored from an iteration ago: all but the
    // stores just issued have read theirs
    bulk_wait_read_but1();
    __syncwarp();
    load(u2, it + 2);
    u = u1;
    u1 = u2;
    u2 = unit_of(it + 3);
  }
  bulk_wait_all();
}

template <typename T, int D>
cudaError_t launch_d(const RopeParams &p, const NormParams &n, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const long long row = (long long)(p.H + 2 * p.H_kv) * D * (int)sizeof(T);
  const int half = p.rot / 2;
  // parts of a token's row; tokens of a unit: a warp each while there are warps for them
  const int heads = p.H + 2 * p.H_kv, head = D * (int)sizeof(T);
  int parts = (int)((row + kPartBytes - 1) / kPartBytes);
  const int part_heads = (heads + parts - 1) / parts;
  parts = (heads + part_heads - 1) / part_heads;
  int tpb = parts == 1 ? (int)(kStageBytes / row) : 1;
  if (tpb > kMostTokens) tpb = kMostTokens;
  while (tpb > 1 && (p.n_tokens < kMostWarps * kSms * tpb || tpb * half > 32 * kMostAngles)) --tpb;
  if (tpb < 1) tpb = 1;
  const long long units = (long long)((p.n_tokens + tpb - 1) / tpb) * parts;
  // a warp's ring and its angles; bulk copies want 16 bytes
  const int warp_bytes = kStages * tpb * part_heads * head + (8 * tpb * half + 15) / 16 * 16;
  const int fit = kRowsSmem / warp_bytes, most = fit < kMostWarps ? fit : kMostWarps;
  const long long each = (units + kSms - 1) / kSms;
  const int warps = each < most ? (int)each : most;
  const long long blocks = (units + warps - 1) / warps;
  auto kernel = p.neighbours     ? qknorm_rows_kernel<T, D, kNeighbours>
                : half % VE == 0 ? qknorm_rows_kernel<T, D, kHalves>
                                 : qknorm_rows_kernel<T, D, kCut>;
  // as in rope_append.cu: less needs no leave, and the attribute is the process's
  const int smem = warps * warp_bytes;
  if (smem > 47 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(blocks < kSms ? (unsigned)blocks : kSms), dim3(32 * warps), smem,
                    stream, p, n, tpb, parts, part_heads, warp_bytes, FastDiv64(parts), FastDiv(p.H),
                    FastDiv(p.H_kv), FastDiv(half > 0 ? half : 1));
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
