// sample.cu -- one token for each row of logits: temperature, top-k, top-p and
// min-p, from a given random number.
//
//   w_i = exp((x_i - max x) / temperature)
//   kept = the first n of the descending order (equal logits: lower index first)
//   token = first kept index, by index, whose running mass passes u * mass
//
// Bound by HBM: a row is read once; a cluster of up to 8 blocks holds it in
// shared memory and makes all further passes there. Measured on one GB300 (bytes at
// the copy rate in brackets): 64 rows of 131072 bf16, top k and top p 37.4 us (2.5);
// 512 rows of 150001 fp32, top p and min p, 523 us (45.2): some 140 instructions a
// logit, and a third of the time at barriers of blocks and clusters.
//  * Masses decide between tokens by whole numbers: a weight is an integer in
//    units of 2^-44 of (about) the largest, so a sum has the same value in any
//    order, and with it the token. Logits lie on a grid of 2^-8 to 2^-7 octaves of
//    weight; a weight is the product of two table entries for its grid point and
//    a polynomial for the rest, in 32-bit mantissas: some 2^-30 of itself off.
//    Tokens below 2^-45 of the largest have mass 0.
//  * The order is never made. The last kept value is found by histograms:
//    16 grid points a bin first, then the bin's values by their ordered
//    bits, 512 bins at a time, until a bin is one value. Of the tokens with
//    that value the lowest indexes are kept.
//  * The first histogram of masses adds a weight as three numbers of 16 bits,
//    by 32-bit atomics that are skipped where they are 0, as the upper ones
//    mostly are; one 64-bit addition to shared memory is a loop.
//  * The last bin's logits are listed while they are counted (and those before
//    it, where a count left few), and later passes go by the list.
//  * A bin is looked for in sums of 32 bins first, then in those 32: blocks read
//    one another's shared memory slowly (all bins by all blocks took 6 us).
#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.cuh"

namespace gdn {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;       // of a cluster
constexpr int kBins = 768, kFineBins = 512;  // of the first histograms and of a bin's
constexpr int kSms = 152;
constexpr float kOctaves = 44.9f;     // further down, weights are 0
constexpr int kGroups = 16;          // pieces of a warp's share with a mass of their own
constexpr int kList = 1024;          // logits that a block lists
constexpr int kFine = 64, kCoarse = 184;  // table entries: 45 octaves x 256 points, by 64

struct SampleParams {
  const void *logits;
  long long stride;
  const float *temperature, *top_p, *min_p, *uniform;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  int rows, vocab;
};

// A float's bits in the order of the values, +0 and -0 the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu));
}
// The largest value below x. The key before 0's is no value's (it would be -0): the
// largest negative number's is the one before that.
__device__ __forceinline__ float below(float x) {
  const uint32_t k = key_of(x) - 1;
  return of_key(k == 0x7fffffffu ? 0x7ffffffeu : k);
}

__device__ __forceinline__ u64 ld_cluster_u64(const void *local, uint32_t rank) {
  u64 v;
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void *local, uint32_t rank) {
  uint32_t v, remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += up;
  }
  return v;
}

// The row's grid of logits. Its step is the power of two that makes 2^-8 to 2^-7
// octaves; point j lies j steps below the largest logit's.
struct Grid {
  // A coarse entry: 2^(-64 j steps) as mantissa, and the factors that take a
  // product of mantissas to units of 2^-44: 2^(12 - n) above, 2^(44 - n) below 2^32.
  struct Coarse {
    uint32_t mantissa, above, below, pad;
  };
  float from;      // logits less this, 0 or the largest: exact (Sterbenz) where it is not 0
  float low;       // the lowest logit with any weight
  float magic;     // 1.5 x 2^23 steps: adding it leaves the point in the low bits
  int top;         // bits of the largest logit's sum
  float ln_step;   // logits to natural logarithms of weight
  const Coarse *coarse;
  const uint32_t *fine;

  // The point of x >= low: the same for equal logits, never smaller for a smaller one.
  __device__ __forceinline__ int point(float x) const {
    return top - __float_as_int(__fadd_rd(x - from, magic));
  }
  // The weight of x >= low, and its point.
  __device__ __forceinline__ u64 weight(float x, int &j) const {
    const float d = x - from, sum = __fadd_rd(d, magic);
    j = top - __float_as_int(sum);
    const float t = (d - (sum - magic)) * ln_step;  // 0 <= t < 2^-7.5, from an exact rest
    const Coarse c = coarse[j >> 6];
    const uint32_t m = __umulhi(c.mantissa, fine[j & 63]);
    // e^t - 1
    const float e = fmaf(t * t, fmaf(t, 1.f / 6, 0.5f), t);
    const uint32_t v = m + __umulhi(m, __float2uint_rn(e * 4294967296.f));
    return (u64)v * c.above + (((u64)v * c.below + 0x80000000u) >> 32);
  }
  __device__ __forceinline__ u64 weight(float x) const {
    int j;
    return weight(x, j);
  }
};

// Positive numbers below 1 as 64-bit fractions and powers of two: value
// fraction 2^-64 2^-shift, the fraction's top bit set.
struct Small {
  u64 fraction;
  int shift;
};
__device__ __forceinline__ Small operator*(Small a, Small b) {
  u64 f = __umul64hi(a.fraction, b.fraction);
  int n = a.shift + b.shift;
  if (!(f >> 63)) {
    f <<= 1;
    ++n;
  }
  return Small{f, n};
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ explicit Vec(uint4 u) {
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
  __device__ __forceinline__ uint4 pack() const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        w[i] = __float_as_uint(v[2 * i]) >> 16 | (__float_as_uint(v[2 * i + 1]) & 0xffff0000u);
      else
        w[i] = __float_as_uint(v[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct Shared {
  Grid::Coarse coarse[kCoarse];
  uint32_t fine[kFine];
  // two histograms in turn, so that one is cleared while the other is read
  union Histogram {
    uint32_t part[3][kBins];  // of the grid's bins: a number in parts of 16 bits
    struct {                  // of one bin's values: mass, tokens, largest key
      u64 mass[kFineBins];
      uint32_t count[kFineBins], most[kFineBins];
    } fine;
  };
  alignas(16) Histogram hist[2];
  u64 group[2][32];        // sums of 32 bins
  Small power[14];         // 2^(-2^k steps)
  float queue[kWarps][64];
  float list[kList];
  u64 warp_part[kWarps], warp_part2[kWarps];
  u64 seg_mass[kWarps][kGroups];
  uint32_t seg_ties[kWarps][kGroups];
  alignas(16) u64 warp_mass[kWarps];
  u64 warp_kept[kWarps];
  alignas(16) uint32_t warp_ties[kWarps];
  float top, step, ln_step, least;
  float depth;             // logits from the largest to weight 0
  double min_drop;         // t * log(min_p)
  float warp_top[kWarps];
  int found, listed;
  u64 before, there, goal, total;
};

// A row's share of one block, and the passes over it.
template <typename T>
struct Share {
  static constexpr int VE = 16 / (int)sizeof(T);
  const T *row;      // the row's first 16-byte boundary at or below its start
  int before, cols;  // elements before the row's start, and after it begins
  int v0, v1;        // this warp's vectors, counted from `row`
  uint4 *own;        // this warp's place in shared memory
  float *queue;      // and its queue of 64

  // A vector of the row's ends: what is not of the row is -inf.
  __device__ __forceinline__ Vec<T> fetch_end(int v) const {
    const T *p = row + (long long)v * VE;
    const int e0 = v * VE - before;  // index of the first element
    Vec<T> x(make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int i = 0; i < VE; ++i)
      x.v[i] = e0 + i >= 0 && e0 + i < cols ? to_f32(p[i]) : -INFINITY;
    return x;
  }
  // The share to shared memory: whole vectors by asynchronous copies, all of
  // them under way at once; each lane's are those that it reads later.
  __device__ __forceinline__ void load() const {
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
    const int lane = threadIdx.x & 31;
    const int f0 = max(v0, before ? 1 : 0), f1 = min(v1, (before + cols) / VE);
    for (int v = v0 + lane; v < v1; v += 32) {
      if (v >= f0 && v < f1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(own + (v - v0))),
                     "l"(p + v)
                     : "memory");
      else
        own[v - v0] = fetch_end(v).pack();
    }
  }
  __device__ __forceinline__ Vec<T> get(int v) const { return Vec<T>(own[v - v0]); }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = v0 + (threadIdx.x & 31); v < v1; v += 32) {
      const Vec<T> x = get(v);
#pragma unroll
      for (int i = 0; i < VE; ++i) f(x.v[i]);
    }
  }
  // f(x) for the logits lo <= x <= hi of the warp's chunks c0 .. c1 of 32 vectors;
  // every lane of the warp takes part. Where they are few, a lane would wait for
  // another's f at each of its own logits: they are queued, and 32 of them
  // done at once.
  template <class F>
  __device__ __forceinline__ void each_between(float lo, float hi, int c0, int c1, F f) const {
    const int lane = threadIdx.x & 31;
    int n = 0;  // in the queue
    for (int c = c0; c < c1; ++c) {
      const int v = v0 + c * 32 + lane;
      Vec<T> x(make_uint4(0, 0, 0, 0));
      if (v < v1) x = get(v);
      bool in[VE];
      int mine = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        in[i] = v < v1 && x.v[i] >= lo && x.v[i] <= hi;
        mine += in[i];
      }
      const uint32_t some = __ballot_sync(0xffffffffu, mine);
      if (!some) continue;
      if (__reduce_add_sync(0xffffffffu, mine) >= 16 * VE) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (in[i]) f(x.v[i]);
        continue;
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, in[i]);
        if (!m) continue;
        if (in[i]) queue[n + __popc(m & ((1u << lane) - 1))] = x.v[i];
        n += __popc(m);
        if (n >= 32) {
          __syncwarp();
          const float first = queue[lane], rest = queue[32 + lane];
          __syncwarp();
          n -= 32;
          if (lane < n) queue[lane] = rest;
          f(first);
        }
      }
    }
    __syncwarp();
    if (lane < n) f(queue[lane]);
    __syncwarp();
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const SampleParams p, int blocks, int warp_vecs) {
  constexpr int VE = 16 / (int)sizeof(T);
  // bf16 values differ in the upper half of their bits alone
  constexpr int kLow = sizeof(T) == 2 ? 16 : 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % blocks;
  const long long r = blockIdx.x / blocks;
  auto clear = [&](int b) {
    for (int i = tid; i < (int)sizeof(sh.hist[b]) / 16; i += kThreads)
      reinterpret_cast<uint4 *>(&sh.hist[b])[i] = make_uint4(0, 0, 0, 0);
  };
  clear(0);
  clear(1);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Share<T> share;
  {
    const T *start = static_cast<const T *>(p.logits) + r * p.stride;
    share.before = (int)((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
    share.row = start - share.before;
    share.cols = p.vocab;
    const int vecs = (share.before + p.vocab + VE - 1) / VE;
    share.v0 = min((rank * kWarps + warp) * warp_vecs, vecs);
    share.v1 = min(share.v0 + warp_vecs, vecs);
    share.own = reinterpret_cast<uint4 *>(smem) + warp * warp_vecs;
    share.queue = sh.queue[warp];
  }
  const float temperature = p.temperature ? p.temperature[r] : 1.f;
  const float t = fminf(fmaxf(temperature, 1e-30f), 3e33f);  // as weights count it
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float u = p.uniform[r];

  // ---- the row arrives; its maximum
  share.load();
  // 64-bit floating point is two operations a cycle of an SM, and slow to
  // return: where it is needed, one thread does it.
  if (tid == 0) {
    // octaves of weight for each unit of logit, log2(e) / t, as the sum of two
    // floats; steps stay inside fp32's range
    const float c = 1.442695041f / t;
    const float c_lo = (fmaf(-c, t, 1.442695041f) + 1.925963033e-8f) / t;
    const int e = (__float_as_int(c) >> 23) - 127;
    sh.step = __int_as_float((127 - 8 - e) << 23);
    sh.ln_step = c * 0.693147181f;
    sh.depth = kOctaves / c;
    // octaves of a step (2^-8 to 2^-7), then x = their natural logarithm's size, in
    // units of 2^-64; 2^-step = e^-x by its series
    const u64 octaves = ((u64)(__float_as_int(c) & 0x7fffff | 0x800000) << 33) +
                        (u64)(long long)(c_lo * sh.step * 18446744073709551616.f);
    const u64 x = __umul64hi(octaves, 0xb17217f7d1cf79acull);
    u64 sum = ~0ull / 720;
#pragma unroll
    for (int n = 5; n >= 1; --n) {
      u64 inverse = ~0ull;  // 1 / n!
      for (int i = 2; i <= n; ++i) inverse /= i;
      sum = inverse - __umul64hi(x, sum);
    }
    Small power{0ull - __umul64hi(x, sum), 0};
    for (int k = 0; k < 14; ++k) {
      sh.power[k] = power;
      power = power * power;
    }
  }
  if (tid == kThreads - 1 && min_p > 0.f)
    sh.min_drop = (double)t * log((double)min_p);
  __syncthreads();
  if (tid < kCoarse + kFine) {
    const int i = tid < kCoarse ? tid * kFine : tid - kCoarse;
    Small m{~0ull, 0};
#pragma unroll
    for (int k = 0; k < 14; ++k)
      if (i >> k & 1) m = m * sh.power[k];
    // as a mantissa of up to 2^32 and 2^-n
    const int n = m.shift;
    const uint32_t mantissa = (uint32_t)(m.fraction >> 32);
    if (tid < kCoarse)
      // 0.99: room for what the polynomial adds
      sh.coarse[tid] = Grid::Coarse{__umulhi(mantissa, 4252017623u), n <= 12 ? 1u << (12 - n) : 0u,
                                    n > 12 && n <= 44 ? 1u << (44 - n) : 0u, 0u};
    else
      sh.fine[tid - kCoarse] = mantissa >> n;  // n = 0 or 1
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  float top = -INFINITY;
  share.each([&](float x) { top = fmaxf(top, x); });
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
    sh.top = top;
  }
  cluster_sync();
  top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMostBlocks; ++k)
    if (k < blocks) top = fmaxf(top, __uint_as_float(ld_cluster_u32(&sh.top, k)));
  if (top == -INFINITY) {  // nothing to choose from
    if (rank == 0 && tid == 0) {
      p.tokens[r] = -1;
      if (p.probs) p.probs[r] = 0.f;
    }
    cluster_sync();
    return;
  }
  if (top == INFINITY) {  // tokens at infinity share all of the mass
    for (int v = share.v0 + lane; v < share.v1; v += 32) {
      Vec<T> x = share.get(v);
#pragma unroll
      for (int i = 0; i < VE; ++i) x.v[i] = x.v[i] == INFINITY ? 0.f : -INFINITY;
      share.own[v - share.v0] = x.pack();
    }
    top = 0.f;
  }
  Grid grid;
  {
    // far from 0, fp32 has no room for the grid beside the logit's own size;
    // less the largest, all that have weight are exact
    grid.from = fabsf(top) > 32.f * sh.depth ? top : 0.f;
    grid.magic = 12582912.f * sh.step;
    // upwards: rounded down it could admit the logit before the largest, further than
    // the table's octaves below it, or -inf
    grid.low = __fsub_ru(top, sh.depth);
    grid.top = __float_as_int(__fadd_rd(top - grid.from, grid.magic));
    grid.ln_step = sh.ln_step;
    grid.coarse = sh.coarse;
    grid.fine = sh.fine;
  }

  // the smallest logit that is not below min_p's bound
  if (tid == kThreads - 1 && min_p > 0.f)
    sh.least = fminf(__double2float_ru((double)top + sh.min_drop), top);

  // What is kept: logits above `cut`, and the first `ties` tokens at it.
  float cut = -INFINITY;
  u64 ties = 0;
  int buf = 0;  // histogram in use
  auto bin_of = [&](float x) { return grid.point(x) >> 4; };
  const int chunks = (share.v1 - share.v0 + 31) / 32;  // of 32 vectors

  // The end of a pass that filled a histogram: value(bin) is what is looked for
  // in it. Whoever is behind the cluster's barrier has read the histogram
  // before, which is cleared for the pass after.
  auto pass_done = [&](int bins, auto value) {
    __syncthreads();
    u64 sum = 0;
    if (2 * tid < bins) sum = value(sh.hist[buf], 2 * tid) + value(sh.hist[buf], 2 * tid + 1);
#pragma unroll
    for (int off = 8; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if ((lane & 15) == 0) sh.group[buf][tid >> 4] = sum;
    cluster_sync();
    clear(buf ^ 1);
  };
  // Finds the bin where the running value, `have` before the first, first reaches
  // want(sum of all): one warp, first in the groups of 32 bins, then in one. far(k, bin)
  // reads block k's. Leaves sh.found (-1: none), sh.before it, and sh.goal = want.
  auto search = [&](u64 have, auto want_of, auto far) {
    if (warp == 0) {
      u64 x = 0;
#pragma unroll
      for (int k = 0; k < kMostBlocks; ++k)
        if (k < blocks) x += ld_cluster_u64(&sh.group[buf][lane], k);
      u64 end = have + warp_scan(x);
      const u64 total = __shfl_sync(0xffffffffu, end, 31);
      const u64 want = want_of(total);
      uint32_t at = __ballot_sync(0xffffffffu, end - x < want && want <= end);
      int found = -1;
      u64 before = 0;
      if (at) {
        const int g = __ffs(at) - 1;
        before = __shfl_sync(0xffffffffu, end - x, g);
        x = 0;
#pragma unroll
        for (int k = 0; k < kMostBlocks; ++k)
          if (k < blocks) x += far(k, g * 32 + lane);
        end = before + warp_scan(x);
        at = __ballot_sync(0xffffffffu, end - x < want && want <= end);
        const int i = __ffs(at) - 1;
        before = __shfl_sync(0xffffffffu, end - x, i & 31);
        found = g * 32 + i;
      }
      if (lane == 0) {
        sh.found = found;
        sh.before = before;
        sh.goal = want;
        sh.total = total;
      }
    }
    __syncthreads();
  };
  auto count_in = [](const Shared::Histogram &h, int i) -> u64 { return h.fine.count[i]; };
  auto mass_in = [](const Shared::Histogram &h, int i) -> u64 { return h.fine.mass[i]; };
  auto low_in = [](const Shared::Histogram &h, int i) -> u64 { return h.part[0][i]; };
  auto parts_in = [](const Shared::Histogram &h, int i) -> u64 {
    return h.part[0][i] + ((u64)h.part[1][i] << 16) + ((u64)h.part[2][i] << 32);
  };
  auto far_count = [&](int k, int i) -> u64 { return ld_cluster_u32(&sh.hist[buf].fine.count[i], k); };
  auto far_mass = [&](int k, int i) { return ld_cluster_u64(&sh.hist[buf].fine.mass[i], k); };
  auto far_low = [&](int k, int i) -> u64 { return ld_cluster_u32(&sh.hist[buf].part[0][i], k); };
  auto far_parts = [&](int k, int i) {
    return ld_cluster_u32(&sh.hist[buf].part[0][i], k) +
           ((u64)ld_cluster_u32(&sh.hist[buf].part[1][i], k) << 16) +
           ((u64)ld_cluster_u32(&sh.hist[buf].part[2][i], k) << 32);
  };

  // f(x) for the block's logits lo <= x <= hi, by all of its threads: from the list where
  // it has them all; or by the row, and then (`list`) they are listed.
  float list_lo = INFINITY, list_hi = -INFINITY;  // what the list was made of
  auto visit = [&](float lo, float hi, bool list, auto f) {
    if (!list && list_lo <= lo && hi <= list_hi && sh.listed <= kList) {
      const int n = sh.listed;
      for (int i = tid; i < n; i += kThreads) {
        const float x = sh.list[i];
        if (x >= lo && x <= hi) f(x);
      }
      return;
    }
    share.each_between(lo, hi, 0, chunks, [&](float x) {
      f(x);
      if (list) {
        const int at = atomicAdd(&sh.listed, 1);
        if (at < kList) sh.list[at] = x;
      }
    });
  };
  // The value at which the order's running count (BY_MASS: mass) first reaches
  // `want`, among the logits from `low` on in bin `bin`; `have` = what comes
  // before that bin. Leaves the value in cut, what comes before it in sh.before
  // and the tokens with it in sh.there.
  auto refine = [&](bool by_mass, u64 want, float low, int bin, u64 have) {
    // a range that holds every value of the bin, by a margin of some roundings
    const int edge = grid.top - __float_as_int(grid.magic) - 16 * bin;  // its first point, in steps
    const float lo = fmaxf(of_key(key_of((edge - 15) * sh.step + grid.from) - 8), low);
    const float hi = fminf(of_key(key_of((edge + 1) * sh.step + grid.from) + 8), top);
    uint32_t khi = key_of(hi) >> kLow, klo = key_of(lo) >> kLow;
    for (;;) {
      int shift = 0;
      while ((khi - klo) >> shift >= (uint32_t)kFineBins) ++shift;
      // the last of a count has few before it, which the masses are made of: they
      // are listed with the bin's
      const bool list = !(list_lo <= lo && hi <= list_hi);
      if (list) {
        list_lo = lo;
        list_hi = !by_mass && have <= kList ? top : hi;
        if (tid == 0) sh.listed = 0;
        __syncthreads();
      }
      visit(lo, list ? list_hi : hi, list, [&](float x) {
        const uint32_t k = key_of(x) >> kLow;
        if (bin_of(x) != bin || k > khi || k < klo) return;
        const int i = (int)((khi - k) >> shift);
        auto &h = sh.hist[buf].fine;
        atomicAdd(&h.count[i], 1u);
        atomicMax(&h.most[i], k);
        if (by_mass) atomicAdd(&h.mass[i], grid.weight(x));
      });
      if (by_mass) {
        pass_done(kFineBins, mass_in);
        search(have, [&](u64) { return want; }, far_mass);
      } else {
        pass_done(kFineBins, count_in);
        search(have, [&](u64) { return want; }, far_count);
      }
      const int i = sh.found;
      have = sh.before;
      // the bin's tokens, and their largest key
      uint32_t there = 0, key = 0;
#pragma unroll
      for (int k = 0; k < kMostBlocks; ++k)
        if (k < blocks) {
          there += ld_cluster_u32(&sh.hist[buf].fine.count[i], k);
          key = max(key, ld_cluster_u32(&sh.hist[buf].fine.most[i], k));
        }
      buf ^= 1;
      if (shift == 0 || there == 1) {  // one value
        key <<= kLow;
        if constexpr (kLow > 0) key |= (int)key < 0 ? 0u : 0xffffu;
        cut = of_key(key);
        if (tid == 0) sh.there = there;
        __syncthreads();
        return;
      }
      __syncthreads();
      khi -= (uint32_t)i << shift;
      const uint32_t span = (1u << shift) - 1;
      klo = khi - klo > span ? khi - span : klo;
    }
  };

  const bool greedy = !(temperature > 0.f) || min_p > 1.f;
  if (greedy) {
    cut = top;
    ties = 1;
  } else {
    if (top_k > 0 && top_k < p.vocab) {
      share.each([&](float x) {
        if (x >= grid.low) atomicAdd(&sh.hist[buf].part[0][bin_of(x)], 1u);
      });
      pass_done(kBins, low_in);
      search(0, [&](u64) { return (u64)top_k; }, far_low);
      const int bin = sh.found;
      const u64 have = sh.before;
      __syncthreads();
      buf ^= 1;
      if (bin >= 0) {  // else fewer tokens than top_k have any mass
        refine(false, (u64)top_k, grid.low, bin, have);
        ties = (u64)top_k - sh.before;
      }
    }
    if (top_p < 1.f) {
      const float low = fmaxf(grid.low, of_key(key_of(cut) + 1));
      visit(low, top, false, [&](float x) {
        int j;
        const u64 w = grid.weight(x, j);
        auto &part = sh.hist[buf].part;
        const int b = j >> 4;
        atomicAdd(&part[0][b], (uint32_t)w & 0xffff);
        const uint32_t up = (uint32_t)(w >> 16);
        if (up) {
          atomicAdd(&part[1][b], up & 0xffff);
          if (up >> 16) atomicAdd(&part[2][b], up >> 16);
        }
      });
      pass_done(kBins, parts_in);
      const u64 tie_weight = ties > 0 ? grid.weight(cut) : 0;
      search(0, [&](u64 total) {
        const double goal = ceil((double)top_p * (double)(total + ties * tie_weight));
        return goal < 1. ? (u64)1 : (u64)goal;
      }, far_parts);
      const u64 want = sh.goal, have = sh.before, total = sh.total;
      const int bin = sh.found;
      __syncthreads();
      buf ^= 1;
      u64 least = want - total, each = tie_weight, most = ties;  // beyond the last of the top k
      if (bin >= 0) {
        refine(true, want, low, bin, have);
        least = want - sh.before;
        each = grid.weight(cut);
        most = sh.there;
      }
      ties = most > 1 && each ? min(most, (least + each - 1) / each) : most;
    }
    if (min_p > 0.f) {
      __syncthreads();
      const float least = sh.least;
      if (least > cut) {  // all of that value: what is below it goes
        cut = below(least);
        ties = 0;
      }
    }
  }

  // ---- the masses of the warps' shares, piece by piece
  const int per = (chunks + kGroups - 1) / kGroups;
  u64 cut_weight = 0;
  if (ties > 0) {
    if (greedy) cut_weight = 1;
    else if (cut >= grid.low) cut_weight = grid.weight(cut);
  }
  // the lowest logit kept: tokens at the cut are counted
  const float low = ties > 0 ? cut : fmaxf(grid.low, of_key(key_of(cut) + 1));
  u64 warp_total = 0;
  uint32_t warp_at_cut = 0;
  for (int g = 0; g < kGroups; ++g) {
    u64 mass = 0;
    uint32_t n = 0;
    if (g * per < chunks)
      share.each_between(low, top, g * per, min((g + 1) * per, chunks), [&](float x) {
        if (x == cut) ++n;
        else if (x >= grid.low) mass += grid.weight(x);
      });
    if (__any_sync(0xffffffffu, (uint32_t)mass | (uint32_t)(mass >> 32) | n)) {
      mass = warp_sum(mass);
      n = __reduce_add_sync(0xffffffffu, n);
    }
    if (lane == 0) {
      sh.seg_mass[warp][g] = mass;
      sh.seg_ties[warp][g] = n;
    }
    warp_total += mass;
    warp_at_cut += n;
  }
  if (lane == 0) {
    sh.warp_mass[warp] = warp_total;
    sh.warp_ties[warp] = warp_at_cut;
  }
  cluster_sync();
  // one warp scans all warps' masses, four of each lane, and leaves its block's
  if (warp == 0) {
    static_assert(kMostBlocks * kWarps == 4 * 32, "four of each lane");
    const int from = lane / (kWarps / 4), w = lane % (kWarps / 4) * 4;
    u64 m[4] = {0, 0, 0, 0}, n[4] = {0, 0, 0, 0}, m_sum = 0, n_sum = 0;
    if (from < blocks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = ld_cluster_u64(&sh.warp_mass[w + i], from);
        n[i] = ld_cluster_u32(&sh.warp_ties[w + i], from);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) n_sum += n[i];
    u64 seen = warp_scan(n_sum) - n_sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 seen_i = seen;
      m[i] += (seen < ties ? min(n[i], ties - seen) : 0) * cut_weight;
      m_sum += m[i];
      seen += n[i];
      n[i] = seen_i;
    }
    u64 run = warp_scan(m_sum) - m_sum;
    if (from == rank) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sh.warp_part[w + i] = run;
        sh.warp_part2[w + i] = n[i];
        sh.warp_kept[w + i] = m[i];
        run += m[i];
      }
      run -= m_sum;
    }
    const u64 total = __shfl_sync(0xffffffffu, run + m_sum, 31);
    if (lane == 0) {
      // the first token whose running mass is above u * total
      u64 x = 0;
      if (u > 0.f) {
        const double at = (double)u * (double)total;
        x = at < (double)total ? min((u64)at, total - 1) : total - 1;
      }
      sh.goal = x;
      sh.total = total;
    }
  }
  __syncthreads();
  const u64 total = sh.total, goal = sh.goal, my_before = sh.warp_part[warp],
            my_seen = sh.warp_part2[warp], my_mass = sh.warp_kept[warp];
  if (my_before <= goal && goal < my_before + my_mass) {
    // the piece, then its vectors in order
    u64 m = lane < kGroups ? sh.seg_mass[warp][lane] : 0, n = lane < kGroups ? sh.seg_ties[warp][lane] : 0;
    const u64 n_before = my_seen + warp_scan(n) - n;
    m += (n_before < ties ? min(n, ties - n_before) : 0) * cut_weight;
    const u64 end = my_before + warp_scan(m);
    const int g = __ffs(__ballot_sync(0xffffffffu, end > goal)) - 1;
    u64 run = __shfl_sync(0xffffffffu, end - m, g), seen = __shfl_sync(0xffffffffu, n_before, g);
    for (int c = g * per; c < min((g + 1) * per, chunks); ++c) {
      const int v = share.v0 + c * 32 + lane;
      Vec<T> x(make_uint4(0, 0, 0, 0));
      if (v < share.v1) x = share.get(v);
      // the lane's masses, and its tokens at the cut
      u64 w[VE];
      m = n = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const bool at = ties > 0 && v < share.v1 && x.v[i] == cut;
        const bool in = v < share.v1 && x.v[i] > cut && x.v[i] >= grid.low;
        w[i] = in ? grid.weight(x.v[i]) : 0;
        n += at;
        m += w[i];
      }
      const u64 n_scan = warp_scan(n), n_from = seen + n_scan - n;  // ties before this lane's
      m += (n_from < ties ? min(n, ties - n_from) : 0) * cut_weight;
      const u64 m_scan = warp_scan(m);
      u64 at = run + m_scan - m, rank_of = n_from;
      const bool mine = at <= goal && goal < at + m;
      if (mine) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if (ties > 0 && x.v[i] == cut && rank_of++ < ties) w[i] = cut_weight;
          if (at <= goal && goal < at + w[i]) {
            p.tokens[r] = v * VE + i - share.before;
            if (p.probs) p.probs[r] = (float)((double)w[i] / (double)total);
          }
          at += w[i];
        }
      }
      if (__any_sync(0xffffffffu, mine)) break;
      run += __shfl_sync(0xffffffffu, m_scan, 31);
      seen += __shfl_sync(0xffffffffu, n_scan, 31);
    }
  }
  cluster_sync();  // no block leaves while its sums are read
}

// Bytes of a row's share in shared memory: two blocks on an SM up to the first;
// the second is what 8 blocks need of the longest rows (2^18 fp32).
constexpr int kShareTwo = 76 * 1024, kShareMost = 136 * 1024;
static_assert(2 * (kShareTwo + sizeof(Shared) + 1024) <= 228 * 1024, "two blocks");
static_assert(((1 << 18) * 4 / 16 + 8 * kWarps) / (8 * kWarps) * kWarps * 16 <= kShareMost, "fits");

template <typename T>
cudaError_t launch_t(const SampleParams &p, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const int vecs = (p.vocab + 2 * VE - 2) / VE;  // wherever the row starts
  int blocks = 1;
  auto share = [&] { return (vecs + blocks * kWarps - 1) / (blocks * kWarps); };
  auto bytes = [&] { return share() * kWarps * 16; };
  while (blocks < kMostBlocks && (bytes() > kShareTwo ||
                        ((long long)p.rows * blocks * 2 <= kSms && bytes() > 8 * 1024)))
    blocks *= 2;
  // above what needs no leave; always the most, since the attribute is the process's
  if (bytes() > 12 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShareMost);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl_cluster(blocks, sample_kernel<T>, dim3((unsigned)p.rows * blocks),
                            dim3(kThreads), bytes(), stream, p, blocks, share());
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
  SampleParams p{};
  p.logits = a.logits; p.stride = a.stride;
  p.temperature = a.temperature; p.top_k = a.top_k; p.top_p = a.top_p; p.min_p = a.min_p;
  p.uniform = a.uniform; p.tokens = a.tokens; p.probs = a.probs;
  p.rows = a.rows; p.vocab = a.vocab;
  return a.bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace gdn
