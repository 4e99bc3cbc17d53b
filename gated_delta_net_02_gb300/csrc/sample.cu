// sample.cu -- one token for each row of logits: temperature, top-k, top-p and
// min-p, from a given random number.
//
//   w_i = exp((x_i - max x) / temperature)
//   kept = the first n of the descending order (equal logits: lower index first)
//   token = first kept index, by index, whose running mass passes u * mass
//
// Bound by HBM: a row is read once; a cluster of up to 8 blocks holds it in
// shared memory and makes all further passes there.
//  * Masses decide between tokens by whole numbers: a weight is an integer in
//    units of 2^-44 of the largest (an error of about one unit of 2^-40, of
//    fp32 pairs and a table of 2^(-i/256)), so a sum has the same value in any
//    order, and with it the token. Tokens below 2^-45 of the largest have
//    mass 0.
//  * The order is never made. The last kept value is found by histograms:
//    16 bins an octave of weight first, then the bin's values by their ordered
//    bits, 1024 bins at a time, until a bin is one value. Of the tokens with
//    that value the lowest indexes are kept.
//  * The top-p mass needs weights of the whole row. The first histogram adds 12
//    bits of each (32-bit atomics), which bounds the masses well enough to leave
//    some neighbouring bins; their masses and all before them are then added
//    exactly.
#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.cuh"

namespace gdn {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;          // of a histogram; two of each thread
constexpr int kSms = 152;
constexpr int kOne = 44;             // log2 of the largest weight
constexpr float kOctaves = 45.f;     // weights below 2^-45 are 0
constexpr int kGroups = 32;          // pieces of a warp's share with a mass of their own

struct SampleParams {
  const void *logits;
  long long stride;
  const float *temperature, *top_p, *min_p, *uniform;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  int rows, vocab;
};

// 2^(40 - i / 256), rounded.
struct PowTable {
  u64 v[256];
  constexpr PowTable() : v() {
    for (int i = 0; i < 256; ++i) {
      const double x = -0.69314718055994530942 * i / 256;
      double term = 1, sum = 1;
      for (int n = 1; n < 30; ++n) {
        term *= x / n;
        sum += term;
      }
      v[i] = (u64)(sum * 1099511627776.0 + 0.5);
    }
  }
};
__device__ constexpr PowTable kPow{};

// A float's bits in the order of the values, +0 and -0 the same (canon()).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu));
}
// NaN counts as -inf, -0 as +0.
__device__ __forceinline__ float canon(float x) { return x == x ? x + 0.f : -INFINITY; }

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

// Weights of a row. y = log2(1 / weight), as the sum of two floats.
struct Scale {
  float top, c_hi, c_lo;  // log2(e) / temperature
  // the high part of y: the same for equal logits, and never smaller for a
  // smaller one
  __device__ __forceinline__ float y_of(float x) const {
    if (top == INFINITY) return x == top ? 0.f : INFINITY;
    return (top - x) * c_hi;
  }
  // The weight, y < kOctaves being its high part.
  __device__ __forceinline__ u64 weight(float x, float y, const u64 *table) const {
    float lo = 0.f;
    if (top != INFINITY) {
      const float s = top - x;  // and what s is short of top - x (Knuth's two-sum)
      const float b = s - top;
      const float e = (top - (s - b)) + (-x - b);
      lo = fmaf(s, c_hi, -y) + fmaf(s, c_lo, e * c_hi);
    }
    // y = i / 256 + r, 0 <= r < 1 / 256
    const float t = __fadd_rd(y * 256.f, 8388608.f);
    const int i = __float_as_int(t) & 0x7fffff;
    const float r = fmaf(t - 8388608.f, -1.f / 256, y);
    // 1 - 2^-(r + lo) = z + (rest): z = r ln 2 with its error
    const float ln2 = 0.693147182464599609375f, ln2_lo = -1.904654299957767e-9f;
    const float z = r * ln2;
    const float rr = r + lo;
    const float q = rr * rr * (0.24022651f - rr * (0.055504109f - rr * 0.0096181291f));
    const float rest = fmaf(r, ln2, -z) + fmaf(r, ln2_lo, fmaf(lo, ln2, -q));
    const uint32_t u = (uint32_t)(int)__float2uint_rn(z * 1099511627776.f) +
                       (uint32_t)__float2int_rn(rest * 1099511627776.f);
    const u64 p = table[i & 255];
    const uint32_t p32 = p >> 40 ? 0xffffffffu : (uint32_t)(p >> 8);
    const int n = i >> 8;
    // r + lo below 0 is a weight just above the table's (|lo| ln 2 < 1e-5)
    const u64 w = z < 1e-4f && (int)u < 0 ? p + __umulhi(p32, 0u - u) : p - __umulhi(p32, u);
    return ((w << 4) + ((1ull << n) >> 1)) >> n;
  }
};

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
  u64 table[256];
  u64 mass[2][kBins];      // two histograms in turn, so that one is cleared
  uint32_t count[2][kBins];  // while the other is read by the cluster
  u64 part[2];             // this block's sums of two passes
  u64 warp_part[kWarps], warp_part2[kWarps];
  u64 seg_mass[kWarps][kGroups];
  uint32_t seg_ties[kWarps][kGroups];
  u64 warp_mass[kWarps];
  uint32_t warp_ties[kWarps];
  float top;
  float warp_top[kWarps];
  int found[4];
  u64 found64[4];
};

// A row's share of one block, and the passes over it.
template <typename T>
struct Share {
  static constexpr int VE = 16 / (int)sizeof(T);
  const T *row;      // the row's first 16-byte boundary at or below its start
  int before, cols;  // elements before the row's start, and after it begins
  int v0, v1;        // this warp's vectors, counted from `row`
  uint4 *own;        // this warp's place in shared memory

  __device__ __forceinline__ Vec<T> fetch(int v) const {
    const T *p = row + (long long)v * VE;
    const int e0 = v * VE - before;  // index of the first element
    if (e0 >= 0 && e0 + VE <= cols) {
      Vec<T> x(__ldg(reinterpret_cast<const uint4 *>(p)));
#pragma unroll
      for (int i = 0; i < VE; ++i) x.v[i] = canon(x.v[i]);
      return x;
    }
    Vec<T> x(make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int i = 0; i < VE; ++i)
      x.v[i] = e0 + i >= 0 && e0 + i < cols ? canon(to_f32(p[i])) : -INFINITY;
    return x;
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
};

// Sum of `mine` over the block's threads into part[i], for the cluster to read
// behind its next barrier.
__device__ __forceinline__ void block_part(Shared &sh, int i, u64 mine) {
  mine = warp_sum(mine);
  if ((threadIdx.x & 31) == 0) sh.warp_part[threadIdx.x >> 5] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    u64 sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += sh.warp_part[w];
    sh.part[i] = sum;
  }
}

// Block-wide inclusive scan of two numbers of each thread: the sums before the
// thread's own in *a and *b.
__device__ __forceinline__ void block_scan(Shared &sh, u64 &a, u64 &b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 sa = warp_scan(a), sb = warp_scan(b);
  __syncthreads();
  if (lane == 31) {
    sh.warp_part[warp] = sa;
    sh.warp_part2[warp] = sb;
  }
  __syncthreads();
  u64 ba = 0, bb = 0;
  for (int w = 0; w < warp; ++w) {
    ba += sh.warp_part[w];
    bb += sh.warp_part2[w];
  }
  a = ba + sa - a;
  b = bb + sb - b;
}

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
  for (int i = tid; i < kBins; i += kThreads) {
    sh.mass[0][i] = sh.mass[1][i] = 0;
    sh.count[0][i] = sh.count[1][i] = 0;
  }
  if (tid < 256) sh.table[tid] = kPow.v[tid];
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
  }
  const float temperature = p.temperature ? p.temperature[r] : 1.f;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float u = p.uniform[r];

  // ---- the row arrives; its maximum
  float top = -INFINITY;
#pragma unroll 4
  for (int v = share.v0 + lane; v < share.v1; v += 32) {
    const Vec<T> x = share.fetch(v);
#pragma unroll
    for (int i = 0; i < VE; ++i) top = fmaxf(top, x.v[i]);
    share.own[v - share.v0] = x.pack();
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh.warp_top[w]);
    sh.top = top;
  }
  cluster_sync();
  for (int k = 0; k < blocks; ++k) {
    const float other = __uint_as_float(ld_cluster_u32(&sh.top, k));
    top = k == 0 ? other : fmaxf(top, other);
  }
  if (top == -INFINITY) {  // nothing to choose from
    if (rank == 0 && tid == 0) {
      p.tokens[r] = -1;
      if (p.probs) p.probs[r] = 0.f;
    }
    cluster_sync();
    return;
  }
  Scale sc;
  {
    sc.top = top;
    const double c = temperature > 0.f ? fmin(1.4426950408889634074 / (double)temperature, 1e30) : 0.;
    sc.c_hi = (float)c;
    sc.c_lo = (float)(c - (double)sc.c_hi);
  }

  // What is kept: keys above `cut`, and the first `ties` tokens at it.
  uint32_t cut = 0;
  u64 ties = 0;
  int buf = 0;  // histogram in use
  // A pass's barrier. Whoever is behind it has read the histogram before,
  // which is cleared for the pass after (block_scan's barriers come between).
  auto pass_done = [&] {
    cluster_sync();
    for (int i = tid; i < kBins; i += kThreads) {
      sh.mass[buf ^ 1][i] = 0;
      sh.count[buf ^ 1][i] = 0;
    }
  };
  auto bin_of = [&](float y) {  // 16 an octave
    return (__float_as_int(__fadd_rd(y * 16.f, 8388608.f)) & 0x7fffff);
  };
  // A key range that holds every value of bins b0 .. b1, by a margin.
  auto range_of = [&](int b0, int b1, uint32_t &khi, uint32_t &klo) {
    if (sc.top == INFINITY || sc.c_hi == 0.f) {
      khi = key_of(top);
      klo = sc.top == INFINITY ? khi : 0;
    } else {
      const float near = b0 / 16.f / sc.c_hi, far = (b1 + 1) / 16.f / sc.c_hi;
      const float margin = 1e-5f * (fabsf(top) + far);
      const float hi = top - near + margin, lo = top - far - margin;
      khi = min(key_of(canon(hi)), key_of(top));
      klo = lo > -INFINITY ? key_of(canon(lo)) : 0;
    }
    khi >>= kLow;
    klo >>= kLow;
  };
  auto merged = [&](int i, u64 &count, u64 &mass) {
    count = mass = 0;
    for (int k = 0; k < blocks; ++k) {
      count += ld_cluster_u32(&sh.count[buf][i], k);
      mass += ld_cluster_u64(&sh.mass[buf][i], k);
    }
  };
  // The value at which the order's running count (BY_MASS: mass) first reaches
  // `want`, among the values above key `above` whose first bin is b0 .. b1;
  // `have` = what comes before those bins. Result in cut (its key); have then
  // is what comes before that value, and *there the tokens with it.
  auto refine = [&](bool by_mass, u64 want, uint32_t above, int b0, int b1, u64 have, u64 &there) {
    uint32_t khi, klo;
    range_of(b0, b1, khi, klo);
    for (;;) {
      int shift = 0;
      while ((khi - klo) >> shift >= (uint32_t)kBins) ++shift;
      share.each([&](float x) {
        const float y = sc.y_of(x);
        const uint32_t key = key_of(x), k = key >> kLow;
        if (!(y < kOctaves) || key <= above || k > khi || k < klo) return;
        const int b = bin_of(y);
        if (b < b0 || b > b1) return;
        const int i = (int)((khi - k) >> shift);
        atomicAdd(&sh.count[buf][i], 1u);
        if (by_mass) atomicAdd(&sh.mass[buf][i], sc.weight(x, y, sh.table));
      });
      pass_done();
      u64 n[2], m[2];
      merged(2 * tid, n[0], m[0]);
      merged(2 * tid + 1, n[1], m[1]);
      u64 nb = n[0] + n[1], mb = m[0] + m[1];
      block_scan(sh, nb, mb);
      u64 at = have + (by_mass ? mb : nb);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u64 step = by_mass ? m[j] : n[j];
        if (at < want && want <= at + step) {
          sh.found[0] = 2 * tid + j;
          sh.found64[0] = at;
          sh.found64[1] = n[j];
        }
        at += step;
      }
      __syncthreads();
      const int i = sh.found[0];
      have = sh.found64[0];
      there = sh.found64[1];
      __syncthreads();
      buf ^= 1;
      const uint32_t first = khi - ((uint32_t)i << shift);
      if (shift == 0) {
        cut = first << kLow;
        if constexpr (kLow > 0) cut |= (int)cut < 0 ? 0u : 0xffffu;
        return have;
      }
      const uint32_t span = (1u << shift) - 1;
      klo = first - klo > span ? first - span : klo;
      khi = first;
    }
  };

  const bool greedy = !(temperature > 0.f) || min_p > 1.f;
  if (greedy) {
    cut = key_of(top);
    ties = 1;
  } else {
    if (top_k > 0 && top_k < p.vocab) {
      share.each([&](float x) {
        const float y = sc.y_of(x);
        if (y < kOctaves) atomicAdd(&sh.count[buf][bin_of(y)], 1u);
      });
      pass_done();
      u64 n[2], m[2], none = 0;
      merged(2 * tid, n[0], m[0]);
      merged(2 * tid + 1, n[1], m[1]);
      u64 before = n[0] + n[1];
      if (tid == 0) sh.found[0] = -1;
      block_scan(sh, before, none);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (before < (u64)top_k && (u64)top_k <= before + n[j]) {
          sh.found[0] = 2 * tid + j;
          sh.found64[0] = before;
        }
        before += n[j];
      }
      __syncthreads();
      const int b = sh.found[0];
      const u64 have = sh.found64[0];
      __syncthreads();
      buf ^= 1;
      if (b >= 0) {  // else fewer tokens than top_k have any mass
        u64 there;
        ties = (u64)top_k - refine(false, (u64)top_k, 0, b, b, have, there);
      }
    }
    if (top_p < 1.f) {
      const uint32_t above = cut;
      u64 sum = 0;
      share.each([&](float x) {
        const float y = sc.y_of(x);
        if (!(y < kOctaves) || key_of(x) <= above) return;
        const u64 w = sc.weight(x, y, sh.table);
        sum += w;
        const int b = bin_of(y);
        // 12 bits below the octave's largest
        atomicAdd(reinterpret_cast<uint32_t *>(&sh.mass[buf][b]), (uint32_t)(w >> 1 << (b >> 4) >> 31));
        atomicAdd(&sh.count[buf][b], 1u);
      });
      block_part(sh, 0, sum);
      pass_done();
      u64 total = 0;
      for (int k = 0; k < blocks; ++k) total += ld_cluster_u64(&sh.part[0], k);
      u64 tie_weight = 0;
      if (ties > 0) {
        const float x = of_key(cut);
        tie_weight = sc.weight(x, sc.y_of(x), sh.table);
      }
      const double goal = ceil((double)top_p * (double)(total + ties * tie_weight));
      const u64 want = goal < 1. ? 1 : (u64)goal;
      // the running mass of a bin's end, from below and above
      u64 n[2], m[2], lo[2], hi[2];
      merged(2 * tid, n[0], m[0]);
      merged(2 * tid + 1, n[1], m[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int octave = (2 * tid + j) >> 4;
        const u64 at_least = (m[j] << 32) >> octave, at_most = ((m[j] + n[j]) << 32) >> octave;
        lo[j] = at_least > n[j] ? at_least - n[j] : 0;
        hi[j] = n[j] ? at_most + n[j] + 1 : 0;
      }
      u64 before_lo = lo[0] + lo[1], before_hi = hi[0] + hi[1];
      if (tid == 0) {
        sh.found[0] = kBins - 1;
        sh.found[1] = kBins - 1;
      }
      block_scan(sh, before_lo, before_hi);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (before_hi < want && want <= before_hi + hi[j]) sh.found[0] = 2 * tid + j;
        if (before_lo < want && want <= before_lo + lo[j]) sh.found[1] = 2 * tid + j;
        before_hi += hi[j];
        before_lo += lo[j];
      }
      __syncthreads();
      const int b0 = sh.found[0], b1 = sh.found[1];
      __syncthreads();
      buf ^= 1;
      if (want > total) {  // among the last of the top k
        ties = tie_weight ? min(ties, (want - total + tie_weight - 1) / tie_weight) : ties;
      } else {
        // what comes before the bins, exactly
        sum = 0;
        share.each([&](float x) {
          const float y = sc.y_of(x);
          if (y < kOctaves && key_of(x) > above && bin_of(y) < b0) sum += sc.weight(x, y, sh.table);
        });
        block_part(sh, 1, sum);
        cluster_sync();
        u64 have = 0, there;
        for (int k = 0; k < blocks; ++k) have += ld_cluster_u64(&sh.part[1], k);
        have = refine(true, want, above, b0, b1, have, there);
        const float x = of_key(cut);
        const u64 w = sc.weight(x, sc.y_of(x), sh.table);
        ties = w ? min(there, (want - have + w - 1) / w) : there;
      }
    }
    if (min_p > 0.f && sc.top != INFINITY) {
      // the smallest logit that is not below the bound
      const float x = __double2float_ru((double)top + (double)temperature * log((double)min_p));
      uint32_t k = min(key_of(canon(x)), key_of(top));
      if (k > cut) {  // all of that value: what is below it goes
        cut = k - 1;
        ties = 0;
      }
    }
  }

  // ---- the masses of the warps' shares, piece by piece
  const int chunks = (warp_vecs + 31) / 32, per = (chunks + kGroups - 1) / kGroups;
  u64 cut_weight = 0;
  if (ties > 0) {
    const float x = of_key(cut);
    const float y = sc.y_of(x);
    if (greedy) cut_weight = 1ull << kOne;
    else if (y < kOctaves) cut_weight = sc.weight(x, y, sh.table);
  }
  auto mass_of = [&](const Vec<T> &x, bool live, u64 &mass, uint32_t &at_cut) {
    mass = 0;
    at_cut = 0;
    if (!live) return;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const uint32_t key = key_of(x.v[i]);
      at_cut += ties > 0 && key == cut;
      if (key <= cut) continue;
      const float y = sc.y_of(x.v[i]);
      if (y < kOctaves) mass += sc.weight(x.v[i], y, sh.table);
    }
  };
  u64 warp_total = 0;
  uint32_t warp_at_cut = 0;
  for (int g = 0; g < kGroups; ++g) {
    u64 mass = 0;
    uint32_t n = 0;
    for (int c = g * per; c < min((g + 1) * per, chunks); ++c) {
      const int v = share.v0 + c * 32 + lane;
      const bool live = v < share.v1;
      u64 m;
      uint32_t at;
      mass_of(share.get(live ? v : share.v0), live, m, at);
      mass += m;
      n += at;
    }
    if (g * per < chunks) {
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
  // every warp scans all warps' masses, 32 at a time
  u64 run = 0, total = 0, seen = 0;
  u64 my_before = 0, my_mass = 0, my_seen = 0;
  for (int w0 = 0; w0 < blocks * kWarps; w0 += 32) {
    const int w = w0 + lane;
    u64 m = 0, n = 0;
    if (w < blocks * kWarps) {
      m = ld_cluster_u64(&sh.warp_mass[w % kWarps], w / kWarps);
      n = ld_cluster_u32(&sh.warp_ties[w % kWarps], w / kWarps);
    }
    const u64 n_scan = warp_scan(n), n_before = seen + n_scan - n;
    const u64 kept = n_before < ties ? min(n, ties - n_before) : 0;
    m += kept * cut_weight;
    const u64 m_scan = warp_scan(m);
    const int me = rank * kWarps + warp - w0;
    if (me >= 0 && me < 32) {
      my_before = __shfl_sync(0xffffffffu, run + m_scan - m, me);
      my_mass = __shfl_sync(0xffffffffu, m, me);
      my_seen = __shfl_sync(0xffffffffu, n_before, me);
    }
    run += __shfl_sync(0xffffffffu, m_scan, 31);
    seen += __shfl_sync(0xffffffffu, n_scan, 31);
  }
  total = run;
  // the first token whose running mass is above u * total
  u64 goal = 0;
  if (u > 0.f) {
    const double x = (double)u * (double)total;
    goal = x < (double)total ? (u64)x : total - 1;
    if (goal >= total) goal = total - 1;
  }
  if (my_before <= goal && goal < my_before + my_mass) {
    // the piece, then its vectors in order
    u64 m = sh.seg_mass[warp][lane], n = sh.seg_ties[warp][lane];
    const u64 n_before = my_seen + warp_scan(n) - n;
    m += (n_before < ties ? min(n, ties - n_before) : 0) * cut_weight;
    const u64 end = my_before + warp_scan(m);
    const int g = __ffs(__ballot_sync(0xffffffffu, end > goal)) - 1;
    run = __shfl_sync(0xffffffffu, end - m, g);
    seen = __shfl_sync(0xffffffffu, n_before, g);
    for (int c = g * per; c < min((g + 1) * per, chunks); ++c) {
      const int v = share.v0 + c * 32 + lane;
      const bool live = v < share.v1;
      const Vec<T> x = share.get(live ? v : share.v0);
      uint32_t at;
      mass_of(x, live, m, at);
      const u64 at_scan = warp_scan((u64)at);
      u64 rank_of = seen + at_scan - at;  // ties before this lane's
      m += (rank_of < ties ? min((u64)at, ties - rank_of) : 0) * cut_weight;
      const u64 m_scan = warp_scan(m);
      const bool mine = run + m_scan - m <= goal && goal < run + m_scan;
      if (mine) {
        u64 at_mass = run + m_scan - m;
        for (int i = 0; i < VE; ++i) {
          const uint32_t key = key_of(x.v[i]);
          u64 w = 0;
          if (key > cut) {
            const float y = sc.y_of(x.v[i]);
            if (y < kOctaves) w = sc.weight(x.v[i], y, sh.table);
          } else if (ties > 0 && key == cut && rank_of++ < ties) {
            w = cut_weight;
          }
          if (at_mass <= goal && goal < at_mass + w) {
            p.tokens[r] = v * VE + i - share.before;
            if (p.probs) p.probs[r] = (float)((double)w / (double)total);
          }
          at_mass += w;
        }
      }
      if (__any_sync(0xffffffffu, mine)) break;
      run += __shfl_sync(0xffffffffu, m_scan, 31);
      seen += __shfl_sync(0xffffffffu, at_scan, 31);
    }
  }
  cluster_sync();  // no block leaves while its sums are read
}

// Bytes of a row's share in shared memory: two blocks on an SM up to the first;
// the second is what 8 blocks need of the longest rows (2^18 fp32).
constexpr int kShareTwo = 72 * 1024, kShareMost = 136 * 1024;
static_assert(((1 << 18) * 4 / 16 + 8 * kWarps) / (8 * kWarps) * kWarps * 16 <= kShareMost, "fits");

template <typename T>
cudaError_t launch_t(const SampleParams &p, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(T);
  const int vecs = (p.vocab + 2 * VE - 2) / VE;  // wherever the row starts
  int blocks = 1;
  auto share = [&] { return (vecs + blocks * kWarps - 1) / (blocks * kWarps); };
  auto bytes = [&] { return share() * kWarps * 16; };
  while (blocks < 8 && (bytes() > kShareTwo ||
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
