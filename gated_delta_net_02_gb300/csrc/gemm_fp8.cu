// gemm_fp8.cu -- product of two e4m3 matrices with fp32 scales: one for each
// row and 128 columns of A, one for each 128 x 128 block of B.
//
//   out[m][n] = sum_b sa[m][b] sb[n/128][b] sum_{k in block b} A[m][k] B[n][k]
//
// The scales change every 128 elements of k, so a block's product (four
// tcgen05 instructions of K = 32, fp32 accumulators in tensor memory) is
// taken to registers and added there as acc += (sa sb) * product: one load
// from tensor memory and one fused multiply-add for every 128 products of
// the tensor cores. Two tensor-memory buffers let the tensor cores form one
// block while the epilogue warps take the other.
//
// Roles of a block of threads: one thread issues TMA loads into a ring of
// 128-byte-swizzled stages (one scale block of k each), one warp the
// tensor-core instructions, and the epilogue warps keep the fp32 sums of the
// whole k in registers; scales reach them a group of stages at a time.
//
// Three forms, by the sizes (figures: one GB300, bf16 output):
//  * up to 64 rows of A: the rows of B are the instruction's 128 rows and the
//    rows of A its 16 to 64 columns, so that no tensor-core row idles. Bound
//    by the read of B: k is split over a cluster of up to 8 blocks, which add
//    their sums through distributed shared memory in rank order. 64 x 2560 x
//    2048 6.0 us, 16 x 8192 x 4096 7.4 us (4.6 TB/s).
//  * at most one 128 x 128 tile for each SM: rows of A as the instruction's
//    rows (a row's scale is then a lane's own, not a read for each column);
//    split and joined alike. 256 x 4096 x 4096 10.2 us, 512 x 4096 x 4096
//    13.4 us (17.7 us as 256 x 256 tiles).
//  * more: 256 x 256 tiles of a pair of blocks (cta_group::2), persistent.
//    8192 x 8192 x 4096 196 us (2800 TFLOP/s), 1024 x 4096 x 4096 17.7 us. It
//    should be bound by the tensor cores: its instructions alone take 123 us,
//    with the stages' loads and barriers 163. Two tensor-memory buffers are
//    all there is, and a block's product cannot start before the buffer of
//    two blocks ago has been read in both blocks of the pair, which takes
//    about as long again as the product.
#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.cuh"
#include "tensor_map.h"

namespace gdn {
namespace {

constexpr int kBlockK = 128;      // k of a stage, of a scale and of a swizzle row
constexpr int kScaleGroup = 8;    // stages whose scales share one barrier

struct GemmParams {
  const float *a_scale, *b_scale;
  void *out;
  int M, N, KB;  // KB = blocks of k
  int split;     // blocks of a cluster along k (few rows)
  int bf16_out;
  int *err;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return pack_bf16(lo, hi); }

// Four consecutive outputs of one row; `full` when all four exist and the
// address allows one store.
__device__ __forceinline__ void store_out4(const GemmParams &p, long long at, float4 v, int n_left,
                                           bool vec) {
  if (p.bf16_out) {
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at;
    if (vec && n_left >= 4) {
      *reinterpret_cast<uint2 *>(o) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
    } else {
      if (n_left > 0) o[0] = __float2bfloat16_rn(v.x);
      if (n_left > 1) o[1] = __float2bfloat16_rn(v.y);
      if (n_left > 2) o[2] = __float2bfloat16_rn(v.z);
      if (n_left > 3) o[3] = __float2bfloat16_rn(v.w);
    }
  } else {
    float *o = static_cast<float *>(p.out) + at;
    if (vec && n_left >= 4) {
      *reinterpret_cast<float4 *>(o) = v;
    } else {
      if (n_left > 0) o[0] = v.x;
      if (n_left > 1) o[1] = v.y;
      if (n_left > 2) o[2] = v.z;
      if (n_left > 3) o[3] = v.w;
    }
  }
}

// acc += v * f for two neighbours in one instruction (each rounds alone).
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float f, float g) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mov.b64 w, {%4, %5};\n\tfma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(f), "f"(g));
}
// acc[at ..] += v f for 32 loaded columns. The empty statement keeps each use
// behind the wait that stands before it.
__device__ __forceinline__ void add_part(float (&acc)[128], float (&v)[32], float f, int at) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    asm volatile("" : "+f"(v[j]), "+f"(v[j + 1]));
    fma2(acc[at + j], acc[at + j + 1], v[j], v[j + 1], f, f);
  }
}

struct Bars {
  uint64_t sfull[2], sempty[2];  // two groups of scale vectors
  uint64_t tfull[4], tempty[4];  // tensor-memory buffers
};

// The scales of a lane's row of A and of a block of B, four stages at a time
// and the next four under way. (Brought by a warp of their own through shared
// memory they cost each stage a barrier, and a wait some 150 cycles.)
struct RowScales {
  const float *a, *b;  // NULL a: no such row
  int n;               // stages
  float next_a[4], next_b[4], cur[4];
  __device__ __forceinline__ void fetch(int i0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = i0 + u < n && a;
      next_a[u] = in ? a[i0 + u] : 0.f;
      next_b[u] = in ? b[i0 + u] : 0.f;
    }
  }
  // Scales of stages i0 .. i0 + 3 into cur.
  __device__ __forceinline__ void advance(int i0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) cur[u] = next_a[u] * next_b[u];
    fetch(i0 + 4);
  }
};

// ---- few rows of A, and few tiles -----------------------------------------------

// TOKENS: the instruction's 128 rows are rows of A, its NT = 128 columns rows
// of B; otherwise the other way round, with NT rows of A.
template <int NT, bool TOKENS>
struct SmallCfg {
  static_assert(!TOKENS || NT == 128, "square tiles");
  static constexpr int A_BYTES = 128 * kBlockK;  // the instruction's rows
  static constexpr int STAGE = A_BYTES + NT * kBlockK;
  static constexpr int STAGES = NT <= 32 ? 5 : 4;
  static constexpr int GROUPS = NT >= 64 ? 2 : 1;  // of four epilogue warps, each on its columns
  static constexpr int COLS = NT / GROUPS;
  static constexpr int THREADS = 128 + 128 * GROUPS;
  static constexpr int BUFS = 4, TCOLS = BUFS * NT;  // tensor-memory buffers
  // The square tiles take all columns: 8 KB that nothing uses keep a block of
  // any other form off their SM (see tmem_never_waits_crosswise).
  static constexpr int SMEM = STAGES * STAGE + 1024 + (TOKENS ? 8 * 1024 : 0);
  // The sums on their way out: [NT][128], or [128][NT + 4] so that a lane's
  // 16-byte stores of its own row and the reads along rows meet no conflict.
  static constexpr int PITCH = TOKENS ? NT + 4 : 128;
  static_assert(4 * PITCH * (TOKENS ? 128 : NT) <= STAGES * STAGE, "the sums reuse the stages");
};

template <int NT, bool TOKENS>
__global__ void __launch_bounds__(SmallCfg<NT, TOKENS>::THREADS)
    gemm_small_kernel(const GemmParams p,
                                                         const __grid_constant__ CUtensorMap mb,
                                                         const __grid_constant__ CUtensorMap ma) {
  using C = SmallCfg<NT, TOKENS>;
  constexpr int S = C::STAGES, NB = C::BUFS, SG = kScaleGroup;
  extern __shared__ unsigned char raw[];
  unsigned char *sm =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[S], empty[S];
  __shared__ Bars bars;
  __shared__ __align__(16) float sc[2][TOKENS ? 1 : SG][NT];
  __shared__ uint32_t tm_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * 128, m0 = blockIdx.y * NT;
  const int kb0 = (int)((long long)rank * p.KB / p.split);
  const int nk = (int)((long long)(rank + 1) * p.KB / p.split) - kb0;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.sfull[i], 32);
      mbar_init(&bars.sempty[i], 4 * C::GROUPS);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&bars.tfull[i], 1);
      mbar_init(&bars.tempty[i], 4 * C::GROUPS);
    }
    fence_mbar_init();
    prefetch_tmap(&mb);
    prefetch_tmap(&ma);
  }
  // Tensor memory only once the kernel before has completed, and the next
  // kernel only once this one has its own: of two kernels of one stream on one
  // SM that both allocate, the earlier never waits for the later. Of kernels of
  // different streams see tmem_never_waits_crosswise.
  // The first tiles of B start for the L2 while the kernel before still runs:
  // a hint, which changes nothing if that kernel writes them.
  if (tid == 0)
    for (int i = 0; i < min(nk, S); ++i) tma_prefetch_2d(&mb, (kb0 + i) * kBlockK, n0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 2) {
    tmem_alloc(&tm_s, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = tm_s;

  float acc[C::COLS];
  const int col0 = warp < 4 ? 0 : (warp - 4) / 4 * C::COLS;  // the epilogue warp's columns
  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < nk; ++i) {
        const int s = i % S;
        if (i >= S && !mbar_wait(&empty[s], (i / S - 1) & 1, p.err, kSiteGemmEmpty)) break;
        unsigned char *st = sm + s * C::STAGE;
        mbar_arrive_expect_tx(&full[s], C::STAGE);
        tma_load_2d(TOKENS ? st + C::A_BYTES : st, &mb, (kb0 + i) * kBlockK, n0, &full[s]);
        tma_load_2d(TOKENS ? st : st + C::A_BYTES, &ma, (kb0 + i) * kBlockK, m0, &full[s]);
      }
      for (int j = max(i - S, 0); j < i; ++j) mbar_drain(&full[j % S], (j / S) & 1);
    }
  } else if (warp == 1) {
    int i = 0;
    for (; i < nk; ++i) {
      const int s = i % S, b = i % NB;
      // a buffer never used yet counts as the phase before the first: given back
      const bool ok = mbar_wait_both(&bars.tempty[b], (i / NB + 1) & 1, &full[s], (i / S) & 1,
                                     p.err, kSiteGemmStage);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t st = smem_u32(sm) + s * C::STAGE;
      umma_e4m3_k128(tm + b * NT, sdesc_kmajor(st), sdesc_kmajor(st + C::A_BYTES),
                     idesc_e4m3_f32(128, NT), smem_u32(&empty[s]), smem_u32(&bars.tfull[b]));
    }
    if (i > 0) mbar_drain(&empty[(i - 1) % S], ((i - 1) / S) & 1);
  } else if (warp == 2 && !TOKENS) {
    // Scales of the tile's rows of A times that of its block of B, a group of
    // stages at a time; the next group's loads are under way while this one
    // waits for its place.
    constexpr int PER = (NT + 31) / 32;
    const float *bs = p.b_scale + (long long)(n0 >> 7) * p.KB + kb0;
    float v[SG][PER], next[SG][PER];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < SG; ++u)
#pragma unroll
        for (int c = 0; c < PER; ++c) {
          const int j = c * 32 + lane;
          next[u][c] = 0.f;
          if (i0 + u < nk && j < NT && m0 + j < p.M)
            next[u][c] = p.a_scale[(long long)(m0 + j) * p.KB + kb0 + i0 + u] * bs[i0 + u];
        }
    };
    fetch(0);
    for (int g = 0; g * SG < nk; ++g) {
#pragma unroll
      for (int u = 0; u < SG; ++u)
#pragma unroll
        for (int c = 0; c < PER; ++c) v[u][c] = next[u][c];
      fetch((g + 1) * SG);
      const int s = g & 1;
      if (g >= 2 && !mbar_wait(&bars.sempty[s], (g / 2 - 1) & 1, p.err, kSiteGemmScale)) break;
#pragma unroll
      for (int u = 0; u < SG; ++u)
#pragma unroll
        for (int c = 0; c < PER; ++c)
          if (c * 32 + lane < NT) sc[s][u][c * 32 + lane] = v[u][c];
      mbar_arrive(&bars.sfull[s]);
    }
  } else if (warp >= 4) {
#pragma unroll
    for (int j = 0; j < C::COLS; ++j) acc[j] = 0.f;
    const uint32_t src = tm + ((uint32_t)((warp & 3) * 32) << 16) + col0;
    RowScales rs;
    if (TOKENS) {
      const int m = m0 + (warp & 3) * 32 + lane;
      rs.a = m < p.M ? p.a_scale + (long long)m * p.KB + kb0 : nullptr;
      rs.b = p.b_scale + (long long)(n0 >> 7) * p.KB + kb0;
      rs.n = nk;
      rs.fetch(0);
    }
    bool ok = true;
    for (int i0 = 0; i0 < nk && ok; i0 += 4) {
      if (TOKENS) rs.advance(i0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u, b = i % NB, g = i / SG;
        if (i >= nk) break;
        if (!TOKENS && i % SG == 0)
          ok = mbar_wait(&bars.sfull[g & 1], (g / 2) & 1, p.err, kSiteGemmScale);
        ok = ok && mbar_wait(&bars.tfull[b], (i / NB) & 1, p.err, kSiteGemmAcc);
        if (!ok) break;
        tc_fence_after();
        float v[C::COLS];
        if constexpr (C::COLS == 16) {
          tmem_ld16(src + b * NT, v);
        } else {
#pragma unroll
          for (int c = 0; c < C::COLS; c += 32) tmem_ld32_async(src + b * NT + c, v + c);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.tempty[b]);
        float4 f;
        if (TOKENS) f.x = f.y = f.z = f.w = rs.cur[u];
#pragma unroll
        for (int j = 0; j < C::COLS; j += 4) {
          if (!TOKENS) f = *reinterpret_cast<const float4 *>(&sc[g & 1][TOKENS ? 0 : i % SG][col0 + j]);
          asm volatile("" : "+f"(v[j]), "+f"(v[j + 1]), "+f"(v[j + 2]), "+f"(v[j + 3]));
          fma2(acc[j], acc[j + 1], v[j], v[j + 1], f.x, f.y);
          fma2(acc[j + 2], acc[j + 3], v[j + 2], v[j + 3], f.z, f.w);
        }
        if (!TOKENS && (i % SG == SG - 1 || i == nk - 1)) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sempty[g & 1]);
        }
      }
    }
  }
  __syncthreads();  // every stage has been read by the tensor cores
  float *sums = reinterpret_cast<float *>(sm);
  if (warp >= 4) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < C::COLS; j += TOKENS ? 4 : 1) {
      if (TOKENS)
        *reinterpret_cast<float4 *>(sums + row * C::PITCH + col0 + j) =
            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      else
        sums[(col0 + j) * C::PITCH + row] = acc[j];
    }
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  const int mine = NT / p.split;  // rows of A that this block finishes, 128 columns each
  const bool vec = (p.N & 3) == 0;
  for (int e = tid; e < mine * 32; e += C::THREADS) {
    const int j = rank * mine + (e >> 5), r = (e & 31) * 4;
    const float *at = sums + j * C::PITCH + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < p.split; ++c) {
      const float4 t = p.split > 1 ? ld_cluster_f4(smem_u32(at), c)
                                   : *reinterpret_cast<const float4 *>(at);
      v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
    }
    if (m0 + j < p.M && n0 + r < p.N)
      store_out4(p, (long long)(m0 + j) * p.N + n0 + r, v, p.N - n0 - r, vec);
  }
  if (p.split > 1) cluster_sync();  // no block leaves while its sums are read
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tm, C::TCOLS);
}

// ---- many rows of A --------------------------------------------------------------

// A pair of blocks on one 256 x 256 tile: each holds 128 rows of A and 128 of
// B a stage (half of what a block alone would load for the same products) and
// the sums of its own 128 rows.
struct LargeCfg {
  static constexpr int TM = 256, TN = 256;
  static constexpr int HALF = 128 * kBlockK, STAGE = 2 * HALF;
  static constexpr int STAGES = 4, BOXES = 2;
  static constexpr int BOX = 32 * 128;  // output box of a warp: 32 rows of 128 bytes
  static_assert(32 * 33 * 4 <= BOXES * BOX, "32 rows of 32 sums and a pad");
  static constexpr int SMEM = STAGES * STAGE + 8 * BOXES * BOX + 1024;
  static constexpr int THREADS = 384;  // four warps of roles, eight of epilogue
  static constexpr int TCOLS = 512;
};

// Kernels of different streams that hold tensor memory while they wait for
// other blocks of their cluster. A block waits in its allocation, without a
// limit, until the columns are free; were two such kernels to share SMs that
// lack columns for both, each could hold the columns that a block of the
// other's cluster waits for. So of any two forms, either their blocks do not
// fit one SM together (228 KB, 1 KB of it reserved for each block; static
// shared memory is left out, which errs towards fitting) or their columns do.
// Three blocks of any forms do not fit. The attention and the chunk kernels
// allocate too, but none of them waits for another block while it holds what a
// block of these could wait for: chunk_prep's and the attention's blocks end by
// themselves, and a chunk scan fills an SM alone.
constexpr int kSmSmem = 228 * 1024, kBlockReserve = 1024, kTmemCols = 512;
template <class A, class B>
constexpr bool tmem_never_waits_crosswise() {
  return A::SMEM + B::SMEM + 2 * kBlockReserve > kSmSmem || A::TCOLS + B::TCOLS <= kTmemCols;
}
template <class A, class... Rest>
constexpr bool tmem_all_pairs() {
  if constexpr (sizeof...(Rest) == 0) {
    return tmem_never_waits_crosswise<A, A>();
  } else {
    return tmem_never_waits_crosswise<A, A>() && (tmem_never_waits_crosswise<A, Rest>() && ...) &&
           tmem_all_pairs<Rest...>();
  }
}
static_assert(tmem_all_pairs<SmallCfg<16, false>, SmallCfg<32, false>, SmallCfg<64, false>,
                             SmallCfg<128, true>, LargeCfg>(),
              "two kernels' clusters could wait for each other's tensor memory");
static_assert(3 * (SmallCfg<16, false>::SMEM + kBlockReserve) > kSmSmem, "three blocks on an SM");

// The warp's 32 rows x 128 columns of acc, lane = row, in boxes of 128 bytes.
template <bool BF16>
__device__ __forceinline__ void store_boxes(unsigned char *box, int lane, const CUtensorMap &mo,
                                            int n0, int m0, const float (&acc)[128]) {
  constexpr int COLS = BF16 ? 64 : 32;
#pragma unroll
  for (int i = 0; i < 128 / COLS; ++i) {
    unsigned char *at = box + i % LargeCfg::BOXES * LargeCfg::BOX;
    if (i % LargeCfg::BOXES == 0) {  // the boxes' last contents have left
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = BF16 ? pack2(acc[i * 64 + c * 8 + 2 * k], acc[i * 64 + c * 8 + 2 * k + 1])
                    : __float_as_uint(acc[i * 32 + c * 4 + k]);
      *reinterpret_cast<uint4 *>(at + lane * 128 + ((c ^ (lane & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&mo, n0 + i * COLS, m0, at);
      bulk_commit();
    }
  }
}

// The same for rows that do not start on 16 bytes: transposed through shared
// memory 32 columns at a time, so that a store's lanes write one run of a row.
__device__ __forceinline__ void store_rows(const GemmParams &p, float *buf, int lane, int n0,
                                           int m0, const float (&acc)[128]) {
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += 32) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 32; ++c) buf[lane * 33 + c] = acc[c0 + c];
    __syncwarp();
    const int n = n0 + c0 + lane;
    if (n >= p.N) continue;
    const int rows = min(32, p.M - m0);
    long long at = (long long)m0 * p.N + n;
#pragma unroll 4
    for (int r = 0; r < rows; ++r, at += p.N) {
      const float v = buf[r * 33 + lane];
      if (p.bf16_out) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
      else static_cast<float *>(p.out)[at] = v;
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LargeCfg::THREADS, 1)
    gemm_large_kernel(const GemmParams p, const __grid_constant__ CUtensorMap ma,
                      const __grid_constant__ CUtensorMap mb,
                      const __grid_constant__ CUtensorMap mo, int m_tiles, int n_tiles,
                      bool boxes) {
  using C = LargeCfg;
  constexpr int S = C::STAGES, SG = kScaleGroup;
  extern __shared__ unsigned char raw[];
  unsigned char *sm =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[S], empty[S];  // full and tempty: those of rank 0 serve the pair
  __shared__ Bars bars;
  __shared__ float sc[2][SG][130];  // a stage's 128 rows of A, then the two blocks of B
  __shared__ uint32_t tm_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.sfull[i], 32);
      mbar_init(&bars.sempty[i], 8);
      mbar_init(&bars.tfull[i], 1);
      mbar_init(&bars.tempty[i], 16);
    }
    fence_mbar_init();
    prefetch_tmap(&mb);
    prefetch_tmap(&ma);
  }
  // Tensor memory as in gemm_small_kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  if (warp == 2) tmem_alloc_pair(&tm_s, C::TCOLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers stand
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = tm_s;
  const int tiles = m_tiles * n_tiles;

  // registers: 384 x 168 at launch = 128 x 72 + 256 x 216
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0) {
        int i = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          const int m0 = t % m_tiles * C::TM + rank * 128, n0 = t / m_tiles * C::TN + rank * 128;
          for (int kb = 0; kb < p.KB; ++kb, ++i) {
            const int s = i % S;
            if (i >= S && !mbar_wait(&empty[s], (i / S - 1) & 1, p.err, kSiteGemmEmpty)) {
              ok = false;
              break;
            }
            unsigned char *st = sm + s * C::STAGE;
            const uint32_t bar = cluster_addr(&full[s], 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE);
            tma_load_2d_pair(st, &ma, kb * kBlockK, m0, bar);
            tma_load_2d_pair(st + C::HALF, &mb, kb * kBlockK, n0, bar);
          }
        }
        // a stage's barrier counts the copies of both blocks, and neither leaves
        // before the other
        if (rank == 0)
          for (int j = max(i - S, 0); j < i; ++j) mbar_drain(&full[j % S], (j / S) & 1);
      }
    } else if (warp == 1) {
      if (rank == 0) {
        int i = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs)
          for (int kb = 0; kb < p.KB; ++kb, ++i) {
            const int s = i % S, b = i & 1;
            ok = mbar_wait_both(&bars.tempty[b], ((i >> 1) + 1) & 1, &full[s], (i / S) & 1, p.err,
                                kSiteGemmStage);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = smem_u32(sm) + s * C::STAGE;
            umma_e4m3_k128_pair(tm + b * C::TN, sdesc_kmajor(st), sdesc_kmajor(st + C::HALF),
                                idesc_e4m3_f32(C::TM, C::TN), smem_u32(&empty[s]),
                                smem_u32(&bars.tfull[b]));
          }
        if (i > 0) mbar_drain(&empty[(i - 1) % S], ((i - 1) / S) & 1);
      }
    } else if (warp == 2) {
      // scales of the block's rows of A and of the tile's two blocks of B, a
      // group of stages at a time (registers are short for the epilogue warps
      // to load them, which is how the square tiles have it)
      int g = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const int m0 = t % m_tiles * C::TM + rank * 128, nb = (t / m_tiles * C::TN >> 7) + lane;
        for (int k0 = 0; k0 < p.KB; k0 += SG, ++g) {
          const int s = g & 1;
          if (g >= 2 && !mbar_wait(&bars.sempty[s], (g / 2 - 1) & 1, p.err, kSiteGemmScale)) {
            ok = false;
            break;
          }
          for (int u0 = 0; u0 < SG; u0 += 4) {
            float v[4][5];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int kb = k0 + u0 + u;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int m = m0 + c * 32 + lane;
                v[u][c] = kb < p.KB && m < p.M ? p.a_scale[(long long)m * p.KB + kb] : 0.f;
              }
              v[u][4] = kb < p.KB && lane < 2 && nb * 128 < p.N
                            ? p.b_scale[(long long)nb * p.KB + kb]
                            : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
              for (int c = 0; c < 4; ++c) sc[s][u0 + u][c * 32 + lane] = v[u][c];
              if (lane < 2) sc[s][u0 + u][128 + lane] = v[u][4];
            }
          }
          mbar_arrive(&bars.sfull[s]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t taddr = tm + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
    unsigned char *box = sm + S * C::STAGE + (warp - 4) * C::BOXES * C::BOX;
    const uint32_t freed[2] = {cluster_addr(&bars.tempty[0], 0), cluster_addr(&bars.tempty[1], 0)};
    int i = 0, g = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      for (int k0 = 0; k0 < p.KB && ok; k0 += SG, ++g) {
        const int s = g & 1;
        ok = mbar_wait(&bars.sfull[s], (g / 2) & 1, p.err, kSiteGemmScale);
        for (int u = 0; u < SG && k0 + u < p.KB; ++u, ++i) {
          const int b = i & 1;
          ok = ok && mbar_wait(&bars.tfull[b], (i >> 1) & 1, p.err, kSiteGemmAcc);
          if (!ok) break;
          const float f = sc[s][u][row] * sc[s][u][128 + half];
          tc_fence_after();
          // Columns in four parts, two in registers at a time: the third and
          // fourth are under way while the first two are added, and the buffer
          // is given back before the last two are.
          const uint32_t src = taddr + b * C::TN;
          float v0[32], v1[32];
          tmem_ld32_async(src, v0);
          tmem_ld32_async(src + 32, v1);
          tmem_wait_ld();
          add_part(acc, v0, f, 0);
          tmem_ld32_async(src + 64, v0);
          add_part(acc, v1, f, 32);
          tmem_ld32_async(src + 96, v1);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(b ? freed[1] : freed[0]);
          add_part(acc, v0, f, 64);
          add_part(acc, v1, f, 96);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sempty[s]);
      }
      if (!ok) break;
      const int m0 = t % m_tiles * C::TM + rank * 128 + (warp & 3) * 32;
      const int n0 = t / m_tiles * C::TN + half * 128;
      if (boxes) {
        // through shared memory in swizzled boxes of 32 rows x 128 bytes, which
        // bulk copies take to the output while the next tile begins (stores
        // from registers, 32 rows at a time, took a sixth of the whole call)
        if (p.bf16_out) store_boxes<true>(box, lane, mo, n0, m0, acc);
        else store_boxes<false>(box, lane, mo, n0, m0, acc);
      } else {
        store_rows(p, reinterpret_cast<float *>(box), lane, n0, m0, acc);
      }
    }
    if (boxes && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the pair arrives in a block that has left
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tm, C::TCOLS);
}

// ---- host side ------------------------------------------------------------------

// e4m3 [rows][K], boxes of 128 bytes x box_rows, 128-byte swizzle; what lies
// beyond the matrix reads as zeros.
bool map_e4m3(CUtensorMap *m, const void *base, int rows, int K, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {kBlockK, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [M][N], boxes of 128 bytes x 32 rows, 128-byte swizzle; rows must
// start on 16 bytes. What a box has beyond the matrix is not written.
bool map_out(CUtensorMap *m, void *out, int M, int N, bool bf16) {
  const cuuint64_t e = bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M}, strides[1] = {N * e};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / e), 32}, es[2] = {1, 1};
  return encode_fn()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                     2, out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 152;

template <int NT, bool TOKENS>
cudaError_t launch_small(const GemmArgs &a, GemmParams p, cudaStream_t stream) {
  using C = SmallCfg<NT, TOKENS>;
  CUtensorMap ma, mb;
  if (!map_e4m3(&ma, a.a, a.M, a.K, NT) || !map_e4m3(&mb, a.b, a.N, a.K, 128))
    return cudaErrorInvalidValue;
  const int nt = (a.N + 127) / 128, mt = (a.M + NT - 1) / NT;
  // As many blocks of k as keep the grid within the GPU, two stages each at
  // least. Clusters of 8 only while 12 of them cover the tiles: more do not all
  // find eight free SMs of one processing cluster (64 x 2048 x 4096, 16 tiles:
  // 6.7 us split in 4, 11.4 in 8; 16 x 1024 x 8192, 8 tiles: 7.0 and 5.3).
  p.split = 1;
  const long long tiles = (long long)nt * mt;
  while (p.split < (tiles <= 12 ? 8 : 4) && tiles * p.split * 2 <= kSms && p.KB >= 4 * p.split)
    p.split *= 2;
  auto kernel = gemm_small_kernel<NT, TOKENS>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(p.split, kernel, dim3(nt * p.split, mt), dim3(C::THREADS), C::SMEM,
                            stream, p, mb, ma);
}

cudaError_t launch_large(const GemmArgs &a, const GemmParams &p, cudaStream_t stream) {
  using C = LargeCfg;
  CUtensorMap ma, mb, mo{};
  const bool boxes = a.N % (a.bf16_out ? 8 : 4) == 0;
  if (!map_e4m3(&ma, a.a, a.M, a.K, 128) || !map_e4m3(&mb, a.b, a.N, a.K, 128) ||
      (boxes && !map_out(&mo, a.out, a.M, a.N, a.bf16_out)))
    return cudaErrorInvalidValue;
  const int mt = (a.M + C::TM - 1) / C::TM, nt = (a.N + C::TN - 1) / C::TN;
  cudaError_t e = cudaFuncSetAttribute(gemm_large_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)mt * nt;
  return launch_pdl(gemm_large_kernel, dim3(2 * (tiles < kSms / 2 ? (unsigned)tiles : kSms / 2)),
                    dim3(C::THREADS), C::SMEM, stream, p, ma, mb, mo, mt, nt,
                    boxes);
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmArgs &a, cudaStream_t stream) {
  if (!encode_fn()) return cudaErrorNotSupported;
  GemmParams p{};
  p.a_scale = a.a_scale; p.b_scale = a.b_scale; p.out = a.out;
  p.M = a.M; p.N = a.N; p.KB = (a.K + kBlockK - 1) / kBlockK;
  p.bf16_out = a.bf16_out; p.err = a.err; p.split = 1;
  if (a.M <= 16) return launch_small<16, false>(a, p, stream);
  if (a.M <= 32) return launch_small<32, false>(a, p, stream);
  if (a.M <= 64) return launch_small<64, false>(a, p, stream);
  const long long tiles = (long long)((a.M + 127) / 128) * ((a.N + 127) / 128);
  if (tiles <= kSms) return launch_small<128, true>(a, p, stream);
  return launch_large(a, p, stream);
}

}  // namespace gdn
