// attention.cuh -- attention of the last T tokens of each sequence over a paged
// key-value cache, split over the cache's length and joined; the T tokens in a
// line (paged_attention.cu) or as the nodes of a tree (tree_attention.cu).
//
//   out[t] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_t . k_j - m),
//   j = 0 .. len - T + t
//
// One pass over the keys with a running maximum m and sum l (fp32). Bound by
// HBM: a key and its value are read once for the G = H / H_kv query heads of
// their kv head and for the T tokens, 4 G T D flops for 2 D elements.
//
//  * Rows: the T x G (token, query head) pairs of a kv head are the rows of
//    one matrix product, in blocks of up to 128, so that the cache is read
//    once for all of them.
//  * Work: an item is one (sequence, kv head, row block); its keys are cut
//    into tiles. All items' tiles form one line, and each block of the grid
//    takes an equal run of it, whatever the lengths (every block reads the
//    lengths and finds its place by a scan). An item that one block holds
//    whole is finished there; of a cut item each block writes its (m, l,
//    sum p v) to the workspace and a second kernel joins them, in the fixed
//    order of the line.
//  * bf16: products on the warp-level matrix instruction (m16n8k16), or with
//    many rows on tcgen05 (below). p is rounded to bf16 for the second product
//    (the sum l takes the unrounded p): up to 2^-8 of each term, as the inputs
//    are. fp32: fp32 products on the CUDA cores, in blocks of 4 to 32 rows.
//  * Keys reach shared memory by 16-byte asynchronous copies, several tiles
//    ahead; each key's address comes from its page, looked up a tile earlier.
//    Rows beyond the length are filled with zeros, so what an unused part of
//    a page holds (NaN included) reaches no result.
//
// Measured on one GB300 (us; the cache's bytes at the copy rate in brackets):
// 64 sequences of 512 to 8192 tokens, 16 heads on 2 of 128, bf16, one token
// 53.0 (42.2), of 2048 to 32768 173 (169); 8 x 8 tokens over 30k to 65k keys,
// heads of 256, 137 (115); one sequence of 513 tokens 5.9 (in a page table
// that ends with it; 10.2 in a wide one, see short_split), of 60000 22.8 (9.1).
// Some 10 us of a long call are no transfer: the launches, the chain of
// lengths, page table and first keys, and the join (4 us of the 52.6).
#pragma once

#include <cuda_bf16.h>
#include <limits.h>

#include "kernels.h"
#include "layer.cuh"
#include "tensor_map.h"

namespace gdn {
namespace {

constexpr int kMinTiles = 2;  // shortest run of tiles worth a block of its own

struct AttnParams {
  const void *q, *k, *v;
  void *out;
  const int32_t *table, *lens;
  const int32_t *n_nodes;            // trees: [n_seqs] or NULL (T each)
  const unsigned long long *tree;    // trees: [n_seqs][T]
  float *part_o;    // [2 grid][rows][D] unnormalised sums of cut items
  float2 *part_ml;  // [2 grid][rows]
  int4 *cut;        // [joins] x = item (-1: none), y = its first piece, z = its tiles
                    // beyond that block's, w = tiles of a block
  int joins;        // items, listed by item, or the grid, by block: the fewer
  bool by_item;
  long long page_stride, token_stride, head_stride;
  FastDiv page_size, G, row_blocks;
  int n_seqs, T, H, H_kv, n_pages, max_pages, grouped;
  float scale_log2;  // scale * log2(e)
  int *err;
};

// 2^x, 0 below the normal numbers: no probability that small reaches a sum.
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  const int n = live ? 16 : 0;  // 0 source bytes: filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// Tile geometry. bf16: WM warps along the rows, 16 rows each; the other warps
// share out the tile's keys. fp32: four warps along the rows, WM rows each; the
// other warps share out the keys, and a warp's lanes a key's columns.
template <typename T, int D_, int WM_>
struct Cfg {
  using In = T;
  static constexpr bool kTensorMemory = false;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int D = D_, WM = WM_;
  static constexpr int ROWS = kBf16 ? 16 * WM : 4 * WM;
  // Two warps for each of an SM's schedulers: two blocks of four, or one of
  // eight where the tiles leave room for one block only and a warp has at
  // least 16 keys of its own. fp32: eight from heads of 128 or 32 rows on (us,
  // eight and four: 16 sequences of 5000, 4 rows of 256, 137 and 168; of 10000,
  // 4 rows of 128 125 and 128, of 64 71.5 and 73, but 16 rows of 64 133 and 119).
  static constexpr int WARPS = (kBf16 ? D == 256 && WM > 1 : D > 64 || WM > 4) ? 8 : 4;
  static constexpr int THREADS = 32 * WARPS;
  // fp32 from 16 rows on: warps of 8 rows (TileF32Wide)
  static constexpr bool kWide = !kBf16 && ROWS >= 16;
  static constexpr int WK = WARPS / (kBf16 ? WM : kWide ? ROWS / 8 : 4);  // key groups with their own m, l and sum
  static constexpr int KT = kBf16 ? 64 : 32;     // keys of a tile
  static constexpr int ROW_BYTES = D * (int)sizeof(T);
  static constexpr int CH = ROW_BYTES / 16;      // 16-byte chunks of a row
  static constexpr int TILE = KT * ROW_BYTES;    // K or V
  static constexpr int STAGES = 3;
  static constexpr int Q_BYTES = ROWS * ROW_BYTES;
  static constexpr int P_PITCH = KT + (kWide ? 4 : 0);
  static constexpr int P_BYTES = kBf16 ? 0 : ROWS * P_PITCH * 4;
  // q fragments stay in registers up to D = 128: q then only passes through
  // the last stage's place before that stage is first used
  static constexpr bool QREG = kBf16 && D <= 128;
  static constexpr int SMEM = STAGES * 2 * TILE + (QREG ? 0 : Q_BYTES) + P_BYTES;
  // blocks of an SM: what its shared memory holds, up to four of them
  static constexpr int FIT = 224 * 1024 / (SMEM + 4 * 1024);
  static constexpr int MOST = kWide && WARPS == 8 ? 2 : 4;  // 128 registers a thread
  static constexpr int PER_SM = FIT > MOST ? MOST : FIT < 1 ? 1 : FIT;
  static_assert(!QREG || Q_BYTES <= 2 * TILE, "q fits a stage");
  static_assert(WK * ROWS * D * 4 <= STAGES * 2 * TILE, "the join reuses the tiles");
};

// Chunk c of row r: rows are at least 128 bytes, and eight consecutive rows
// place one chunk in eight different bank groups.
template <class C>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return (uint32_t)(row * C::ROW_BYTES + ((c ^ (row & 7)) << 4));
}

constexpr long long kMaxLen = 1LL << 30;  // key indexes of a few tiles beyond it still fit

__device__ __forceinline__ int seq_len(const AttnParams &p, int s, bool report) {
  const int len = p.lens[s];
  const long long most = min((long long)p.max_pages * p.page_size.d, kMaxLen);
  if (len > most) {
    if (report) set_error(p.err, kDevBadPage);
    return (int)most;
  }
  return len < 0 ? 0 : len;
}

// Tiles of one item of a sequence: at least one, so that an empty sequence
// still has its zeros written.
__device__ __forceinline__ int item_tiles(int len, int kt) {
  return len <= 0 ? 1 : (len - 1) / kt + 1;
}

struct Place {
  int seq, len;     // sequence of the block's first tile
  long long first;  // line position of that sequence's first tile
};

// Quotient of line positions, in 32 bits where they fit (a 64-bit division
// costs some hundred instructions at the head of every block).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Block-wide: finds where line position begin(total) lies. Each thread sums
// a run of sequences; the thread whose run holds the position walks it.
// False when the position is beyond the line.
template <int THREADS, class F>
__device__ bool find_place(const AttnParams &p, int kt, int items_per_seq, F begin,
                           long long (&warp_sum)[THREADS / 32], Place &found) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n_seqs + THREADS - 1) / THREADS;
  const int s0 = min(tid * per, p.n_seqs), s1 = min(s0 + per, p.n_seqs);
  long long sum = 0;
  int len = 0;
  for (int s = s0; s < s1; ++s) {
    len = seq_len(p, s, blockIdx.x == 0);
    sum += (long long)item_tiles(len, kt) * items_per_seq;
  }
  long long scan = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += up;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  before += scan - sum;
  const long long x = begin(total);
  if (x >= before && x < before + sum) {
    long long at = before;
    for (int s = s0; s < s1; ++s) {
      if (per > 1) len = seq_len(p, s, false);
      const long long n = (long long)item_tiles(len, kt) * items_per_seq;
      if (x < at + n) {
        found = Place{s, len, at};
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return x < total;
}

// ---- trees -------------------------------------------------------------------
// A row's keys are those below its limit; a node of a tree also sees the nodes
// of its word, which stand in the cache from the limit on.
template <bool TREE>
__device__ __forceinline__ bool sees(int key, int lim, unsigned long long word) {
  if (key < lim) return true;
  if constexpr (!TREE) return false;
  const unsigned j = (unsigned)(key - lim);
  return j < 64 && (word >> j & 1);
}

// Nodes of a sequence's tree.
__device__ __forceinline__ int seq_nodes(const AttnParams &p, int s, bool report) {
  if (!p.n_nodes) return p.T;
  const int n = p.n_nodes[s];
  if (report && (n < 0 || n > p.T)) set_error(p.err, kDevBadTree);
  return min(max(n, 0), p.T);
}

// The word of node t, without what is no node.
__device__ __forceinline__ unsigned long long node_word(const AttnParams &p, int s, int t,
                                                        int nodes) {
  if (t >= nodes) return 0;
  const unsigned long long w = p.tree[(long long)s * p.T + t];
  return nodes < 64 ? w & ((1ull << nodes) - 1) : w;
}

// Mark of an output row whose node is not there: it takes part like any other,
// unmasked, and becomes 0 at the end.
constexpr long long kAbsent = 1LL << 62;

// ---- one tile on the matrix instruction (bf16) -------------------------------

template <class C, bool TREE>
struct TileBf16 {
  static constexpr int D = C::D, KW = C::KT / C::WK;  // keys of a warp
  static constexpr bool QREG = C::QREG;
  float o[D / 8][4];
  float m[2], l[2];
  uint32_t qf[QREG ? D / 16 : 1][4];
  uint32_t q_addr;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
  __device__ __forceinline__ void start(uint32_t q_s) {
    const int lane = threadIdx.x & 31, wm = (threadIdx.x >> 5) % C::WM;
    const int row = wm * 16 + (lane & 15);
    clear();
    q_addr = q_s;
    if constexpr (QREG) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        ldsm4(qf[ks], q_s + chunk_at<C>(row, ks * 2 + (lane >> 4)));
    }
  }

  // Keys key0 .. of the tile; `lim` = keys the lane's two rows see.
  __device__ __forceinline__ void tile(uint32_t k_s, uint32_t v_s, int key0, const int (&lim)[2],
                                       const unsigned long long (&word)[2], float scale_log2,
                                       float *) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kbase = warp / C::WM * KW;
    const int qrow = warp % C::WM * 16 + (lane & 15);
    float s[KW / 8][4];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      if constexpr (QREG) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = qf[ks][i];
      } else {
        ldsm4(a, q_addr + chunk_at<C>(qrow, ks * 2 + (lane >> 4)));
      }
      // a step's fragments are all under way before its first product
      uint32_t b[KW / 16][4];
#pragma unroll
      for (int n = 0; n < KW / 16; ++n)
        ldsm4(b[n], k_s + chunk_at<C>(kbase + n * 16 + krow, ks * 2 + kch));
#pragma unroll
      for (int n = 0; n < KW / 16; ++n) {
        mma16816(s[2 * n], a, b[n][0], b[n][1]);
        mma16816(s[2 * n + 1], a, b[n][2], b[n][3]);
      }
    }
    // scaled scores, masked beyond each row's last key; running maximum
    const int col = key0 + kbase + (lane & 3) * 2;
    const bool cut = key0 + C::KT > min(lim[0], lim[1]);
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[i][e] * scale_log2;
        if (cut && !sees<TREE>(col + i * 8 + (e & 1), lim[e >> 1], word[e >> 1])) x = -INFINITY;
        s[i][e] = x;
        mx[e >> 1] = fmaxf(mx[e >> 1], x);
      }
    float ref[2], alpha[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      const float mn = fmaxf(m[r], mx[r]);
      ref[r] = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every p is 0
      alpha[r] = exp2_ftz(m[r] - ref[r]);
      m[r] = mn;
      l[r] *= alpha[r];
    }
    // the sums are only touched when some row's maximum has moved
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
    }
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = exp2_ftz(s[i][e] - ref[e >> 1]);
        l[e >> 1] += s[i][e];
      }
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;
#pragma unroll
    for (int n = 0; n < KW / 16; ++n) {
      const uint32_t a[4] = {bf16x2(s[2 * n][0], s[2 * n][1]), bf16x2(s[2 * n][2], s[2 * n][3]),
                             bf16x2(s[2 * n + 1][0], s[2 * n + 1][1]),
                             bf16x2(s[2 * n + 1][2], s[2 * n + 1][3])};
#pragma unroll
      for (int d0 = 0; d0 < D / 16; d0 += 4) {
        uint32_t b[4][4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
          ldsm4_t(b[d], v_s + chunk_at<C>(kbase + n * 16 + vrow, (d0 + d) * 2 + vch));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          mma16816(o[2 * (d0 + d)], a, b[d][0], b[d][1]);
          mma16816(o[2 * (d0 + d) + 1], a, b[d][2], b[d][3]);
        }
      }
    }
  }

  // Row limits of the lane's two rows, as tile() takes them.
  template <class F, class V>
  static __device__ __forceinline__ void limits(F limit_of, V (&lim)[2]) {
    const int lane = threadIdx.x & 31, wm = (threadIdx.x >> 5) % C::WM;
    lim[0] = limit_of(wm * 16 + (lane >> 2));
    lim[1] = limit_of(wm * 16 + (lane >> 2) + 8);
  }

  // Sums to shared memory: so[key group][row][D], sml[key group][row].
  __device__ __forceinline__ void flush(float *so, float2 *sml) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wk = warp / C::WM, wm = warp % C::WM;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float t = l[r];
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      const int row = wk * C::ROWS + wm * 16 + (lane >> 2) + 8 * r;
      if ((lane & 3) == 0) sml[row] = make_float2(m[r], t);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2 *>(so + row * D + i * 8 + (lane & 3) * 2) =
            make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
  }
};

// ---- one tile on the CUDA cores (fp32) -----------------------------------------
// A warp has R rows. Scores: a lane has one key of the 32, and reads its row
// of K in 16-byte chunks (eight lanes, eight bank groups) beside broadcast
// chunks of q. Sums: a lane has D / 32 columns, and reads V rows beside
// broadcast p. Products go two to an instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "mov.b64 w, {%4, %5};\n\tfma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}

template <class C, bool TREE>
struct TileF32 {
  static constexpr int D = C::D, VL = D / 32, R = C::WM;
  static constexpr int KEYS = C::KT / C::WK, PARTS = C::WK;
  static_assert(C::kWide || KEYS * PARTS == 32, "a lane for each key and part of the columns");
  float o[R][VL];
  float m[R], l[R];
  uint32_t q_addr;

  static __device__ __forceinline__ int row_group() { return threadIdx.x >> 5 & 3; }
  static __device__ __forceinline__ int key_group() { return threadIdx.x >> 7; }
  __device__ __forceinline__ void start(uint32_t q_s) {
    q_addr = q_s;
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < VL; ++i) o[r][i] = 0.f;
    }
  }
  static __device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a));
    return v;
  }
  // the lane's columns of a row of V: chunks lane, 32 + lane, or half a chunk
  static __device__ __forceinline__ void lds_v(uint32_t v_s, int row, float (&x)[VL]) {
    const int lane = threadIdx.x & 31;
    if constexpr (VL == 2) {
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                   : "=f"(x[0]), "=f"(x[1])
                   : "r"(v_s + chunk_at<C>(row, lane >> 1) + (lane & 1) * 8));
    } else {
#pragma unroll
      for (int i = 0; i < VL / 4; ++i) {
        const float4 t = lds4(v_s + chunk_at<C>(row, i * 32 + lane));
        x[4 * i] = t.x; x[4 * i + 1] = t.y; x[4 * i + 2] = t.z; x[4 * i + 3] = t.w;
      }
    }
  }
  template <class F, class V>
  static __device__ __forceinline__ void limits(F limit_of, V (&lim)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) lim[r] = limit_of(row_group() * R + r);
  }
  __device__ __forceinline__ void tile(uint32_t k_s, uint32_t v_s, int key0, const int (&lim)[R],
                                       const unsigned long long (&word)[R], float scale_log2,
                                       float *p_s) {
    const int lane = threadIdx.x & 31, row0 = row_group() * R;
    const int key = key_group() * KEYS + lane % KEYS, part = lane / KEYS;
    float s[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = s2[r] = 0.f;
#pragma unroll(R > 4 ? 2 : 4)
    for (int c = part; c < C::CH; c += PARTS) {
      const float4 k = lds4(k_s + chunk_at<C>(key, c));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q = lds4(q_addr + chunk_at<C>(row0 + r, c));
        fma2(s[r], s2[r], q.x, q.y, k.x, k.y);
        fma2(s[r], s2[r], q.z, q.w, k.z, k.w);
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float dot = s[r] + s2[r];
#pragma unroll
      for (int off = 16; off >= KEYS; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      const float x = sees<TREE>(key0 + key, lim[r], word[r]) ? dot * scale_log2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int off = KEYS / 2; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[r], mx), ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2_ftz(m[r] - ref), e = exp2_ftz(x - ref);
      m[r] = mn;
      l[r] = l[r] * alpha + e;  // this lane's keys; summed over the lanes at the end
      if (part == 0) p_s[(row0 + r) * C::KT + key] = e;
#pragma unroll
      for (int i = 0; i < VL; ++i) o[r][i] *= alpha;
    }
    __syncwarp();
#pragma unroll(R > 4 ? 2 : 4)
    for (int jk = 0; jk < KEYS; jk += 2) {
      const int j = key_group() * KEYS + jk;
      float2 pj[R];
#pragma unroll
      for (int r = 0; r < R; ++r)
        pj[r] = *reinterpret_cast<const float2 *>(p_s + (row0 + r) * C::KT + j);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        float x[VL];
        lds_v(v_s, j + jj, x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float e = jj ? pj[r].y : pj[r].x;
#pragma unroll
          for (int i = 0; i < VL; i += 2) fma2(o[r][i], o[r][i + 1], x[i], x[i + 1], e, e);
        }
      }
    }
  }
  __device__ __forceinline__ void flush(float *so, float2 *sml) {
    const int lane = threadIdx.x & 31, row0 = key_group() * C::ROWS + row_group() * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float t = l[r];
#pragma unroll
      for (int off = KEYS / 2; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
      if (lane == 0) sml[row0 + r] = make_float2(m[r], t);
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int col = VL == 2 ? lane * 2 + i : (i / 4) * 128 + lane * 4 + (i & 3);
        so[(row0 + r) * D + col] = o[r][i];
      }
    }
  }
};

// fp32, 16 rows or more. With four rows a warp the shared memory is the
// limit: a read of 512 bytes of K serves 4 x 4 products a lane. Here a warp
// has 8 rows, and a lane the products of all 8 with KL keys over an eighth of
// the columns: 8 parts (lane bits 1 to 3) x 4 key lanes (bits 0 and 4).
// Neighbours read the same q, which lets the hardware take half a warp's
// 16-byte reads at once (with the key lanes in bits 3 and 4 a read of q took
// four turns, not two), and keys 4 apart, which the swizzle places in other
// banks. The parts' sums fold into one row a lane (half of the rows given away
// at each step), so that a row's maximum, exponentials and sum are one lane's
// work and two shuffles. 18 sequences of 357 to 1821 tokens, 40 rows of 256 on
// 8 kv heads 242 us (27 TFLOP/s, of some 80; 323 with four rows a warp), 16
// sequences of 5000, 32 rows of 128 144 us (197). Both loops are unrolled
// whole: 280 us otherwise, each read waited for by two warps a scheduler.
template <class C, bool TREE>
struct TileF32Wide {
  static constexpr int D = C::D, VL = D / 32, R = 8, RG = C::ROWS / R;
  static constexpr int KEYS = C::KT / C::WK, KL = KEYS / 4;
  using Narrow = TileF32<C, TREE>;
  float o[R][VL];
  float m[1], l[1];  // of row part(); l of this lane's keys
  uint32_t q_addr;

  static __device__ __forceinline__ int part() { return threadIdx.x >> 1 & 7; }
  static __device__ __forceinline__ int row_group() { return (threadIdx.x >> 5) % RG; }
  static __device__ __forceinline__ int key_group() { return (threadIdx.x >> 5) / RG; }
  __device__ __forceinline__ void start(uint32_t q_s) {
    q_addr = q_s;
    clear();
  }
  __device__ __forceinline__ void clear() {
    m[0] = -INFINITY;
    l[0] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < VL; ++i) o[r][i] = 0.f;
  }
  template <class F, class V>
  static __device__ __forceinline__ void limits(F limit_of, V (&lim)[1]) {
    lim[0] = limit_of(row_group() * R + part());
  }
  __device__ __forceinline__ void tile(uint32_t k_s, uint32_t v_s, int key0, const int (&lim)[1],
                                       const unsigned long long (&word)[1], float scale_log2,
                                       float *p_s) {
    const int lane = threadIdx.x & 31, part = this->part(), row0 = row_group() * R;
    const int key = key_group() * KEYS + (lane & 1) * 4 + (lane >> 4);
    auto step = [](int j) { return j / 2 * 8 + j % 2 * 2; };  // to the lane's j-th key
    float v[R][KL], v2[R][KL];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < KL; ++j) v[r][j] = v2[r][j] = 0.f;
#pragma unroll
    for (int c0 = 0; c0 < C::CH; c0 += 8) {
      const int c = c0 + part;
      float4 k[KL];
#pragma unroll
      for (int j = 0; j < KL; ++j) k[j] = Narrow::lds4(k_s + chunk_at<C>(key + step(j), c));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q = Narrow::lds4(q_addr + chunk_at<C>(row0 + r, c));
#pragma unroll
        for (int j = 0; j < KL; ++j) {
          fma2(v[r][j], v2[r][j], q.x, q.y, k[j].x, k[j].y);
          fma2(v[r][j], v2[r][j], q.z, q.w, k[j].z, k[j].w);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < KL; ++j) v[r][j] += v2[r][j];
#pragma unroll
    for (int off = 4; off; off >>= 1) {
#pragma unroll
      for (int r = 0; r < off; ++r)
#pragma unroll
        for (int j = 0; j < KL; ++j) {
          const bool up = part & off;
          const float give = up ? v[r][j] : v[r + off][j], keep = up ? v[r + off][j] : v[r][j];
          v[r][j] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * off);
        }
    }
    // now v[0] is row `part`
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      v[0][j] = sees<TREE>(key0 + key + step(j), lim[0], word[0]) ? v[0][j] * scale_log2 : -INFINITY;
      mx = fmaxf(mx, v[0][j]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const float mn = fmaxf(m[0], mx), ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2_ftz(m[0] - ref);
    m[0] = mn;
    l[0] *= alpha;
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      const float e = exp2_ftz(v[0][j] - ref);
      l[0] += e;
      p_s[(row0 + part) * C::P_PITCH + key + step(j)] = e;
    }
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, alpha, 2 * r);
#pragma unroll
        for (int i = 0; i < VL; ++i) o[r][i] *= f;
      }
    }
    __syncwarp();
#pragma unroll
    for (int jk = 0; jk < KEYS; jk += 4) {
      const int j = key_group() * KEYS + jk;
      float4 pj[R];
#pragma unroll
      for (int r = 0; r < R; ++r)
        pj[r] = *reinterpret_cast<const float4 *>(p_s + (row0 + r) * C::P_PITCH + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float x[VL];
        Narrow::lds_v(v_s, j + jj, x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float e = jj == 0 ? pj[r].x : jj == 1 ? pj[r].y : jj == 2 ? pj[r].z : pj[r].w;
#pragma unroll
          for (int i = 0; i < VL; i += 2) fma2(o[r][i], o[r][i + 1], x[i], x[i + 1], e, e);
        }
      }
    }
    __syncwarp();  // p_s is read before the next tile's takes its place
  }
  __device__ __forceinline__ void flush(float *so, float2 *sml) {
    const int lane = threadIdx.x & 31, row0 = key_group() * C::ROWS + row_group() * R;
    float t = l[0];
    t += __shfl_xor_sync(0xffffffffu, t, 1);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if ((lane & 17) == 0) sml[row0 + part()] = make_float2(m[0], t);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int col = VL == 2 ? lane * 2 + i : (i / 4) * 128 + lane * 4 + (i & 3);
        so[(row0 + r) * D + col] = o[r][i];
      }
  }
};

template <class C, bool TREE, bool WIDE>
struct TileF32Of {
  using type = TileF32<C, TREE>;
};
template <class C, bool TREE>
struct TileF32Of<C, TREE, true> {
  using type = TileF32Wide<C, TREE>;
};
template <class C, bool TREE>
struct TileOf {
  using type = typename TileF32Of<C, TREE, C::kWide>::type;
};
template <int D, int WM, bool TREE>
struct TileOf<Cfg<__nv_bfloat16, D, WM>, TREE> {
  using type = TileBf16<Cfg<__nv_bfloat16, D, WM>, TREE>;
};

// Row of q and out (in units of D elements) of row r of an item's block of
// rows, or -1 beyond the item's rows.
__device__ __forceinline__ long long out_row(const AttnParams &p, int s, int kvh, int r) {
  const int G = p.G.d;
  if (r >= p.T * G) return -1;
  const int t = p.G.div(r), g = r - t * G;
  const int h = p.grouped ? kvh * G + g : g * p.H_kv + kvh;
  return ((long long)s * p.T + t) * p.H + h;
}

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
  else
    *reinterpret_cast<float4 *>(p) = v;
}

// The end of an item's tiles in a block: the key groups' sums so[group][row]
// (pitch floats apart) and (m, l) become output rows, or a piece for the join.
template <class C, bool TREE>
__device__ __forceinline__ void finish_item(const AttnParams &p, const float *so, int pitch,
                                            const float2 *sml, const long long *rows, bool whole,
                                            long long slot) {
  using T = typename C::In;
  constexpr int D = C::D, ROWS = C::ROWS, WK = C::WK;
#pragma unroll 1
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += C::THREADS) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < WK; ++w) mm = fmaxf(mm, sml[w * ROWS + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float2 ml = sml[w * ROWS + r];
      const float f = exp2_ftz(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4 *>(so + (w * ROWS + r) * pitch + c);
      ll += f * ml.y;
      sum.x = fmaf(f, v.x, sum.x);
      sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z);
      sum.w = fmaf(f, v.w, sum.w);
    }
    long long row = rows[r];
    if (row < 0) continue;
    if (TREE && (row & kAbsent)) {
      row ^= kAbsent;
      mm = -INFINITY;
      ll = 0.f;
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (whole) {
      // a row without keys has ll = 0 and sum = 0: its output is 0
      const float inv = 1.f / (ll == 0.f ? 1.f : ll);
      store4(static_cast<T *>(p.out) + row * D + c,
             make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    } else {
      *reinterpret_cast<float4 *>(p.part_o + (slot * ROWS + r) * D + c) = sum;
      if (c == 0) p.part_ml[slot * ROWS + r] = make_float2(mm, ll);
    }
  }
}

// What a block holds: tiles of a run of items, walked item by item.
struct Walk {
  long long pos, end, run;
  int s, len, nt, x, tile0, block;
  // The first item of block `block` of `blocks`; false when there is nothing for it.
  template <int KT, int NT>
  __device__ __forceinline__ bool begin(const AttnParams &p, int items_per_seq,
                                        long long (&warp_sum)[NT / 32], Place &place, int block,
                                        int blocks) {
    this->block = block;
    long long total = 0;
    if (!find_place<NT>(
            p, KT, items_per_seq,
            [&](long long n) {
              total = n;
              run = max(quotient(n + blocks - 1, blocks), (long long)kMinTiles);
              return run * block;
            },
            warp_sum, place))
      return false;
    pos = run * block;
    end = min(pos + run, total);
    s = place.seq;
    len = place.len;
    nt = item_tiles(len, KT);
    x = (int)quotient(pos - place.first, nt);  // item of the sequence
    tile0 = (int)(pos - place.first - (long long)x * nt);
    return true;
  }
  // Tiles of the current item in this block.
  __device__ __forceinline__ int tiles() const {
    return (int)min((long long)(nt - tile0), end - pos);
  }
  // Lists whether the current item, which starts here, has to be joined, and
  // from which blocks: by item where items are few, else by block (of a
  // block's items only the last can go on elsewhere).
  __device__ __forceinline__ void list_join(const AttnParams &p, int items_per_seq, int n) const {
    if (p.by_item ? tile0 != 0 : pos + n < end) return;
    const int item = s * items_per_seq + x;
    int4 cut = make_int4(-1, 0, 0, 0);
    if (tile0 == 0 && n < nt)
      cut = make_int4(item, 2 * block + (pos == run * block ? 0 : 1), nt - n,
                      (int)min(run, (long long)INT_MAX));
    p.cut[p.by_item ? item : block] = cut;
  }
  template <int KT>
  __device__ __forceinline__ void next(const AttnParams &p, int items_per_seq, int n) {
    pos += n;
    tile0 = 0;
    if (++x == items_per_seq && pos < end) {
      x = 0;
      len = seq_len(p, ++s, false);
      nt = item_tiles(len, KT);
    }
  }
};

// SHORT: no cache is long enough to be worth the line of tiles. A cluster of
// `split` blocks has one item, its tiles dealt out evenly, and joins it through
// distributed shared memory in rank order: one launch, no workspace.
template <class C, bool SHORT, bool TREE>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM)
    attn_kernel(const AttnParams p, int split) {
  using T = typename C::In;
  using Tile = typename TileOf<C, TREE>::type;
  constexpr int D = C::D, KT = C::KT, ROWS = C::ROWS, WK = C::WK, S = C::STAGES;
  constexpr bool Q_IN_STAGE = C::QREG;
  constexpr int NT = C::THREADS;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long offs[4][KT], rows[ROWS], warp_sum[NT / 32];
  __shared__ Place place;
  // the key groups' (m, l) at the end of an item take the place of its keys' addresses
  static_assert(WK * ROWS * sizeof(float2) <= sizeof(offs), "m and l fit");
  float2 *sml = reinterpret_cast<float2 *>(offs);
  const int tid = threadIdx.x;
  const uint32_t tiles_s = smem_u32(smem);
  const uint32_t q_s = tiles_s + (Q_IN_STAGE ? S - 1 : S) * 2 * C::TILE;
  float *p_s = reinterpret_cast<float *>(smem + S * 2 * C::TILE + C::Q_BYTES);  // fp32 only
  float *so = reinterpret_cast<float *>(smem);
  const int items_per_seq = p.H_kv * p.row_blocks.d;
  const T *kc = static_cast<const T *>(p.k), *vc = static_cast<const T *>(p.v);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Walk w;
  const int rank = SHORT ? (int)(blockIdx.x % split) : 0;
  if constexpr (SHORT) {
    const int item = blockIdx.x / split;
    w.s = item / items_per_seq;
    w.x = item - w.s * items_per_seq;
    w.len = seq_len(p, w.s, w.x == 0 && rank == 0);
    w.nt = item_tiles(w.len, KT);
    w.tile0 = rank * w.nt / split;
    w.pos = 0;
    w.end = (rank + 1) * w.nt / split - w.tile0;  // may be none
  } else if (!w.begin<KT, NT>(p, items_per_seq, warp_sum, place, blockIdx.x, gridDim.x)) {
    if (tid == 0 && !p.by_item) p.cut[blockIdx.x].x = -1;
    return;
  }
  for (int seg = 0; w.pos < w.end || (SHORT && seg == 0); ++seg) {
    const int n = w.tiles(), s = w.s, x = w.x, len = w.len, tile0 = w.tile0;
    const int kvh = p.row_blocks.div(x), r0 = (x - kvh * (int)p.row_blocks.d) * ROWS;
    const int nodes = TREE ? seq_nodes(p, s, x == 0 && tile0 == 0 && tid == 0) : 0;
    const long long head = (long long)kvh * p.head_stride;
    const int32_t *table = p.table + (long long)s * p.max_pages;

    // address of key tid of tile i, for its turn in offs (-1: zeros)
    auto page_of = [&](int i) -> int {
      const int key = (tile0 + i) * KT + tid;
      return tid < KT && i < n && key < len ? table[p.page_size.div(key)] : -1;
    };
    auto put_offs = [&](int i, int page) {
      if (tid >= KT) return;
      const int key = (tile0 + i) * KT + tid;
      long long off = -1;
      if (i < n && key < len) {
        if (page < 0 || page >= p.n_pages) {
          set_error(p.err, kDevBadPage);
        } else {
          const int in_page = key - p.page_size.div(key) * (int)p.page_size.d;
          off = page * p.page_stride + in_page * p.token_stride + head;
        }
      }
      offs[i & 3][tid] = off;
    };
    auto load_tile = [&](int i) {
      if (i < n) {
        const uint32_t st = tiles_s + (uint32_t)(i % S) * 2 * C::TILE;
        constexpr int RSTEP = NT / C::CH;
        const int c = tid % C::CH;
#pragma unroll
        for (int j = 0; j < KT / RSTEP; ++j) {
          const int row = tid / C::CH + j * RSTEP;
          const long long off = offs[i & 3][row];
          const bool live = off >= 0;
          const long long e = (live ? off : 0) + c * (16 / (int)sizeof(T));
          cp_async16(st + chunk_at<C>(row, c), kc + e, live);
          cp_async16(st + C::TILE + chunk_at<C>(row, c), vc + e, live);
        }
      }
      cp_async_commit();
    };

    // the first tiles' pages are looked up together
    int page[S + 1];
#pragma unroll
    for (int i = 0; i <= S; ++i) page[i] = page_of(i);
    for (int r = tid; r < ROWS; r += NT) {
      rows[r] = out_row(p, s, kvh, r0 + r);
      if (TREE && rows[r] >= 0 && p.G.div(r0 + r) >= nodes) rows[r] |= kAbsent;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) put_offs(i, page[i]);
    __syncthreads();
    // q rows of the item (zeros beyond them) join the first tile's copies
#pragma unroll 1
    for (int e = tid; e < ROWS * C::CH; e += NT) {
      const int r = e / C::CH, c = e % C::CH;
      const long long row = rows[r];
      const bool live = row >= 0 && !(TREE && (row & kAbsent));
      cp_async16(q_s + chunk_at<C>(r, c),
                 static_cast<const T *>(p.q) + (live ? row : 0) * D + c * (16 / (int)sizeof(T)),
                 live);
    }
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) load_tile(i);
    int next_page = page[S];

    if (!SHORT && tid == NT - 1) w.list_join(p, items_per_seq, n);

    int lim[sizeof(Tile::m) / sizeof(float)];
    unsigned long long word[sizeof(Tile::m) / sizeof(float)];
    Tile::limits(
        [&](int r) {
          const int row = r0 + r, t = p.G.div(row);
          // rows beyond the item's are not stored: no mask for their sake
          if (row >= p.T * (int)p.G.d) return INT_MAX;
          if (TREE) return t < nodes ? len - nodes : INT_MAX;
          return len - p.T + t + 1;
        },
        lim);
    if constexpr (TREE)
      Tile::limits(
          [&](int r) {
            const int row = r0 + r;
            return row < p.T * (int)p.G.d ? node_word(p, s, p.G.div(row), nodes) : 0ull;
          },
          word);
    Tile acc;
    if (SHORT && n == 0) acc.clear();
    for (int i = 0; i < n; ++i) {
      cp_async_wait<S - 2>();
      __syncthreads();
      if (i == 0) {
        acc.start(q_s);
        if (Q_IN_STAGE) __syncthreads();  // q is in registers before its place is loaded
      }
      load_tile(i + S - 1);
      put_offs(i + S, next_page);
      next_page = page_of(i + S + 1);
      const uint32_t st = tiles_s + (uint32_t)(i % S) * 2 * C::TILE;
      acc.tile(st, st + C::TILE, (tile0 + i) * KT, lim, word, p.scale_log2, p_s);
    }
    cp_async_wait<0>();
    __syncthreads();  // the tiles are free: the key groups' sums take their place
    acc.flush(so, sml);
    __syncthreads();

    if (SHORT && split > 1) {
      // this block's piece of the item, behind its key groups' sums
      float *piece = so + WK * ROWS * D;
      float2 *piece_ml = reinterpret_cast<float2 *>(piece + ROWS * D);
      AttnParams local = p;
      local.part_o = piece;
      local.part_ml = piece_ml;
      finish_item<C, TREE>(local, so, D, sml, rows, false, 0);
      cluster_sync();
#pragma unroll 1
      for (int e = rank * NT + tid; e < ROWS * (D / 4); e += split * NT) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        if (rows[r] < 0) continue;
        const long long row = TREE ? rows[r] & ~kAbsent : rows[r];
        const uint32_t at_ml = smem_u32(piece_ml + r), at = smem_u32(piece + r * D + c);
        float mm = -INFINITY, ll = 0.f;
        for (int k = 0; k < split; ++k) mm = fmaxf(mm, ld_cluster_f2(at_ml, k).x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < split; ++k) {
          const float2 ml = ld_cluster_f2(at_ml, k);
          const float4 v = ld_cluster_f4(at, k);
          const float f = exp2_ftz(ml.x - ref);
          ll += f * ml.y;
          sum.x = fmaf(f, v.x, sum.x);
          sum.y = fmaf(f, v.y, sum.y);
          sum.z = fmaf(f, v.z, sum.z);
          sum.w = fmaf(f, v.w, sum.w);
        }
        const float inv = 1.f / (ll == 0.f ? 1.f : ll);
        store4(static_cast<T *>(p.out) + row * D + c,
               make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
      }
      cluster_sync();  // no block leaves while its piece is read
      return;
    }
    finish_item<C, TREE>(p, so, D, sml, rows, n == w.nt, (long long)blockIdx.x * 2 + (seg > 0));
    if (SHORT) return;
    __syncthreads();  // before the next item's copies reuse the tiles

    w.next<KT>(p, items_per_seq, n);
  }
}

// ---- many rows (bf16): products on tcgen05, sums in tensor memory --------------
//
// From some 33 rows the warp-level instruction leaves each scheduler two warps that
// wait on one another's latencies. Here the 128 rows of the tensor-core
// instruction are COPIES copies of up to 128 / COPIES rows: copy c takes the
// c-th part of a tile's 64 keys, with a reference and sums of its own, as a
// warp's key group does above. So every lane of four warps has one row and
// 64 / COPIES keys, and a row's maximum and sum need no other lane.
//
// Warp 0 loads keys by TMA, a box of a page's tokens and 64 columns at a time,
// into 128-byte-swizzled units of 64 keys (K and V in turn); warps 1-3 bring
// q, and clear what the last page holds beyond the length from the last unit
// of V; warps 4-7 turn scores into probabilities; warp 8 issues: S(i+1) =
// Q K^T while the probabilities of tile i are made, then O += P V. The sums
// stay in tensor memory; they are rescaled only when a row's maximum passes
// its reference by more than 2^8, which keeps every probability below 2^8 and
// the rescaling rare.
template <int D_, int COPIES_>
struct TcCfg {
  using In = __nv_bfloat16;
  static constexpr bool kTensorMemory = true;
  static constexpr int D = D_, COPIES = COPIES_, KT = 64;
  static constexpr int ROWS = 128 / COPIES, WK = COPIES, KC = KT / COPIES;
  static constexpr int THREADS = 288;
  static constexpr int UNIT = KT * D * 2, UNITS = D == 256 ? 4 : 8;
  static constexpr int P_BYTES = 128 * 128, Q_BYTES = 128 * D * 2;
  static constexpr int PITCH = D + 4;  // of the sums on their way out
  static constexpr int SMEM = UNITS * UNIT + P_BYTES + Q_BYTES + 1024;
  static constexpr int OUT_BYTES = 128 * PITCH * 4;
  static constexpr int TCOLS = D + 2 * KT <= 256 ? 256 : 512;  // sums, then two tiles of scores
  static constexpr int PER_SM = 1;
  static_assert(KC % 32 == 0, "a lane reads its keys' scores 32 at a time");
  static_assert(OUT_BYTES <= UNITS * UNIT + P_BYTES + Q_BYTES, "the sums fit");
};

constexpr float kMaxGrowth = 8.f;  // log2 of a probability's bound

template <class C, bool TREE>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM)
    attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, int box) {
  using T = __nv_bfloat16;
  constexpr int D = C::D, KT = C::KT, ROWS = C::ROWS, NT = C::THREADS, U = C::UNITS, KC = C::KC;
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  extern __shared__ unsigned char raw[];
  unsigned char *sm =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[U], empty[U], s_full[2], s_empty[2];
  __shared__ uint64_t p_full, o_done, q_full, landed, patched;
  __shared__ long long rows[ROWS], warp_sum[NT / 32];
  __shared__ Place place;
  __shared__ float2 sml[128];
  __shared__ uint32_t tm_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t units_s = smem_u32(sm), p_s = units_s + U * C::UNIT, q_s = p_s + C::P_BYTES;
  const int items_per_seq = p.H_kv * p.row_blocks.d;
  if (tid == 0) {
    for (int i = 0; i < U; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(&p_full, 4);
    mbar_init(&o_done, 1);
    mbar_init(&q_full, 3);
    mbar_init(&landed, 1);
    mbar_init(&patched, 3);
    fence_mbar_init();
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  // a copy's probabilities of the other copies' keys are zero, for good
  for (int e = tid; e < C::P_BYTES / 16; e += NT)
    *reinterpret_cast<uint4 *>(sm + U * C::UNIT + e * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  // tensor memory after the kernel before, and the next kernel after that (as
  // in gemm_fp8.cu): of two kernels on an SM the earlier never waits for the later
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 8) {
    tmem_alloc(&tm_s, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = tm_s, tm_score = tm + D;

  Walk w{};
  const bool any =
      w.begin<KT, NT>(p, items_per_seq, warp_sum, place, blockIdx.x, gridDim.x);
  if (!any && tid == 0 && !p.by_item) p.cut[blockIdx.x].x = -1;
  int tb = 0, patches = 0;  // tiles and cleared units of the items before
  int loaded = 0, used = 0;  // units that warp 0 has loaded, and warp 8 given back last, plus one
  bool gave_up = false;
  for (int seg = 0; any && w.pos < w.end; ++seg) {
    const int n = w.tiles(), s = w.s, len = w.len, tile0 = w.tile0;
    const int kvh = p.row_blocks.div(w.x), r0 = (w.x - kvh * (int)p.row_blocks.d) * ROWS;
    // the item's last tile is here, and ends inside a unit
    const int patch_from = len - (tile0 + n - 1) * KT;
    const bool patch = patch_from < KT;
    const int nodes = TREE ? seq_nodes(p, s, w.x == 0 && tile0 == 0 && tid == 0) : 0;
    if (tid < ROWS) {
      rows[tid] = out_row(p, s, kvh, r0 + tid);
      if (TREE && rows[tid] >= 0 && p.G.div(r0 + tid) >= nodes) rows[tid] |= kAbsent;
    }
    if (tid == NT - 1) w.list_join(p, items_per_seq, n);
    __syncthreads();
    bool ok = true;
    if (warp == 0) {
      // lane: one box of a unit; boxes of `box` tokens, D / 64 of them side by side
      const int32_t *table = p.table + (long long)s * p.max_pages;
      const int j = lane / (D / 64), c = lane % (D / 64);  // box row, 64 columns
      const bool mine = j * box < KT;
      auto page_of = [&](int i) -> int {
        const int key = (tile0 + i) * KT + j * box;
        return mine && i < n && key < len ? table[p.page_size.div(key)] : -1;
      };
      int page = page_of(0);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int key = (tile0 + i) * KT + j * box, next = page_of(i + 1);
        bool live = mine && key < len;
        if (live && (page < 0 || page >= p.n_pages)) {
          set_error(p.err, kDevBadPage);
          live = false;
        }
        const int in_page = key - p.page_size.div(key) * (int)p.page_size.d;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * box * 128;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int u = 2 * (tb + i) + v, slot = u % U;
          ok = ok && mbar_wait(&empty[slot], (u / U + 1) & 1, p.err, kSiteAttnTile);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
          __syncwarp();
          loaded = u + 1;
          if (live)
            tma_load_4d(sm + slot * C::UNIT + c * (KT * 128) + j * box * 128, v ? &mv : &mk, c * 64,
                        kvh, in_page, page, &full[slot]);
        }
        page = next;
      }
    } else if (warp < 4) {
      const int t96 = tid - 32;
#pragma unroll 4
      for (int e = t96; e < 128 * CH; e += 96) {
        const int r = e / CH, c = e % CH;
        const long long row = rows[r % ROWS];
        const bool live = row >= 0 && !(TREE && (row & kAbsent));
        cp_async16(q_s + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                   static_cast<const T *>(p.q) + (live ? row : 0) * D + c * 8, live);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      if (patch) {
        // told by the issuing warp: a wait for the unit's own barrier from here
        // could be phases early, which a parity does not show
        const int slot = (2 * (tb + n - 1) + 1) % U;
        ok = mbar_wait(&landed, patches & 1, p.err, kSiteAttnTile);
        ok = __all_sync(0xffffffffu, ok);
        const int from = max(patch_from, 0);
        if (ok)
          for (int e = t96; e < (KT - from) * CH; e += 96) {
            const int row = from + e / CH, c = e % CH;
            *reinterpret_cast<uint4 *>(sm + slot * C::UNIT + (c >> 3) * (KT * 128) + row * 128 +
                                       ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&patched);
      }
    } else if (warp == 8) {
      auto sums = [&](int i) {  // O (+)= P V of tile i
        const int t = tb + i, u = 2 * t + 1, slot = u % U;
        ok = ok && mbar_wait_both(&p_full, t & 1, &full[slot], (u / U) & 1, p.err, kSiteAttnSum);
        ok = __all_sync(0xffffffffu, ok);
        if (patch && i == n - 1) {
          if (ok && lane == 0) mbar_arrive(&landed);
          ok = ok && mbar_wait(&patched, patches & 1, p.err, kSiteAttnTile);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks)
          umma_bf16_elect(tm, sdesc_kmajor(p_s + ks * 32),
                          sdesc_mnmajor(units_s + slot * C::UNIT + ks * 2048, KT * 128),
                          idesc_bf16_f32(128, D, false, true), i > 0 || ks > 0);
        umma_commit_elect(&empty[slot]);
        umma_commit_elect(&o_done);
        used = u + 1;
      };
      ok = mbar_wait(&q_full, seg & 1, p.err, kSiteAttnTile);
      ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int t = tb + i, b = t & 1, u = 2 * t, slot = u % U;
        ok = mbar_wait_both(&s_empty[b], ((t >> 1) + 1) & 1, &full[slot], (u / U) & 1, p.err,
                            kSiteAttnScore);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_bf16_elect(tm_score + b * KT,
                          sdesc_kmajor(q_s + (ks >> 2) * (128 * 128) + (ks & 3) * 32),
                          sdesc_kmajor(units_s + slot * C::UNIT + (ks >> 2) * (KT * 128) +
                                       (ks & 3) * 32),
                          idesc_bf16_f32(128, KT, false, false), ks > 0);
        umma_commit_elect(&empty[slot]);
        umma_commit_elect(&s_full[b]);
        used = u + 1;
        if (i > 0) sums(i - 1);
      }
      if (ok) sums(n - 1);
    } else {
      const int R = (warp & 3) * 32 + lane, r = R % ROWS, part = R / ROWS * KC;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, tm_sum = tm + lanes;
      const int row = r0 + r;
      const int t_row = p.G.div(row);
      const bool live = row < p.T * (int)p.G.d;
      const int lim = !live ? 0 : !TREE ? len - p.T + t_row + 1 : t_row < nodes ? len - nodes : len;
      const unsigned long long word = TREE && live ? node_word(p, s, t_row, nodes) : 0;
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int t = tb + i, b = t & 1;
        ok = mbar_wait(&s_full[b], (t >> 1) & 1, p.err, kSiteAttnScore);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float x[KC];
#pragma unroll
        for (int c = 0; c < KC; c += 32) {
          float part32[32];
          tmem_ld32(tm_score + lanes + b * KT + part + c, part32);
#pragma unroll
          for (int j = 0; j < 32; ++j) x[c + j] = part32[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[b]);
        const int key0 = (tile0 + i) * KT + part;
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          x[j] = sees<TREE>(key0 + j, lim, word) ? x[j] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, x[j]);
        }
        const bool grow = mx > ref + kMaxGrowth;
        const float next = grow ? mx : ref;
        const float alpha = grow ? exp2_ftz(ref - next) : 1.f;
        ref = next;
        l *= alpha;
        // the tile before has left P, and its product is in the sums
        if (i > 0) ok = mbar_wait(&o_done, (t - 1) & 1, p.err, kSiteAttnSum);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tm_sum + c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= alpha;
            tmem_st32(tm_sum + c, o);
          }
          tmem_wait_st();
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        unsigned char *prow = sm + U * C::UNIT + R * 128;
#pragma unroll
        for (int j = 0; j < KC; j += 8) {
          uint32_t q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = exp2_ftz(x[j + 2 * k] - base), e = exp2_ftz(x[j + 2 * k + 1] - base);
            l += a + e;
            q[k] = bf16x2(a, e);
          }
          *reinterpret_cast<uint4 *>(prow + ((((part + j) >> 3) ^ (R & 7)) << 4)) =
              make_uint4(q[0], q[1], q[2], q[3]);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full);
      }
      ok = ok && mbar_wait(&o_done, (tb + n - 1) & 1, p.err, kSiteAttnSum);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        // all copies and products of the item are done: the sums take their place
        tc_fence_after();
        float *so = reinterpret_cast<float *>(sm) + R * C::PITCH;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tm_sum + c, o);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(so + c + j) =
                make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
        sml[R] = make_float2(ref, l);
        tc_fence_before();
      }
    }
    gave_up = __syncthreads_or(!ok);
    if (gave_up) break;
    finish_item<C, TREE>(p, reinterpret_cast<const float *>(sm), C::PITCH, sml, rows, n == w.nt,
                   (long long)blockIdx.x * 2 + (seg > 0));
    fence_proxy_async();  // the sums' place is loaded by TMA next
    __syncthreads();
    tb += n;
    patches += patch;
    w.next<KT>(p, items_per_seq, n);
    if (C::COPIES > 1 && C::OUT_BYTES > U * C::UNIT && w.pos < w.end) {
      // the sums have overwritten P's zeros
      for (int e = tid; e < C::P_BYTES / 16; e += NT)
        *reinterpret_cast<uint4 *>(sm + U * C::UNIT + e * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
    }
  }
  if (gave_up) {  // otherwise every item's copies and products have been waited for
    if (warp == 0)
      for (int u = max(loaded - U, 0); u < loaded; ++u) mbar_drain(&full[u % U], (u / U) & 1);
    if (warp == 8 && used > 0) mbar_drain(&empty[(used - 1) % U], ((used - 1) / U) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tm, C::TCOLS);
}

// ---- more rows (bf16): tiles of 128 rows and 128 keys, probabilities in tensor memory ----
//
// Rows x keys of more than a tile of 128 rows are bound by the products and the
// exponentials together (128 rows, 128 keys, heads of 128: some 1,100 cycles of
// products at the measured bf16 rate, 1,024 of exponentials), so neither may wait
// for the other. Two tiles of scores are under way for every tile of rows: while one
// is turned into probabilities, the other's products run. With two tiles of rows
// (NQ = 2: every key and value then serves 256 rows) tensor memory has room for
// tiles of 64 keys; with one (heads of 256, whose sums fill half of it, or up to
// 128 rows) for 128. One tile of 128 keys a tile of rows instead of two of 64 was
// slower (32 sequences x 32 nodes, below: 71 us for 66).
// A lane of the four warps of a row tile has a whole row, so maximum and sum need
// no other lane; probabilities go back to tensor memory over their scores, as the
// next product's first operand, and cost no shared memory. Scores overwrite the
// probabilities of the tile before the last once the product that reads those is
// over.
// Every wait costs some 200 to 500 cycles, so each kind of work has a warp of its
// own (the first case below took 90 us with one warp for a tile's products and one
// for all copies, 66 with these). Polls by one lane, the others of its warp waiting,
// were slower (75).
// A copy takes some 250 cycles to begin, whatever its size: a unit of V has all its
// columns in one where pages allow (338 us for 447, the last case below).
// The blocks of rows of an item (64 nodes x 8 heads of 256 are four) go to
// neighbouring blocks of the grid with the same run of keys, which then pass from L2:
// one behind the other they read memory 3.6 times over (645 us for 524, then). Copies
// shared by two of them (a cluster, each loading every other box for both) were
// slower, 349 us for 327: each then waits for the other's places.
//
// Measured (16 heads on 2, bf16): 32 sequences of 512 to 8192 with 32 nodes, heads
// of 128, pages of 16: 55 us (22.2 by bytes, 19.1 by products; the warp-level kernel
// for up to 128 rows took 225); 8 of 30k to 65k with 64 nodes, heads of 256: 331 us,
// 1.20 PFLOP/s of 1.92 (985).
template <int D_, int NQ_>
struct WideCfg {
  using In = __nv_bfloat16;
  static constexpr bool kTensorMemory = true;
  static constexpr int D = D_, NQ = NQ_, KT = 128 / NQ, ROWS = 128 * NQ;
  // four warps of copies and products, one a row for each lane for each tile of rows,
  // two of products for the second tile
  static constexpr int THREADS = 256 + 192 * (NQ - 1);
  // K and V arrive in units, each in a ring of its own: of K KA times 64 columns of
  // the tile's keys, of V KV of its keys, which is what a few products read, so that
  // a place is loaded again while the rest of its tile is still in use
  static constexpr int TILE = KT * D * 2, CC = TILE > 16384 ? TILE / 16384 : 1, UNIT = TILE / CC;
  static constexpr int KA = D / 64 / CC, KV = KT / CC;
  static constexpr int Q_BYTES = ROWS * D * 2;
  // places of the rings: a tile of heads of 256 is all four of K's, and a product starts
  // with the first unit of V while the last is on its way
  static constexpr int UK = 4, UV = D == 256 ? 6 : 4;
  static constexpr int SMEM = (UK + UV) * UNIT + Q_BYTES + 1024;
  static constexpr int TCOLS = 512;  // sums, then two tiles of scores for each tile of rows
  static constexpr int PER_SM = 1;
  static_assert(NQ * D + 256 <= TCOLS && UK >= CC && UV >= CC && SMEM <= 225 * 1024, "it fits");
};

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, int c3, int c4, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem], A in the lanes of its rows, two bf16 a column; from a whole
// converged warp, as umma_bf16_elect.
__device__ __forceinline__ void umma_bf16_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                   uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// 64 columns in one load and one wait: a lane's values are valid when it retires.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]),
        "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
        "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]),
        "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]),
        "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]),
        "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]),
        "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr)
      : "memory");
}

// Which of the 64 keys from `key` on a row sees, as bits (sees() for each).
__device__ __forceinline__ unsigned long long seen64(int key, int lim, unsigned long long word) {
  const int past = key - lim;  // of the limit
  if (past <= -64) return ~0ull;
  if (past < 0) return (word << -past) | ((1ull << -past) - 1);
  return past < 64 ? word >> past : 0;
}

__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

template <class C, bool TREE>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM)
    attn_wide_kernel(const AttnParams p, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, int box) {
  using T = __nv_bfloat16;
  constexpr int D = C::D, KT = C::KT, NT = C::THREADS, NQ = C::NQ, UK = C::UK, UV = C::UV;
  constexpr int CH = D / 8, CC = C::CC, KA = C::KA, KV = C::KV;  // 16-byte chunks of a row; see WideCfg
  extern __shared__ unsigned char raw[];
  unsigned char *sm =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[2][UV], empty[2][UV];  // of K, of V
  __shared__ uint64_t s_full[2 * NQ], p_full[2 * NQ], o_done[2 * NQ], o_free[NQ];
  __shared__ uint64_t q_full[NQ], landed, patched, over[2 * NQ];
  __shared__ long long warp_sum[NT / 32];
  __shared__ Place place;
  __shared__ uint32_t tm_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // warps: 0 K, 1 V, 2 and 12 products of queries and K, 3 and 13 of
  // probabilities and V, 4 .. 4 + 4 NQ rows. A product's polls (some 200 cycles
  // each, of phases long over too) and the copies it waits for then hold up no other's.
  const bool scores = warp == 2 || warp == 12, sums = warp == 3 || warp == 13;
  static_assert(UV >= UK, "places of either");
  // unit u of K (of V): its place, there and in shared memory, and the round of the ring
  auto slot_of = [](int v, int u) { return v ? u % UV : u % UK; };
  auto round_of = [](int v, int u) { return v ? u / UV : u / UK; };
  auto unit_at = [](int v, int slot) { return (v * UK + slot) * C::UNIT; };
  const uint32_t units_s = smem_u32(sm), q_s = units_s + (UK + UV) * C::UNIT;
  const int items_per_seq = p.H_kv, RB = p.row_blocks.d;
  const int group = p.row_blocks.div(blockIdx.x), rb = blockIdx.x - group * RB;
  const int groups = p.row_blocks.div(gridDim.x), r0 = rb * C::ROWS;
  if (tid == 0) {
    for (int i = 0; i < 2 * UV; ++i) {
      mbar_init(&full[0][0] + i, 1);
      mbar_init(&empty[0][0] + i, NQ);
    }
    for (int i = 0; i < 2 * NQ; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&o_free[i], 4);
      mbar_init(&q_full[i], 4);
    }
    for (int i = 0; i < 2 * NQ; ++i) mbar_init(&over[i], 1);
    mbar_init(&landed, NQ);
    mbar_init(&patched, 1);
    fence_mbar_init();
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as attn_tc_kernel
  if (warp == 3) {
    tmem_alloc(&tm_s, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = tm_s, tm_score = tm + NQ * D;

  // Every role walks the block's items on its own.
  Walk w{};
  const bool any = w.begin<KT, NT>(p, items_per_seq, warp_sum, place, group, groups);
  if (!any && tid == 0 && rb == 0 && !p.by_item) p.cut[group].x = -1;
  int tb = 0, patches = 0;   // tiles and cleared tiles of the items before
  int loaded = 0;  // units of K (of V) loaded
  bool ok = any;
  for (int seg = 0; ok && w.pos < w.end; ++seg) {
    const int n = w.tiles(), s = w.s, len = w.len, tile0 = w.tile0, kvh = w.x;
    // the item's last tile is here, and ends inside a tile of V
    const int patch_from = len - (tile0 + n - 1) * KT;
    const bool patch = patch_from < KT;
    // `count` units of K (of V) from u on have arrived, and phase `phase` of `bar` is over.
    auto wait_units = [&](int v, int u0, auto count, uint64_t *bar, int phase) {
      bool all = false;
      for (uint32_t i = 0; i < kMaxPolls && !all; ++i) {
        all = !bar || mbar_try_wait(bar, phase & 1);
#pragma unroll
        for (int c = 0; c < count; ++c)
          all &= mbar_try_wait(&full[v][slot_of(v, u0 + c)], round_of(v, u0 + c) & 1);
      }
      if (!all) set_error(p.err, kDevTimeout | (kSiteAttnTile << 8));
      all = __all_sync(0xffffffffu, all);
      tc_fence_after();
      return all;
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, CC> whole_tile;
    if (warp < 2) {
      const int v = warp;  // K, V
      if (v == 0 && lane == 0 && rb == 0) w.list_join(p, items_per_seq, n);
      if (TREE && v == 1 && lane == 0) seq_nodes(p, s, w.x == 0 && tile0 == 0);
      // A lane's boxes of a tile, at most two, unit by unit: 64 columns of `keys` keys, or
      // all of a unit's columns where a box has all of its keys (a copy takes some 250
      // cycles to begin, whatever its size)
      const int32_t *table = p.table + (long long)s * p.max_pages;
      const int unit_keys = v ? KV : KT, keys = min(box, unit_keys);  // of a unit, of a box
      const int cols = keys == unit_keys ? 1 : v ? D / 64 : KA;       // boxes side by side
      const int per = unit_keys / keys * cols;                        // boxes of a unit
      const int bytes = C::UNIT / per, log_cols = 31 - __clz(cols), log_per = 31 - __clz(per);
      auto key_of = [&](int e) {  // first key of box e in its tile
        return (v ? (e >> log_per) * KV : 0) + ((e & (per - 1)) >> log_cols) * keys;
      };
      auto page_of = [&](int i, int e) -> int {
        const int key = (tile0 + i) * KT + key_of(e);
        return e < CC * per && i < n && key < len ? table[p.page_size.div(key)] : -1;
      };
      int page[2] = {page_of(0, lane), page_of(0, lane + 32)};
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        int next[2], at[2];
        bool live[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int e = lane + 32 * x, key = (tile0 + i) * KT + key_of(e);
          next[x] = page_of(i + 1, e);
          live[x] = e < CC * per && key < len;
          if (live[x] && (page[x] < 0 || page[x] >= p.n_pages)) {
            set_error(p.err, kDevBadPage);
            live[x] = false;
          }
          at[x] = key - p.page_size.div(key) * (int)p.page_size.d;
        }
#pragma unroll 1
        for (int c = 0; c < CC; ++c) {
          const int u = (tb + i) * CC + c, slot = slot_of(v, u);
          ok = ok && mbar_wait(&empty[v][slot], (round_of(v, u) + 1) & 1, p.err, kSiteAttnTile);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          bool mine[2];
          uint32_t boxes = 0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mine[x] = live[x] && (lane + 32 * x) >> log_per == c;
            boxes += __popc(__ballot_sync(0xffffffffu, mine[x]));
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[v][slot], boxes * bytes);
          __syncwarp();
          loaded = u + 1;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int e = (lane + 32 * x) & (per - 1), col = e & (cols - 1);
            if (mine[x])
              tma_load_5d(sm + unit_at(v, slot) + (col * unit_keys + (e >> log_cols) * keys) * 128,
                          v ? &mv : &mk, 0, at[x], (v ? 0 : c * KA) + col, kvh, page[x],
                          &full[v][slot]);
          }
        }
        page[0] = next[0];
        page[1] = next[1];
      }
      if (v && ok && patch) {
        // told by the warp of the products, as in attn_tc_kernel
        ok = mbar_wait(&landed, patches & 1, p.err, kSiteAttnTile);
        ok = __all_sync(0xffffffffu, ok);
        const int from = max(patch_from, 0);
        if (ok)
          for (int e = lane; e < (KT - from) * CH; e += 32) {
            const int key = from + e / CH, c = e % CH;
            const int slot = slot_of(1, (tb + n - 1) * CC + key / KV);
            *reinterpret_cast<uint4 *>(sm + unit_at(1, slot) + (c >> 3) * (KV * 128) +
                                       key % KV * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&patched);
      }
    } else if (scores) {  // S = Q K^T
      const int q = warp > 3;
      ok = mbar_wait(&q_full[q], seg & 1, p.err, kSiteAttnTile);
      ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
      for (int t = tb; t < tb + n && ok; ++t) {
        // in the place of the tile before the last, whose product is over (of the
        // first two: a phase before the first is over)
        const int b = 2 * q + (t & 1);
        ok = wait_units(0, t * CC, whole_tile, &o_done[b], (t >> 1) + 1);
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < CC; ++c) {
          const int slot = slot_of(0, t * CC + c);
#pragma unroll
          for (int ks = 0; ks < 4 * KA; ++ks)
            umma_bf16_elect(tm_score + b * KT,
                            sdesc_kmajor(q_s + q * (128 * D * 2) +
                                         (c * KA + ks / 4) * (128 * 128) + ks % 4 * 32),
                            sdesc_kmajor(units_s + unit_at(0, slot) + ks / 4 * (KT * 128) +
                                         ks % 4 * 32),
                            idesc_bf16_f32(128, KT, false, false), c > 0 || ks > 0);
          if (c == CC - 1) umma_commit_elect(&s_full[b]);
          umma_commit_elect(&empty[0][slot]);
        }
      }
    } else if (sums) {  // O (+)= P V
      const int q = warp > 3;
      ok = mbar_wait(&o_free[q], (seg + 1) & 1, p.err, kSiteAttnSum);
      ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
      for (int t = tb; t < tb + n && ok; ++t) {
        const int b = 2 * q + (t & 1);
        ok = wait_units(1, t * CC, one, &p_full[b], t >> 1);
        if (patch && t == tb + n - 1) {
          ok = ok && wait_units(1, t * CC, whole_tile, nullptr, 0);
          if (ok && lane == 0) mbar_arrive(&landed);
          ok = ok && mbar_wait(&patched, patches & 1, p.err, kSiteAttnTile);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < CC; ++c) {
          const int slot = slot_of(1, t * CC + c);
          if (c > 0) {
            ok = wait_units(1, t * CC + c, one, nullptr, 0);
            if (!ok) break;
          }
#pragma unroll
          for (int ks = 0; ks < KV / 16; ++ks)
            umma_bf16_ts_elect(tm + q * D, tm_score + b * KT + KT / 2 + (c * (KV / 16) + ks) * 8,
                               sdesc_mnmajor(units_s + unit_at(1, slot) + ks * 2048, KV * 128),
                               idesc_bf16_f32(128, D, false, true), t > tb || c > 0 || ks > 0);
          if (c == CC - 1) umma_commit_elect(&o_done[b]);
          umma_commit_elect(&empty[1][slot]);
        }
      }
    } else {
      // a row of this lane's
      const int q = (warp - 4) >> 2, R = (warp & 3) * 32 + lane, row = r0 + q * 128 + R;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tm_sum = tm + q * D + lanes;
      const int nodes = TREE ? seq_nodes(p, s, false) : p.T;
      const int t_row = p.G.div(row);
      const bool mine = row < p.T * (int)p.G.d, absent = TREE && mine && t_row >= nodes;
      // rows that are not there take part without a mask
      const int lim = !mine || absent ? len : TREE ? len - nodes : len - p.T + t_row + 1;
      const unsigned long long word = TREE && mine ? node_word(p, s, t_row, nodes) : 0;
      // This warp's 32 rows of queries of an item to shared memory, 16 bytes a copy: a
      // lane knows where its row is.
      auto load_q = [&](int s, int x) {
        const int nodes = TREE ? seq_nodes(p, s, false) : p.T;
        const long long from = mine && t_row < nodes ? out_row(p, s, x, row) : -1;
#pragma unroll 8
        for (int e = lane; e < 32 * CH; e += 32) {
          const int i = e / CH, r = (warp & 3) * 32 + i, c = e % CH;
          const long long at = __shfl_sync(0xffffffffu, from, i);
          cp_async16(q_s + q * (128 * D * 2) + (c >> 3) * (128 * 128) + r * 128 +
                         (((c & 7) ^ (r & 7)) << 4),
                     static_cast<const T *>(p.q) + max(at, 0ll) * D + c * 8, at >= 0);
        }
        cp_async_commit();
      };
      auto q_loaded = [&] {
        cp_async_wait<0>();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[q]);
      };
      if (seg == 0) {
        load_q(s, kvh);
        q_loaded();
      }
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int t = tb + i, b = 2 * q + (t & 1);
        ok = mbar_wait(&s_full[b], (t >> 1) & 1, p.err, kSiteAttnScore);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // What every tile runs is kept short, in halves of 64 keys (read twice where a
        // tile has two) and by loops that are not unrolled: longer code is fetched anew
        // for every tile, and the warps that issue products wait for theirs behind it.
        const uint32_t score = tm_score + b * KT + lanes;
        const int key0 = (tile0 + i) * KT;
        float factor = p.scale_log2;
        if (factor < 0.f || __any_sync(0xffffffffu, key0 + KT > lim)) {
          // scaled and masked in their place, so that the rest needs no mask
#pragma unroll 1
          for (int c = 0; c < KT; c += 16) {
            const unsigned seen = (unsigned)seen64(key0 + c, lim, word);
            float x[16];
            tmem_ld16(score + c, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = seen >> j & 1 ? x[j] * factor : -INFINITY;
            tmem_st16(score + c, x);
          }
          tmem_wait_st();
          factor = 1.f;
        }
        float x[64], top = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < KT / 64; ++h) {
          tmem_ld64(score + 64 * h, x);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            float &m = mx[j >> 1 & 3];
            m = fmaxf(fmaxf(m, x[j]), x[j + 1]);
          }
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        }
        top *= factor;  // as the largest product: rounding keeps the order
        const bool grow = top > ref + kMaxGrowth;
        const float next = grow ? top : ref, alpha = grow ? exp2_ftz(ref - next) : 1.f;
        ref = next;
        l *= alpha;
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          ok = mbar_wait(&o_done[2 * q + ((t - 1) & 1)], ((t - 1) >> 1) & 1, p.err, kSiteAttnSum);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(tm_sum + c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= alpha;
            tmem_st16(tm_sum + c, o);
          }
          tmem_wait_st();
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // the later keys first: the probabilities take the place of their scores
#pragma unroll 1
        for (int h = KT / 64 - 1; h >= 0; --h) {
          if (KT > 64) tmem_ld64(score + 64 * h, x);
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float y = -base, z = -base;
              fma2(y, z, x[c + 2 * j], x[c + 2 * j + 1], factor, factor);
              y = exp2_ftz(y);
              z = exp2_ftz(z);
              add2(sum[2 * (j & 1)], sum[2 * (j & 1) + 1], y, z);
              pk[j] = __uint_as_float(bf16x2(y, z));
            }
            tmem_st16(score + KT / 2 + 32 * h + c / 2, pk);
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      // The item's last scores are over: the next one's queries may come.
      Walk after = w;
      after.next<KT>(p, items_per_seq, n);
      const bool more = ok && after.pos < after.end;
      if (more) load_q(after.s, after.x);
      if (ok) {
        const int t = tb + n - 1;
        ok = mbar_wait(&o_done[2 * q + (t & 1)], (t >> 1) & 1, p.err, kSiteAttnSum);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (more) q_loaded();
      if (ok) {
        tc_fence_after();
        const bool whole = n == w.nt;
        const long long to = mine ? out_row(p, s, kvh, row) : -1;
        // pieces: [slot][row block][D / 4][row][4], a lane a row
        const long long piece = ((long long)group * 2 + (seg > 0)) * RB + rb;
        const int pr = q * 128 + R;
        if (absent) l = 0.f;
        // a row without keys has l = 0 and sums of 0: its output is 0
        const float inv = absent ? 0.f : 1.f / (l == 0.f ? 1.f : l);
        if (!whole && mine)
          p.part_ml[piece * C::ROWS + pr] = make_float2(absent ? -INFINITY : ref, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tm_sum + c, o);
          if (!mine) continue;
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = absent ? 0.f : whole ? o[j] * inv : o[j];
          if (whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + to * D + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              dst[j] = make_uint4(bf16x2(o[8 * j], o[8 * j + 1]), bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                  bf16x2(o[8 * j + 4], o[8 * j + 5]), bf16x2(o[8 * j + 6], o[8 * j + 7]));
          } else {
            float4 *dst =
                reinterpret_cast<float4 *>(p.part_o) + (piece * (D / 4) + c / 4) * C::ROWS + pr;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j * C::ROWS] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[q]);
      }
    }
    tb += n;
    patches += patch;
    w.next<KT>(p, items_per_seq, n);
  }
  if (any && !ok) {  // otherwise every copy and product has been waited for
    if (warp < 2)
      for (int u = max(loaded - (warp ? UV : UK), 0); u < loaded; ++u)
        mbar_drain(&full[warp][slot_of(warp, u)], round_of(warp, u) & 1);
    if (scores || sums) {
      const int i = 2 * (warp > 3) + sums;
      umma_commit_elect(&over[i]);
      mbar_drain(&over[i], 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) tmem_dealloc(tm, C::TCOLS);
}

// Joins the cut items of attn_wide_kernel: block (i, y) rows 8 y .. 8 y + 8 of the
// item listed at i; the pieces are taken in turn by W groups of 128 threads, whose
// sums are added in order. A thread has every 16th four columns of a row.
template <class C, int W>
__global__ void __launch_bounds__(128 * W) join_wide_kernel(const AttnParams p, int groups) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int D = C::D, VL = D / 64;
  const int4 cut = p.cut[blockIdx.x];
  // a main kernel that gave up (error word) may have left the list unwritten
  if (cut.x < 0 || cut.x >= p.n_seqs * p.H_kv || cut.y < 0 || cut.z <= 0 || cut.w <= 0) return;
  const int first = cut.y >> 1, np = (cut.z - 1) / cut.w + 2;  // blocks of the item
  if (first + (long long)np > groups) return;
  const int tid = threadIdx.x & 127, turn = threadIdx.x >> 7;
  const int row = blockIdx.y * 8 + (tid & 7), rb = row / C::ROWS, r = row % C::ROWS, c4 = tid >> 3;
  const int s = cut.x / p.H_kv, kvh = cut.x - s * p.H_kv;
  auto slot = [&](int i) {  // as in join_kernel, of this block of rows
    return (i == 0 ? (long long)cut.y : 2LL * (first + i)) * (int)p.row_blocks.d + rb;
  };
  const bool mine = row < p.T * (int)p.G.d;
  float mm = -INFINITY, ll = 0.f;
  float4 sum[VL];
#pragma unroll
  for (int j = 0; j < VL; ++j) sum[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine) {
#pragma unroll 4
    for (int i = 0; i < np; ++i) mm = fmaxf(mm, p.part_ml[slot(i) * C::ROWS + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
    for (int i = turn; i < np; i += W) {
      const float2 ml = p.part_ml[slot(i) * C::ROWS + r];
      const float f = exp2_ftz(ml.x - ref);
      ll += f * ml.y;
      const float4 *o = reinterpret_cast<const float4 *>(p.part_o) + slot(i) * (D / 4) * C::ROWS + r;
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const float4 v = o[(j * 16 + c4) * C::ROWS];
        sum[j].x = fmaf(f, v.x, sum[j].x);
        sum[j].y = fmaf(f, v.y, sum[j].y);
        sum[j].z = fmaf(f, v.z, sum[j].z);
        sum[j].w = fmaf(f, v.w, sum[j].w);
      }
    }
  }
  if constexpr (W > 1) {
    __shared__ float4 others[W - 1][VL][128];
    __shared__ float sl[W - 1][128];
    if (turn > 0) {
#pragma unroll
      for (int j = 0; j < VL; ++j) others[turn - 1][j][tid] = sum[j];
      sl[turn - 1][tid] = ll;
    }
    __syncthreads();
    if (turn > 0) return;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      ll += sl[k][tid];
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const float4 v = others[k][j][tid];
        sum[j].x += v.x; sum[j].y += v.y; sum[j].z += v.z; sum[j].w += v.w;
      }
    }
  }
  if (!mine) return;
  const float inv = 1.f / (ll == 0.f ? 1.f : ll);
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + out_row(p, s, kvh, row) * D;
#pragma unroll
  for (int j = 0; j < VL; ++j)
    store4(out + (j * 16 + c4) * 4,
           make_float4(sum[j].x * inv, sum[j].y * inv, sum[j].z * inv, sum[j].w * inv));
}

// Joins the cut items: block (i, r) row r of the item listed at i. The W warps
// take the pieces in turn, a lane D / 64 pairs of columns.
template <typename T, int D, int ROWS, int W>
__global__ void __launch_bounds__(32 * W) join_kernel(const AttnParams p, int grid) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int VL = D / 64;  // float2 of a lane
  const int4 cut = p.cut[blockIdx.x];
  // a main kernel that gave up (error word) may have left the list unwritten
  if (cut.x < 0 || cut.x >= p.n_seqs * p.H_kv * (int)p.row_blocks.d || cut.y < 0 || cut.z <= 0 ||
      cut.w <= 0)
    return;
  const int first = cut.y >> 1, np = (cut.z - 1) / cut.w + 2;  // blocks of the item
  if (first + (long long)np > grid) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y;
  const int per_seq = p.H_kv * (int)p.row_blocks.d, s = cut.x / per_seq, x = cut.x - s * per_seq;
  const int kvh = p.row_blocks.div(x), rb = x - kvh * (int)p.row_blocks.d;
  const long long row = out_row(p, s, kvh, rb * ROWS + r);
  if (row < 0) return;
  // the item is the first block's last item (its only one if it starts there),
  // and the first of all later blocks
  auto slot = [&](int i) { return i == 0 ? (long long)cut.y : 2LL * (first + i); };
  float mm = -INFINITY;
  for (int i = lane; i < np; i += 32) mm = fmaxf(mm, p.part_ml[slot(i) * ROWS + r].x);
#pragma unroll
  for (int off = 16; off; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
  const float ref = mm == -INFINITY ? 0.f : mm;
  float2 sum[VL];
  float ll = 0.f;
#pragma unroll
  for (int j = 0; j < VL; ++j) sum[j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < np; i += W) {
    const float2 ml = p.part_ml[slot(i) * ROWS + r];
    const float f = exp2_ftz(ml.x - ref);
    ll += f * ml.y;
    const float2 *o = reinterpret_cast<const float2 *>(p.part_o + (slot(i) * ROWS + r) * D);
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      const float2 v = o[j * 32 + lane];
      sum[j].x = fmaf(f, v.x, sum[j].x);
      sum[j].y = fmaf(f, v.y, sum[j].y);
    }
  }
  __shared__ float2 so[W][D / 2];
  __shared__ float sl[W];
#pragma unroll
  for (int j = 0; j < VL; ++j) so[warp][j * 32 + lane] = sum[j];
  if (lane == 0) sl[warp] = ll;
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= D / 2) return;
  float l = 0.f;
  float2 v = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    l += sl[k];
    v.x += so[k][c].x;
    v.y += so[k][c].y;
  }
  const float inv = 1.f / (l == 0.f ? 1.f : l);
  T *out = static_cast<T *>(p.out) + row * D + 2 * c;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint32_t *>(out) = bf16x2(v.x * inv, v.y * inv);
  else
    *reinterpret_cast<float2 *>(out) = make_float2(v.x * inv, v.y * inv);
}

// ---- host side ------------------------------------------------------------------

// Tokens of a page in one TMA box (whole 8-row groups of a unit), 0 when the
// pages do not cut a unit of 64 keys evenly.
int box_of(const KvLayout &c) {
  const int ps = c.page_size;
  if (!c.bf16 || c.n_pages == 0 || ps % 8) return 0;
  // a tensor map's strides end at 2^40 bytes
  if ((c.page_stride | c.token_stride | c.head_stride) >> 39) return 0;
  return ps % 64 == 0 ? 64 : 64 % ps == 0 ? ps : 0;
}

// Calls f with the configuration of a head size, type and number of rows (T
// x G of an item): the smallest block of rows that holds them all, or the
// largest there is (each block of rows reads the keys again).
template <typename T, int D, bool TREE, class F>
auto with_rows(int rows, int box, F f) {
  if constexpr (sizeof(T) == 2) {
    if (rows <= 16) return f(Cfg<T, D, 1>{});
    if constexpr (TREE) {
      // us, 64 sequences of 512 to 8192 (D = 256: to 4096), 2 kv heads, pages of 16 and
      // 64 tokens; what follows below in brackets. 72, 128 and 256 rows: D = 64 42 and
      // 40 (80, 76), 37 and 40 (73, 80), 61 and 50 (160, 127); D = 128 53 and 48 (241,
      // 203), 52 and 56 (163, 173), 71 and 68 (294, 260); D = 256 59 and 61 (150, 166),
      // 67 and 65 (127, 135), 98 and 92 (229, 235). Pages without a box (24, 100 or 7
      // tokens), D = 128, 256 rows: 217 to 235, by the warp-level kernel; fp32 1290.
      if (box && rows > 128) return f(WideCfg<D, D == 256 ? 1 : 2>{});
      if (box && rows > 64) return f(WideCfg<D, 1>{});
    }
    // Tensor memory where it measured faster or even (us, 64 sequences of 512 to
    // 8192, D = 128, or to 4096, D = 256, boxes of 16, 32 and 64 tokens;
    // warp-level kernel in brackets): 64 rows of D = 256 91, 86, 84 (110), 128
    // rows 112, 107, 105 (196); 64 rows of D = 128 96, 82, 77 (80), 128 rows 114,
    // 101, 97 (146). 32 rows of D = 128 91, 77, 72 (60), of D = 256 84, 78, 76
    // (80); 64 rows of D = 64 were even.
    if constexpr (D >= 128) {
      if (box && rows > 64) return f(TcCfg<D, 1>{});
      if (box && rows > 32 && (D == 256 || box >= 32)) return f(TcCfg<D, 2>{});
    }
    if (rows <= 32) return f(Cfg<T, D, 2>{});
    return f(Cfg<T, D, 4>{});
  } else {
    if (rows <= 4) return f(Cfg<T, D, 1>{});
    if (rows <= 8) return f(Cfg<T, D, 2>{});
    if constexpr (D < 256)  // q and the tiles of 32 rows of 256 fill more than an SM has
      if (rows > 16) return f(Cfg<T, D, 8>{});
    return f(Cfg<T, D, 4>{});
  }
}
template <typename T, bool TREE, class F>
auto with_d(int D, int rows, int box, F f) {
  if (D == 64) return with_rows<T, 64, TREE>(rows, box, f);
  if (D == 128) return with_rows<T, 128, TREE>(rows, box, f);
  return with_rows<T, 256, TREE>(rows, box, f);
}
template <bool TREE, class F>
auto with_cfg(const KvLayout &c, int rows, F f) {
  const int box = box_of(c);
  return c.bf16 ? with_d<__nv_bfloat16, TREE>(c.D, rows, box, f)
                : with_d<float, TREE>(c.D, rows, box, f);
}

// A cache as (D, H_kv, page_size, n_pages); boxes of 64 columns x `box` tokens
// of one head and page, 128-byte swizzle.
bool map_cache(CUtensorMap *m, const void *base, const KvLayout &c, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.H_kv, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.head_stride * 2, (cuuint64_t)c.token_stride * 2,
                                 (cuuint64_t)c.page_stride * 2};
  const cuuint32_t b[4] = {64, 1, (cuuint32_t)box, 1}, es[4] = {1, 1, 1, 1};
  return encode_fn() &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                     strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same as (64, page_size, D / 64, H_kv, n_pages); boxes of 64 columns x `box` tokens x
// `cols` times 64 columns, which come to lie one behind the other.
bool map_columns(CUtensorMap *m, const void *base, const KvLayout &c, int box, int cols) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)c.page_size, (cuuint64_t)c.D / 64,
                              (cuuint64_t)c.H_kv, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)c.token_stride * 2, 128, (cuuint64_t)c.head_stride * 2,
                                 (cuuint64_t)c.page_stride * 2};
  const cuuint32_t b[5] = {64, (cuuint32_t)box, (cuuint32_t)cols, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return encode_fn() &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims,
                     strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 152;

template <class C>
constexpr bool kIsWide = false;
template <int D, int NQ>
constexpr bool kIsWide<WideCfg<D, NQ>> = true;

// Blocks of the grid: all that fit the GPU, or as many as there can be tiles.
template <class C>
int grid_of(const KvLayout &c, int n_seqs, int max_pages, int row_blocks) {
  const long long tiles = ((long long)max_pages * c.page_size + C::KT - 1) / C::KT;
  if constexpr (kIsWide<C>) {  // groups of blocks of rows side by side
    const long long items = (long long)n_seqs * c.H_kv;
    const int most = row_blocks < kSms ? kSms / row_blocks : 1;
    const bool few = tiles < most && items * (tiles < 1 ? 1 : tiles) < most;
    return row_blocks * (few ? (int)(items * (tiles < 1 ? 1 : tiles)) : most);
  }
  const long long most = (long long)C::PER_SM * kSms;
  const long long items = (long long)n_seqs * c.H_kv * row_blocks;
  if (tiles < most && items * (tiles < 1 ? 1 : tiles) < most)
    return (int)(items * (tiles < 1 ? 1 : tiles));
  return (int)most;
}

// Blocks for each item when the longest possible sequence is short enough to
// need no line of tiles (0: it is not). The page table's width decides, since
// the lengths are known on the device only: one sequence of 513 tokens takes 5.9
// us in a table of 33 or 64 pages of 16 and 10.2 in one of 512 or 8192. Many items of up to 16 tiles take a
// block each, and the GPU's own scheduling evens them out (256 sequences of 1
// to 1000 tokens, 8 kv heads of 64: 50 us, 77 as a line, where a block's items
// follow one another with a gap at each). Few items are split over a cluster,
// a few tiles a block (one sequence of 513 tokens 5.9 us, 9.2 as a line).
template <class C>
int short_split(const KvLayout &c, const AttnParams &p) {
  const long long tiles = ((long long)p.max_pages * c.page_size + C::KT - 1) / C::KT;
  const long long items = (long long)p.n_seqs * c.H_kv * p.row_blocks.d;
  const long long most = (long long)C::PER_SM * kSms;
  if (tiles <= 2 || items * 2 > most) return tiles <= 16 ? 1 : 0;
  int split = 2;
  // Not more clusters of 8 than find room at once where an SM holds one block:
  // 14 items of 900 tokens, D 256, take 8.5 us by 8 and 10.9 by 4, 18 items
  // 16.4 and 10.9. Where it holds more, all do (72 items, D 64: 6.9 and 7.7).
  const int widest = C::PER_SM > 1 || items <= 14 ? 8 : 4;
  while (split < widest && split * 2 < tiles && items * split * 2 <= most) split *= 2;
  return tiles <= 4 * split ? split : 0;
}

template <class C, bool TREE>
cudaError_t launch_cfg(const AttnParams &p, const KvLayout &c, int grid, cudaStream_t stream) {
  cudaError_t e;
  if constexpr (C::kTensorMemory) {
    static_assert(C::SMEM + (kIsWide<C> ? 2 : 4) * 1024 <= 227 * 1024, "shared memory");
    const int box = box_of(c);
    CUtensorMap mk, mv;
    bool mapped;
    if constexpr (kIsWide<C>) {
      const int kbox = std::min(box, C::KT), vbox = std::min(box, C::KV);
      mapped = map_columns(&mk, p.k, c, kbox, kbox == C::KT ? C::KA : 1) &&
               map_columns(&mv, p.v, c, vbox, vbox == C::KV ? C::D / 64 : 1);
    } else {
      mapped = map_cache(&mk, p.k, c, box) && map_cache(&mv, p.v, c, box);
    }
    if (!mapped) return cudaErrorInvalidValue;
    constexpr auto kernel = [] {
      if constexpr (kIsWide<C>) return attn_wide_kernel<C, TREE>;
      else return attn_tc_kernel<C, TREE>;
    }();
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(grid), dim3(C::THREADS), C::SMEM, stream, p, mk, mv, box);
  } else {
    static_assert(C::SMEM + 4 * C::KT * 8 + 8 * C::ROWS + 128 <= 227 * 1024, "shared memory");
    static_assert((C::WK + 1) * C::ROWS * C::D * 4 + C::ROWS * 8 <= C::SMEM, "a piece fits");
    const int split = short_split<C>(c, p);
    if (split) {
      e = cudaFuncSetAttribute(attn_kernel<C, true, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM);
      if (e != cudaSuccess) return e;
      const unsigned items = (unsigned)(p.n_seqs * p.H_kv * (int)p.row_blocks.d);
      return launch_pdl_cluster(split, attn_kernel<C, true, TREE>, dim3(items * split), dim3(C::THREADS),
                                C::SMEM, stream, p, split);
    }
    e = cudaFuncSetAttribute(attn_kernel<C, false, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attn_kernel<C, false, TREE>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, p, 1);
  }
  if constexpr (kIsWide<C>) {
    const int groups = grid / (int)p.row_blocks.d, rows = p.T * (int)p.G.d;
    if (e != cudaSuccess || groups == 1) return e;
    const dim3 joins(p.joins, (rows + 7) / 8);
    // as below
    if (groups > 32LL * p.n_seqs * p.H_kv)
      return launch_pdl(join_wide_kernel<C, 4>, joins, dim3(512), 0, stream, p, groups);
    return launch_pdl(join_wide_kernel<C, 1>, joins, dim3(128), 0, stream, p, groups);
  }
  if (e != cudaSuccess || grid == 1) return e;
  const int rows = p.row_blocks.d > 1 ? C::ROWS : p.T * (int)p.G.d;
  const long long items = (long long)p.n_seqs * p.H_kv * p.row_blocks.d;
  auto join = [&](auto kernel, int warps) {
    return launch_pdl(kernel, dim3(p.joins, rows), dim3(32 * warps), 0, stream, p, grid);
  };
  // pieces of an item that 4 warps would take in many rounds (one sequence of
  // 60000 tokens, 2 kv heads, 152 pieces: 22.8 us with 16 warps, 27.9 with 4;
  // 8 sequences of 20000, 19 pieces: 35.6 and 34.8)
  if (grid > 32 * items) return join(join_kernel<typename C::In, C::D, C::ROWS, 16>, 16);
  return join(join_kernel<typename C::In, C::D, C::ROWS, 4>, 4);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <bool TREE>
size_t workspace_size(const KvLayout &c, int n_seqs, int T, int H, int max_pages) {
  const int rows = T * (H / c.H_kv);
  return with_cfg<TREE>(c, rows, [&](auto cfg) -> size_t {
    using C = decltype(cfg);
    const int row_blocks = (rows + C::ROWS - 1) / C::ROWS;
    size_t g = (size_t)grid_of<C>(c, n_seqs, max_pages, row_blocks);
    if (kIsWide<C> && (int)g == row_blocks) g = 1;  // one group: no item is cut
    return up256(g * 16) + up256(g * 2 * C::ROWS * 8) + g * 2 * C::ROWS * c.D * 4;
  });
}

template <bool TREE>
cudaError_t launch_attention(const AttnArgs &a, cudaStream_t stream) {
  const KvLayout &c = a.cache;
  const int rows = a.T * (a.H / c.H_kv);
  AttnParams p{};
  p.q = a.q; p.k = a.k_cache; p.v = a.v_cache; p.out = a.out;
  p.table = a.table; p.lens = a.lens; p.n_nodes = a.n_nodes; p.tree = a.tree;
  p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
  p.n_seqs = a.n_seqs; p.T = a.T; p.H = a.H; p.H_kv = c.H_kv;
  p.n_pages = c.n_pages; p.max_pages = a.max_pages;
  p.page_size = FastDiv(c.page_size);
  p.G = FastDiv(a.H / c.H_kv);
  p.grouped = a.grouped;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.err = a.err;
  return with_cfg<TREE>(c, rows, [&](auto cfg) -> cudaError_t {
    using C = decltype(cfg);
    p.row_blocks = FastDiv((rows + C::ROWS - 1) / C::ROWS);
    const int grid = grid_of<C>(c, a.n_seqs, a.max_pages, (int)p.row_blocks.d);
    const long long items = (long long)a.n_seqs * c.H_kv * p.row_blocks.d;
    // By block, a join's empty places are left again after one read, and its
    // others lie evenly on the SMs (64 sequences of 512 to 8192, one row block
    // of 8: 52.6 us, 53.7 by item), until they are more than the GPU holds at
    // once (8 sequences of 30k to 65k, 64 rows: 144 us, 137.5 by item).
    const long long by_block = (long long)grid * (p.row_blocks.d > 1 ? C::ROWS : rows);
    p.by_item = items <= grid && by_block > 16 * kSms;
    p.joins = p.by_item ? (int)items : grid;
    if constexpr (kIsWide<C>) {
      const int groups = grid / (int)p.row_blocks.d;
      p.by_item = (long long)a.n_seqs * c.H_kv <= groups;
      p.joins = p.by_item ? a.n_seqs * c.H_kv : groups;
    }
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    p.cut = reinterpret_cast<int4 *>(ws);
    ws += up256((size_t)grid * 16);
    p.part_ml = reinterpret_cast<float2 *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + up256((size_t)grid * 2 * C::ROWS * 8));
    return launch_cfg<C, TREE>(p, c, grid, stream);
  });
}

}  // namespace
}  // namespace gdn
