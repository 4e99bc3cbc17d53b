// tree_delta.cu -- the gated delta rule along every branch of a tree of drafted
// tokens, and the state after the branch that was accepted.
//
// With c(t, j) the product of the decays on the way from ancestor j (not
// itself) down to node t, and c(t) that from the root on, node t's state is
//   S_t = c(t) S_0 + sum over ancestors j and t of (c(t, j) k_j) d_j^T
// so that no state but the first is needed:
//   d_t = beta_t (v_t - S_0^T (c(t) k_t) - sum_{ancestors j} [k_t . c(t, j) k_j] d_j)
//   o_t = scale (S_0^T (c(t) q_t) + sum_{ancestors j, t} [q_t . c(t, j) k_j] d_j)
// Decays are multiplied up the path, never divided: a gate of -inf is a
// product of 0, and no range of gates is out of reach.
//
// Bound by HBM: the first state is read once (the token loop with a slot for
// each node would write as many states as there are nodes). Heads of 128 x 128 on one
// GB300 (bytes at the copy rate in brackets): 32 sequences x 16 heads x 8 nodes, bf16,
// one decay a head 16.9 us (6.0); 64 x 32 x 32 nodes, a decay for each row of
// the state, 151 us (42). From 34 and 981 with the state through the CUDA cores;
// with it on the matrix instruction 186, with keys by asynchronous copies 157. 32
// nodes are taken at a time: 16 would read and split the state twice.
// The rest is the chain in a block: words, products of keys, products with the
// state, the levels of the tree (some 450 cycles each), and the dots along the
// paths where decays have rows. The commit: 32 x 16 states of 8 nodes 14.5 us
// (10.1), 128 x 32 of 32 nodes 107 (86.0).
#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.cuh"

namespace gdn {
namespace {

using u64 = unsigned long long;

struct TreeParams {
  const void *q, *k, *v;
  const float *g, *beta;
  const float *const *state_in;
  const int32_t *n_nodes, *leaf;
  const u64 *tree;
  float *out, *updates, *state_out;
  int n_seqs, T, H, Hqk, grouped;
  float scale;
  int *err;
};

__device__ __forceinline__ int qk_head(const TreeParams &p, int h) {
  return p.grouped ? h / (p.H / p.Hqk) : h % p.Hqk;
}

// Loads of matrix fragments, and the products of 16 x 16 by 16 x 8 of a warp.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
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

// Two numbers as three bf16 parts each (8 bits of each number in turn: together
// its 24, whatever the size of others), packed in pairs.
__device__ __forceinline__ void split(float x, float y, uint32_t (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    part[i] = pack_bf16(x, y);
    x -= __uint_as_float(part[i] << 16);
    y -= __uint_as_float(part[i] & 0xffff0000u);
  }
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 *u, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(u[i].x); v[4 * i + 1] = __uint_as_float(u[i].y);
      v[4 * i + 2] = __uint_as_float(u[i].z); v[4 * i + 3] = __uint_as_float(u[i].w);
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "n"(BYTES));
}
// Blocks that run at a time: two of an SM, one beyond some 40 nodes with operands in
// parts. (There 152 instead measured the same: 32 x 32 x 64 nodes 242 us.)
constexpr int kBlocksAtOnce = 2 * 152;

// N consecutive elements of shared memory as fp32.
template <int N>
__device__ __forceinline__ void get(const __nv_bfloat16 *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p + i);
    v[i] = __uint_as_float(u << 16);
    v[i + 1] = __uint_as_float(u & 0xffff0000u);
  }
}
template <int N>
__device__ __forceinline__ void get(const float *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 u = *reinterpret_cast<const float2 *>(p + i);
    v[i] = u.x;
    v[i + 1] = u.y;
  }
}

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

// Sizes of a block's shared memory, in bytes, for n nodes.
template <typename T_, int DK_, int DV_, bool KDA_>
struct Form {
  using In = T_;
  static constexpr int DK = DK_, DV = DV_;
  static constexpr bool KDA = KDA_;
  // rows of c k and c q: bf16 keys are their own operand (the scalar c is
  // multiplied afterwards), against the three parts of the state; otherwise three
  // parts of their own against those
  static constexpr bool kPlain = sizeof(In) == 2 && !KDA;
  static constexpr int PARTS = kPlain ? 1 : 3;
  static constexpr int PITCH = DK * 2 + 16;  // of an operand's row: conflict-free ldmatrix
  static constexpr int UP = DV + 4;          // of a row of sums, in floats
  static constexpr int THREADS = DV * 2;     // a warp: 32 columns of one half of the rows
  __host__ __device__ static constexpr int larger(int a, int b) { return a > b ? a : b; }
  // queries follow the keys; tiles of 16 rows start at either
  __host__ __device__ static constexpr int rows(int n) {
    return larger((2 * n + 15) / 16 * 16, n + (n + 15) / 16 * 16);
  }
  __host__ __device__ static constexpr int operand(int n) { return rows(n) * PITCH; }
  __host__ __device__ static constexpr int raw(int n) {  // keys, queries and decays
    return kPlain ? 0 : n * DK * (2 * (int)sizeof(In) + (KDA ? 4 : 0));
  }
  __host__ __device__ static constexpr int sums(int n) { return 4 * 2 * n * UP; }
  // the sums take the place of the raw rows
  __host__ __device__ static constexpr int smem(int n) {
    return PARTS * operand(n) + larger(raw(n), sums(n)) + 4 * n * (n + 1);
  }
};

// Block: one sequence and head.
//  * What needs the tree alone comes first, while the state is on its way to
//    L2: the products of keys along the paths (bf16 keys and one decay a head:
//    all of them on the matrix instruction; else one path a warp, decays
//    multiplied on the way), and the operands c k and c q.
//  * Then S_0^T (c k), S_0^T (c q): a warp takes 32 columns and half of the
//    rows of the state, straight from memory into fragments (a lane's 16 bytes
//    are one row's columns of four products), and splits each element into three
//    bf16 parts that hold its own 24 bits: a sum is as exact beside large elements
//    as without them. (Two fp16 parts under one scale for a warp's elements took 139
//    us for 151 on the second case above, and lost what is small beside the largest.)
//    Of a product's nine pairs of parts the three below 2^-23 of it are left out.
//  * d then goes from the root downwards, nodes of one depth together; a warp
//    has 16 columns, which need no other warp.
// TILES: of 16 rows of the operands taken at once; 1 (up to 8 nodes): keys and
// queries in one.
template <class F, int TILES>
__global__ void __launch_bounds__(F::THREADS, 2) tree_forward_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using T = typename F::In;
  constexpr int DK = F::DK, DV = F::DV, THREADS = F::THREADS, WARPS = THREADS / 32, UP = F::UP;
  constexpr bool KDA = F::KDA;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ u64 words[64];
  __shared__ float root[64], beta[64], alpha[64];  // root: bf16 keys' c(t)
  __shared__ int depth[64], order[64], level_end[65], bad;
  __shared__ alignas(4) unsigned char path[64][64];  // ancestors, the parent first
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.H, s = blockIdx.x / p.H, NT = p.T;
  const long long t0 = (long long)s * NT;
  const int hq = qk_head(p, h);
  const T *vt = static_cast<const T *>(p.v) + (t0 * p.H + h) * DV;  // node t: + t * H * DV
  const long long v_step = (long long)p.H * DV;
  const int op_bytes = F::operand(NT);
  unsigned char *const op = smem;  // [part][k rows, then q rows]
  T *const raw_k = reinterpret_cast<T *>(smem + F::PARTS * op_bytes), *const raw_q = raw_k + NT * DK;
  float *const raw_a = reinterpret_cast<float *>(raw_q + NT * DK);
  float *const uk = reinterpret_cast<float *>(raw_k), *const uq = uk + NT * UP;  // uk becomes d
  float *const ck = reinterpret_cast<float *>(smem + F::PARTS * op_bytes +
                                              F::larger(F::raw(NT), F::sums(NT)));
  float *const cq = ck + NT * (NT + 1) / 2;  // row t: [0, t], from t (t + 1) / 2 on
  auto tri = [](int t) { return t * (t + 1) / 2; };

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // keys, queries and gates on their way to shared memory (padding too: nothing
  // reads it)
  constexpr int VE = 16 / (int)sizeof(T), VECS = DK / VE;
  for (int e = tid; e < 2 * NT * VECS; e += THREADS) {
    const int r = e / VECS, c = e % VECS * VE, t = r < NT ? r : r - NT;
    const T *src = static_cast<const T *>(r < NT ? p.k : p.q) + ((t0 + t) * p.Hqk + hq) * DK + c;
    cp_async16(F::kPlain ? smem_u32(op + r * F::PITCH + c * 2) : smem_u32(raw_k + r * DK + c), src);
  }
  if constexpr (KDA)
    for (int e = tid; e < NT * (DK / 4); e += THREADS) {
      const int t = e / (DK / 4), c = e % (DK / 4) * 4;
      cp_async16(smem_u32(raw_a + t * DK + c), p.g + ((t0 + t) * p.H + h) * DK + c);
    }
  const float *S = p.state_in[s];
  int n = p.n_nodes ? p.n_nodes[s] : NT;
  if (tid < NT) {
    const u64 w = p.tree[t0 + tid];
    const float b = p.beta[(t0 + tid) * p.H + h], g = KDA ? 0.f : p.g[(t0 + tid) * p.H + h];
    asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + tid * v_step));
    if (DV * sizeof(T) > 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + tid * v_step + DV / 2));
    if (DV * sizeof(T) > 256) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + tid * v_step + DV / 4));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + tid * v_step + 3 * DV / 4));
    }
    words[tid] = w;
    beta[tid] = b;
    if (!KDA) alpha[tid] = expf(g);
  }
  if (tid == 0) bad = n < 0 || n > NT;
  n = min(max(n, 0), NT);
  // the state's first fragments to registers, the rest to L2
  constexpr int COLS = DV / 32, HALF = DK / 2, KS = HALF / 16;
  // Steps of the state in registers. Where 32 nodes meet operands in parts, a second
  // one makes a lane spill (64 x 32 x 32 nodes, fp32, row gates: 185 us, 170 with one).
  constexpr int AHEAD = TILES == 1 ? KS : TILES == 4 && !F::kPlain ? 1 : 2;
  const int col0 = warp % COLS * 32, half = warp / COLS;
  if (S) S += (long long)h * DK * DV;
  const float *mine = S ? S + (long long)(half * HALF + (lane & 3) * 2) * DV + col0 + (lane >> 2) * 4
                        : nullptr;
  float4 x[AHEAD][4];
  auto load = [&](int ks) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[ks % AHEAD][i] = ld_stream_f4(mine + (long long)(ks * 16 + (i >> 1) * 8 + (i & 1)) * DV);
  };
  if (S) {
#pragma unroll
    for (int ks = 0; ks < AHEAD; ++ks) load(ks);
    if (AHEAD < KS && tid == 0) prefetch_l2<DK * DV * 4>(S);
  }
  // and to L2 the state of a block that starts when this one ends: without it
  // all blocks that run at a time load together and then compute together
  if (tid == THREADS - 1 && blockIdx.x + kBlocksAtOnce < gridDim.x) {
    const int b = blockIdx.x + kBlocksAtOnce;
    const float *later = p.state_in[b / p.H];
    if (later) prefetch_l2<DK * DV * 4>(later + (long long)(b % p.H) * DK * DV);
  }
  __syncthreads();

  // the tree: its words have to be those of a tree; nodes in order of depth
  if (tid < n) {
    const u64 w = words[tid], up = w & ~(1ull << tid);
    const int parent = up ? 63 - __clzll(up) : -1;
    if (!(w >> tid & 1) || parent >= tid || (parent >= 0 && words[parent] != up)) bad = 1;
    depth[tid] = __popcll(up);
    int l = 0;
    for (u64 left = up; left; ++l) {
      const int j = 63 - __clzll(left);
      left &= ~(1ull << j);
      path[tid][l] = (unsigned char)j;
    }
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) set_error(p.err, kDevBadTree);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  if (tid < n) {
    int before = 0, shallower = 0;
    for (int t = 0; t < n; ++t) {
      shallower += depth[t] < depth[tid];
      before += depth[t] < depth[tid] || (depth[t] == depth[tid] && t < tid);
    }
    order[before] = tid;
    if (before == n - 1) level_end[depth[tid]] = n;
    if (before == shallower && depth[tid] > 0) level_end[depth[tid] - 1] = before;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (KDA)  // each thread what it has brought itself
    for (int e = tid; e < NT * (DK / 4); e += THREADS) {
      float4 *at = reinterpret_cast<float4 *>(raw_a) + e;
      const float4 g = *at;
      *at = make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
    }
  __syncthreads();

  if constexpr (F::kPlain) {
    // all products of keys (and queries) with keys
    const uint32_t op_s = smem_u32(op);
    const int mt = (2 * NT + 15) / 16, nt = (n + 15) / 16;
    for (int tile = warp; tile < mt * nt; tile += WARPS) {
      const int m0 = tile / nt * 16, n0 = tile % nt * 16;
      float g[4][4] = {};  // two chains of each half
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t a[4], b[4];
        ldsm4(a, op_s + (m0 + (lane & 15)) * F::PITCH + (ks * 16 + (lane >> 4) * 8) * 2);
        ldsm4(b, op_s + (n0 + (lane & 7) + ((lane >> 4) << 3)) * F::PITCH +
                     (ks * 16 + ((lane >> 3) & 1) * 8) * 2);
        mma16816(g[ks & 2], a, b[0], b[1]);
        mma16816(g[(ks & 2) + 1], a, b[2], b[3]);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int r = m0 + (lane >> 2) + (x & 2) * 4, j = n0 + (x >> 2) * 8 + (lane & 3) * 2 + (x & 1);
        const int t = r < NT ? r : r - NT;
        if (t < n && j <= t) (r < NT ? ck : cq)[tri(t) + j] = g[x >> 2][x & 3] + g[2 + (x >> 2)][x & 3];
      }
    }
    __syncthreads();
    if (tid < n) {
      float w = alpha[tid];
      const int len = depth[tid];
      float *const k_row = ck + tri(tid), *const q_row = cq + tri(tid);
      for (int l = 0; l < len; l += 4) {
        const uint32_t js = *reinterpret_cast<const uint32_t *>(&path[tid][l]);
        float a[4], x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = l + i < len ? js >> (8 * i) & 0xff : tid;
          a[i] = alpha[j];
          x[i] = k_row[j];
          y[i] = q_row[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (l + i >= len) break;
          const int j = js >> (8 * i) & 0xff;
          k_row[j] = x[i] * w;
          q_row[j] = y[i] * w;
          w *= a[i];
        }
      }
      root[tid] = w;
    }
  } else {
    // one path a warp
    constexpr int PER = DK / 32;
    for (int t = warp; t < n; t += WARPS) {
      float kt[PER], qt[PER], w[PER];
      get(raw_k + t * DK + lane * PER, kt);
      get(raw_q + t * DK + lane * PER, qt);
#pragma unroll
      for (int i = 0; i < PER; ++i) w[i] = 1.f;
      u64 left = words[t];
      while (left) {
        // four ancestors at a time: eight sums, folded over the lanes
        float sum[8];
        int js[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = left ? 63 - __clzll(left) : -1;
          js[x] = j;
          float2 a = {0.f, 0.f}, b = a;
          if (j >= 0) {
            left &= ~(1ull << j);
            float kj[PER], aj[PER];
            get(raw_k + j * DK + lane * PER, kj);
            if constexpr (KDA) get(raw_a + j * DK + lane * PER, aj);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
              float2 c = {w[i], w[i + 1]};
              const float2 y = mul2(c, float2{kj[i], kj[i + 1]});
              a = fma2(float2{kt[i], kt[i + 1]}, y, a);
              b = fma2(float2{qt[i], qt[i + 1]}, y, b);
              c = mul2(c, KDA ? float2{aj[i], aj[i + 1]} : float2{alpha[j], alpha[j]});
              w[i] = c.x;
              w[i + 1] = c.y;
            }
          }
          sum[x] = a.x + a.y;
          sum[4 + x] = b.x + b.y;
        }
#pragma unroll
        for (int half = 4; half; half >>= 1) {
#pragma unroll
          for (int x = 0; x < half; ++x) {
            const bool up = lane & half;
            const float give = up ? sum[x] : sum[x + half], keep = up ? sum[x + half] : sum[x];
            sum[x] = keep + __shfl_xor_sync(0xffffffffu, give, half);
          }
        }
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 8);
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 16);
        // lane x has sum x
        const int j = lane & 2 ? (lane & 1 ? js[3] : js[2]) : (lane & 1 ? js[1] : js[0]);
        if (lane < 8 && j >= 0) (lane < 4 ? ck : cq)[tri(t) + j] = sum[0];
      }
      // the operands: c k and c q in parts
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
          uint32_t part[3];
          split((x ? qt[i] : kt[i]) * w[i], (x ? qt[i + 1] : kt[i + 1]) * w[i + 1], part);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint32_t *>(op + k * op_bytes + (x * NT + t) * F::PITCH +
                                          (lane * PER + i) * 2) = part[k];
        }
      }
    }
  }
  __syncthreads();

  // ---- S_0^T of the operands, 16 or 32 nodes at a time: GROUPS tiles of keys, then of
  // queries
  constexpr int GROUPS = TILES == 4 ? 2 : 1;
  const uint32_t op_s = smem_u32(op);
  for (int c0 = 0; c0 < n; c0 += 16 * GROUPS) {
    float acc[TILES][4][4] = {};
    if (S) {
      if (c0 > 0) {
#pragma unroll
        for (int ks = 0; ks < AHEAD; ++ks) load(ks);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const float4 (&xs)[4] = x[ks % AHEAD];
        // column product i, k pair y: parts
        uint32_t b[4][2][3];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 &lo = xs[2 * y], &hi = xs[2 * y + 1];
          split(lo.x, hi.x, b[0][y]);
          split(lo.y, hi.y, b[1][y]);
          split(lo.z, hi.z, b[2][y]);
          split(lo.w, hi.w, b[3][y]);
        }
        if (ks + AHEAD < KS) load(ks + AHEAD);
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
          const int g0 = c0 + m % GROUPS * 16;
          if (GROUPS > 1 && g0 >= n) continue;
          const uint32_t at = op_s + (g0 + m / GROUPS * NT + (lane & 15)) * F::PITCH +
                              (half * HALF + ks * 16 + (lane >> 4) * 8) * 2;
#pragma unroll
          for (int pa = 0; pa < F::PARTS; ++pa) {
            uint32_t a[4];
            ldsm4(a, at + pa * op_bytes);
#pragma unroll
            for (int pb = 0; pb < 3 - pa; ++pb) {
#pragma unroll
              for (int i = 0; i < 4; ++i) mma16816(acc[m][i], a, b[i][0][pb], b[i][1][pb]);
            }
          }
        }
      }
    }
    // a lane's 8 columns of rows lane / 4 and + 8: the halves of the state are added
    // in turn; the values come while the other half writes
    constexpr int VL = 8 * (int)sizeof(T) / 16;
    uint4 vs[GROUPS][2][VL];
    if (half == 0) {
#pragma unroll
      for (int m = 0; m < GROUPS; ++m)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = min(c0 + m * 16 + (lane >> 2) + 8 * y, n - 1);
          const uint4 *from =
              reinterpret_cast<const uint4 *>(vt + t * v_step + col0 + (lane & 3) * 8);
#pragma unroll
          for (int i = 0; i < VL; ++i) vs[m][y][i] = from[i];
        }
    }
#pragma unroll
    for (int turn = 1; turn >= 0; --turn) {
      if (half == turn) {
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int r = (lane >> 2) + 8 * y;
            int t = c0 + m % GROUPS * 16 + r, is_q = m / GROUPS;
            if (TILES == 1) {
              is_q = r >= NT;
              t = is_q ? r - NT : r;
            }
            if (t >= n) continue;
            const int c = col0 + (lane & 3) * 8;
            float *dst = (is_q ? uq : uk) + t * UP + c;
            float o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[i] = acc[m][i][2 * y];
              o[4 + i] = acc[m][i][2 * y + 1];
            }
            float4 *d4 = reinterpret_cast<float4 *>(dst);
            if (turn == 0) {
              const float w = F::kPlain ? root[t] : 1.f;
              const float4 u0 = d4[0], u1 = d4[1];
              o[0] = (o[0] + u0.x) * w; o[1] = (o[1] + u0.y) * w;
              o[2] = (o[2] + u0.z) * w; o[3] = (o[3] + u0.w) * w;
              o[4] = (o[4] + u1.x) * w; o[5] = (o[5] + u1.y) * w;
              o[6] = (o[6] + u1.z) * w; o[7] = (o[7] + u1.w) * w;
              if (!is_q) {
                float v[8];
                unpack8<T>(vs[m % GROUPS][y], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = v[i] - o[i];
              }
            }
            d4[0] = make_float4(o[0], o[1], o[2], o[3]);
            d4[1] = make_float4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      __syncthreads();
    }
  }

  // ---- d from the root downwards, then o; a warp's 16 columns, 8 nodes at a time
  const int c = warp * 16 + (lane & 3) * 4, slot = lane >> 2;
  // x + sign sum over the ancestors of t of coef[j] d_j
  auto along = [&](float4 x, const float *coef, int t, int len, float sign) {
    for (int l = 0; l < len; l += 4) {
      const uint32_t js = *reinterpret_cast<const uint32_t *>(&path[t][l]);
      // all four at once; beyond the path, the first again by 0
      float w[4];
      float4 d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = js >> (l + i < len ? 8 * i : 0) & 0xff;
        w[i] = l + i < len ? sign * coef[j] : 0.f;
        d[i] = *reinterpret_cast<const float4 *>(uk + j * UP + c);
        if (i > 0 && l + i >= len) d[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.x = fmaf(w[i], d[i].x, x.x);
        x.y = fmaf(w[i], d[i].y, x.y);
        x.z = fmaf(w[i], d[i].z, x.z);
        x.w = fmaf(w[i], d[i].w, x.w);
      }
    }
    return x;
  };
  for (int level = 0, from = 0; from < n; ++level) {
    const int to = level_end[level];
    for (int i = from + slot; i < to; i += 8) {
      const int t = order[i];
      float4 *at = reinterpret_cast<float4 *>(uk + t * UP + c);
      const float4 x = along(*at, ck + tri(t), t, level, -1.f);
      const float b = beta[t];
      *at = make_float4(b * x.x, b * x.y, b * x.z, b * x.w);
    }
    __syncwarp();
    from = to;
  }
  float *const out = p.out + (t0 * p.H + h) * DV + c, *const up = p.updates + (t0 * p.H + h) * DV + c;
  for (int i = slot; i < NT; i += 8) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f), x = o;
    int t = i;
    if (i < n) {
      t = order[i];
      x = *reinterpret_cast<const float4 *>(uk + t * UP + c);
      const float w = cq[tri(t) + t];
      o = *reinterpret_cast<const float4 *>(uq + t * UP + c);
      o = make_float4(fmaf(w, x.x, o.x), fmaf(w, x.y, o.y), fmaf(w, x.z, o.z), fmaf(w, x.w, o.w));
      o = along(o, cq + tri(t), t, depth[t], 1.f);
      o = make_float4(p.scale * o.x, p.scale * o.y, p.scale * o.z, p.scale * o.w);
    }
    st_f4(out + t * v_step, o);
    st_f4(up + t * v_step, x);
  }
}

// Block: one sequence, head and 64 rows of the state, 8 rows of each warp; a
// lane has 4 columns of each.
constexpr int kCommitThreads = 256, kCommitRows = 64;

template <typename T, int DK, int DV, bool KDA>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int LANES = DV / 4, ROWS = kCommitRows / 8 * LANES / 32;  // of a row; rows of a lane
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % (DK / kCommitRows), sh = blockIdx.x / (DK / kCommitRows);
  const int h = sh % p.H, s = sh / p.H, NT = p.T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int leaf = p.leaf[s];
  const long long each = (long long)p.H * DK * DV;
  const float *in = p.state_in[s];
  float *place = p.state_out + s * each;
  const u64 word = leaf >= 0 && leaf < NT ? p.tree[(long long)s * NT + leaf] : 0;
  const bool bad = leaf < -1 || leaf >= NT || (leaf >= 0 && word >> leaf != 1);
  const bool laps = in && in != place && in < p.state_out + p.n_seqs * each &&
                    in + each > p.state_out;
  if (bad || laps) {
    if (tid == 0) set_error(p.err, bad ? kDevBadTree : kDevOverlap);
    return;
  }
  const int n = __popcll(word);
  if (n == 0 && in == place) return;
  float *kk = sm, *al = kk + n * kCommitRows, *dd = al + n * (KDA ? kCommitRows : 1);
  // al and dd start on 16 bytes: n is rounded up for al
  dd = sm + (n * kCommitRows + (KDA ? n * kCommitRows : (n + 3) / 4 * 4));
  const int hq = qk_head(p, h), row0 = part * kCommitRows;
  {
    u64 left = word;
    for (int x = 0; x < n; ++x) {
      const long long tok = (long long)s * NT + __ffsll(left) - 1;
      left &= left - 1;
      if (tid < kCommitRows) {
        kk[x * kCommitRows + tid] =
            to_f32(static_cast<const T *>(p.k)[(tok * p.Hqk + hq) * DK + row0 + tid]);
        if (KDA) al[x * kCommitRows + tid] = expf(p.g[(tok * p.H + h) * DK + row0 + tid]);
        else if (tid == 0) al[x] = expf(p.g[tok * p.H + h]);
      } else if (tid >= 128 && tid - 128 < DV) {
        dd[x * DV + tid - 128] = p.updates[(tok * p.H + h) * DV + tid - 128];
      }
    }
  }
  __syncthreads();
  __shared__ __align__(16) float root[kCommitRows];
  if (tid < kCommitRows) {
    float w = 1.f;
    for (int x = n - 1; x >= 0; --x) {
      kk[x * kCommitRows + tid] *= w;
      w *= KDA ? al[x * kCommitRows + tid] : al[x];
    }
    root[tid] = w;
  }
  __syncthreads();
  const int c = lane % LANES * 4, r0 = warp * 8 + lane / LANES * ROWS;
  const long long at = ((long long)h * DK + row0 + r0) * DV + c;
  float4 st[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    st[r] = in ? *reinterpret_cast<const float4 *>(in + at + r * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float w = root[r0 + r];
    st[r].x *= w; st[r].y *= w; st[r].z *= w; st[r].w *= w;
  }
  for (int x = 0; x < n; ++x) {
    const float4 d = *reinterpret_cast<const float4 *>(dd + x * DV + c);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float w = kk[x * kCommitRows + r0 + r];
      st[r].x = fmaf(w, d.x, st[r].x);
      st[r].y = fmaf(w, d.y, st[r].y);
      st[r].z = fmaf(w, d.z, st[r].z);
      st[r].w = fmaf(w, d.w, st[r].w);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) st_f4(place + at + r * DV, st[r]);
}

template <class F, int TILES>
cudaError_t forward_tiles(const TreeParams &p, cudaStream_t stream) {
  static_assert(F::smem(64) + 8192 <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(
      tree_forward_kernel<F, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::smem(64));
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_forward_kernel<F, TILES>, dim3((unsigned)(p.n_seqs * p.H)),
                    dim3(F::THREADS), F::smem(p.T), stream, p);
}
template <class F>
cudaError_t forward(const TreeParams &p, cudaStream_t stream) {
  return p.T <= 8    ? forward_tiles<F, 1>(p, stream)
         : p.T <= 16 ? forward_tiles<F, 2>(p, stream)
                     : forward_tiles<F, 4>(p, stream);
}

template <typename T, int DK, int DV, bool KDA>
cudaError_t commit(const TreeParams &p, cudaStream_t stream) {
  const int n = p.T, smem = 4 * (n * kCommitRows * (KDA ? 2 : 1) + (n + 3) / 4 * 4 + n * DV);
  const cudaError_t e = cudaFuncSetAttribute(
      tree_commit_kernel<T, DK, DV, KDA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      4 * (64 * kCommitRows * 2 + 64 + 64 * DV));
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_commit_kernel<T, DK, DV, KDA>,
                    dim3((unsigned)(p.n_seqs * p.H * (DK / kCommitRows))), dim3(kCommitThreads),
                    smem, stream, p);
}

// Calls f with the form of a call's types, head sizes and gates.
template <typename T, int DK, int DV, class F>
cudaError_t with_gate(bool kda, F f) {
  return kda ? f(Form<T, DK, DV, true>{}) : f(Form<T, DK, DV, false>{});
}
template <typename T, class F>
cudaError_t with_heads(const TreeDeltaArgs &a, F f) {
  if (a.Dk == 128)
    return a.Dv == 128 ? with_gate<T, 128, 128>(a.kda, f) : with_gate<T, 128, 64>(a.kda, f);
  return a.Dv == 128 ? with_gate<T, 64, 128>(a.kda, f) : with_gate<T, 64, 64>(a.kda, f);
}
template <class F>
cudaError_t with_form(const TreeDeltaArgs &a, F f) {
  return a.bf16 ? with_heads<__nv_bfloat16>(a, f) : with_heads<float>(a, f);
}

TreeParams tree_params(const TreeDeltaArgs &a) {
  TreeParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.beta = a.beta;
  p.state_in = a.state_in; p.n_nodes = a.n_nodes; p.leaf = a.leaf; p.tree = a.tree;
  p.out = a.out; p.updates = a.updates; p.state_out = a.state_out;
  p.n_seqs = a.n_seqs; p.T = a.T; p.H = a.H; p.Hqk = a.Hqk; p.grouped = a.qk_grouped;
  p.scale = a.scale; p.err = a.err;
  return p;
}

}  // namespace

cudaError_t launch_tree_forward(const TreeDeltaArgs &a, cudaStream_t stream) {
  return with_form(a, [&](auto f) {
    using F = decltype(f);
    return forward<F>(tree_params(a), stream);
  });
}

cudaError_t launch_tree_commit(const TreeDeltaArgs &a, cudaStream_t stream) {
  return with_form(a, [&](auto f) {
    using F = decltype(f);
    return commit<typename F::In, F::DK, F::DV, F::KDA>(tree_params(a), stream);
  });
}

}  // namespace gdn
