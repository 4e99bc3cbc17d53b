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
// each node would write as many states as there are nodes).
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

constexpr int kThreads = 128;
constexpr int kCols = 64;  // columns of the state in a block

// Block: one sequence, head and 64 columns.
template <typename T, int DK, int DV, bool KDA>
__global__ void __launch_bounds__(kThreads) tree_forward_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int PER = DK / 32;             // elements of a lane
  constexpr int GROUPS = kThreads / kCols; // threads of a column
  extern __shared__ __align__(16) float sm[];
  __shared__ u64 words[64];
  __shared__ int depth[64], bad, most;
  __shared__ float root[64], beta[64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % (DV / kCols), sh = blockIdx.x / (DV / kCols);
  const int h = sh % p.H, s = sh / p.H, NT = p.T;
  float *kf = sm, *qf = kf + NT * DK, *al = qf + NT * DK;
  float *kc = KDA ? al + NT * DK : kf, *qc = KDA ? kc + NT * DK : qf;
  float *ck = (KDA ? qc + NT * DK : al + NT), *cq = ck + NT * NT;
  float *d = cq + NT * NT, *uq = d + NT * kCols;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int nodes = p.n_nodes ? p.n_nodes[s] : NT;
  if (tid == 0) bad = nodes < 0 || nodes > NT, most = 0;
  nodes = min(max(nodes, 0), NT);
  if (tid < nodes) words[tid] = p.tree[(long long)s * NT + tid];
  __syncthreads();
  const long long t0 = (long long)s * NT;
  if (tid < nodes) {
    const u64 w = words[tid], up = w & ~(1ull << tid);
    const int parent = up ? 63 - __clzll(up) : -1;
    if (!(w >> tid & 1) || parent >= tid || (parent >= 0 && words[parent] != up)) bad = 1;
    depth[tid] = __popcll(up);
    atomicMax(&most, depth[tid]);
    beta[tid] = p.beta[(t0 + tid) * p.H + h];
    if (!KDA) al[tid] = expf(p.g[(t0 + tid) * p.H + h]);
  }
  const int hq = qk_head(p, h);
  for (int e = tid; e < nodes * DK; e += kThreads) {
    const int t = e / DK, i = e % DK;
    const long long at = ((t0 + t) * p.Hqk + hq) * DK + i;
    kf[e] = to_f32(static_cast<const T *>(p.k)[at]);
    qf[e] = to_f32(static_cast<const T *>(p.q)[at]);
    if (KDA) al[e] = expf(p.g[((t0 + t) * p.H + h) * DK + i]);
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) set_error(p.err, kDevBadTree);
    return;
  }
  // products of keys along each node's path, and the decay from the root
  for (int t = warp; t < nodes; t += kThreads / 32) {
    float kt[PER], qt[PER], w[PER];
#pragma unroll
    for (int m = 0; m < PER; ++m) {
      kt[m] = kf[t * DK + m * 32 + lane];
      qt[m] = qf[t * DK + m * 32 + lane];
      w[m] = 1.f;
    }
    u64 left = words[t];
    while (left) {
      const int j = 63 - __clzll(left);
      left &= ~(1ull << j);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int m = 0; m < PER; ++m) {
        const float x = w[m] * kf[j * DK + m * 32 + lane];
        a = fmaf(kt[m], x, a);
        b = fmaf(qt[m], x, b);
        w[m] *= KDA ? al[j * DK + m * 32 + lane] : al[j];
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
      }
      if (lane == 0) {
        ck[t * NT + j] = a;
        cq[t * NT + j] = b;
      }
    }
    if (KDA) {
#pragma unroll
      for (int m = 0; m < PER; ++m) {
        kc[t * DK + m * 32 + lane] = kt[m] * w[m];
        qc[t * DK + m * 32 + lane] = qt[m] * w[m];
      }
    }
    if (lane == 0) root[t] = KDA ? 1.f : w[0];
  }
  __syncthreads();
  // S_0^T of the keys and queries
  const int c = tid % kCols, grp = tid / kCols, col = part * kCols + c;
  const float *S = p.state_in[s];
  if (S) S += (long long)h * DK * DV + col;
  for (int base = grp * 4; base < nodes; base += 4 * GROUPS) {
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    const int n = min(4, nodes - base);
    if (S) {
      for (int i = 0; i < DK; ++i) {
        const float x = S[(long long)i * DV];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = base + (j < n ? j : 0);
          a[j] = fmaf(x, kc[t * DK + i], a[j]);
          b[j] = fmaf(x, qc[t * DK + i], b[j]);
        }
      }
    }
    for (int j = 0; j < n; ++j) {
      d[(base + j) * kCols + c] = a[j] * root[base + j];
      uq[(base + j) * kCols + c] = b[j] * root[base + j];
    }
  }
  __syncthreads();
  // d, one depth after the other
  const T *v = static_cast<const T *>(p.v);
  for (int level = 0; nodes > 0 && level <= most; ++level) {
    for (int t = grp; t < nodes; t += GROUPS) {
      if (depth[t] != level) continue;
      float u = d[t * kCols + c];
      u64 left = words[t] & ~(1ull << t);
      while (left) {
        const int j = __ffsll(left) - 1;
        left &= left - 1;
        u = fmaf(ck[t * NT + j], d[j * kCols + c], u);
      }
      d[t * kCols + c] = beta[t] * (to_f32(v[((t0 + t) * p.H + h) * DV + col]) - u);
    }
    __syncthreads();
  }
  for (int t = grp; t < NT; t += GROUPS) {
    float o = 0.f, x = 0.f;
    if (t < nodes) {
      o = uq[t * kCols + c];
      u64 left = words[t];
      while (left) {
        const int j = __ffsll(left) - 1;
        left &= left - 1;
        o = fmaf(cq[t * NT + j], d[j * kCols + c], o);
      }
      o *= p.scale;
      x = d[t * kCols + c];
    }
    const long long at = ((t0 + t) * p.H + h) * DV + col;
    p.out[at] = o;
    p.updates[at] = x;
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

template <typename T, int DK, int DV, bool KDA>
cudaError_t forward(const TreeParams &p, cudaStream_t stream) {
  const int n = p.T;
  const int smem = 4 * (n * DK * (KDA ? 5 : 2) + (KDA ? 0 : n) + 2 * n * n + 2 * n * kCols);
  const cudaError_t e =
      cudaFuncSetAttribute(tree_forward_kernel<T, DK, DV, KDA>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * 64 * (DK * 5 + 2 * 64 + 2 * kCols));
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_forward_kernel<T, DK, DV, KDA>,
                    dim3((unsigned)(p.n_seqs * p.H * (DV / kCols))), dim3(kThreads), smem, stream, p);
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

// Calls f with the configuration of a call's types, head sizes and gates.
template <typename T, int DK, int DV, bool KDA_>
struct Form {
  using In = T;
  static constexpr int Dk = DK, Dv = DV;
  static constexpr bool KDA = KDA_;
};
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
    return forward<typename F::In, F::Dk, F::Dv, F::KDA>(tree_params(a), stream);
  });
}

cudaError_t launch_tree_commit(const TreeDeltaArgs &a, cudaStream_t stream) {
  return with_form(a, [&](auto f) {
    using F = decltype(f);
    return commit<typename F::In, F::Dk, F::Dv, F::KDA>(tree_params(a), stream);
  });
}

}  // namespace gdn
