/*
 * gdn.h -- C ABI of libgdn, the gated delta-net (GDN) recurrence on NVIDIA
 * GB300 (sm_103a).
 *
 * The op. Per sequence s, head h and token t, the D_k x D_v fp32 state S of
 * that head (row i = key index, column j = value index) is
 *   decayed    S <- exp(g) S               (GDA: one gate per head and token)
 *              S[i,:] <- exp(g_i) S[i,:]   (KDA: one gate per key row)
 *   read       u = S^T k
 *   corrected  d = beta (v - u)
 *   written    S <- S + k d^T
 *   queried    o = scale S^T q             (after the write)
 * This is the gated delta rule of "Gated Delta Networks" (Yang, Kautz,
 * Hatamizadeh, ICLR 2025); the op is GGML_OP_GATED_DELTA_NET with the GDA and
 * KDA modes and head sizes 64/128 of "metal : add GDN kernel (#20361)"
 * (llama.cpp commits, tag b9752, src/models/qwen35.cpp). g is a log-decay used
 * as exp(g) with no clamp; beta is used as given (the caller applies any
 * sigmoid); q and k are used as given (the caller normalises them).
 *
 * Snapshots and rollback ("metal: add GDN partial rollback" and "llama: allow
 * partial seq_rm for GDN models for speculative decoding", koboldcpp commits,
 * tag v1.113.1): a forward keeps K = n_slots states per sequence. After token
 * t of a T-token sequence with t >= T-K the state goes to slot t-(T-K), so
 * slot K-1 is the final state and K = 1 is the plain single-state forward.
 * When T < K, slots j < K-T are not written. The input state is a separate
 * buffer and is never written. Rolling back to n accepted tokens is a slot
 * select (gdn_rollback), not a recompute.
 *
 * Conventions for every call below.
 *  - Ownership: the caller allocates and owns every buffer and the stream.
 *    The library allocates no device memory on these calls and never
 *    synchronises the stream, except gdn_check_device_error.
 *  - Layouts: dense, row-major, innermost index last, exactly as written in
 *    each comment; no strides. Ntok is the number of packed tokens.
 *  - Alignment: every device buffer must be 16-byte aligned.
 *  - Supported shapes: D_k, D_v in {64, 128}. Anything else returns
 *    GDN_ERR_UNSUPPORTED; there is no fallback path of any kind.
 *  - Errors: every call returns a gdn_status; gdn_last_error() gives the
 *    calling thread's last message. Kernel launches are asynchronous: a
 *    condition only the device can see (a bad cu_seqlens entry, a bounded
 *    wait that ran out) sets a per-device error word that
 *    gdn_check_device_error reads and clears.
 *  - Streams: gdn_stream_t is a cudaStream_t (NULL = the legacy default).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *gdn_stream_t; /* same type as cudaStream_t */

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,    /* null pointer, bad size, misaligned buffer, overlap */
  GDN_ERR_UNSUPPORTED = 2,    /* valid but not implemented (e.g. D_k = 32) */
  GDN_ERR_ROLLBACK_RANGE = 3, /* the requested state was not stored */
  GDN_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed */
  GDN_ERR_TIMEOUT = 5,        /* a bounded device-side wait ran out */
  GDN_ERR_DEVICE_ARG = 6      /* the device found a bad argument (cu_seqlens, or a
                                 gate range the chunked path cannot represent) */
} gdn_status;

typedef enum { GDN_MODE_GDA = 0, GDN_MODE_KDA = 1 } gdn_mode;
typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

/* Grouped-query heads: q and k may carry H_qk heads for H value heads (H a
 * multiple of H_qk), and the op reads them per value head instead of the
 * caller repeating them ("models : avoid Q and K repeats when using fused
 * GDA", llama.cpp commits page, tag b9752). Value head h reads q/k head
 *   GDN_QK_TILED:   h % H_qk            (heads repeated as a whole block)
 *   GDN_QK_GROUPED: h / (H / H_qk)      (each q/k head repeated in place)
 * Both orders occur ("reorder v heads for linear attention to avoid
 * expensive interleaved repeat", same page, "support qwen3.5 series"). */
typedef enum { GDN_QK_TILED = 0, GDN_QK_GROUPED = 1 } gdn_qk_map;

/* Message of the calling thread's last failed call ("" if none). */
const char *gdn_last_error(void);

/* Version string of the library. */
const char *gdn_version(void);

/* ------------------------------------------------------------------------
 * Uniform-length forward: decode (T = 1) and speculative verify
 * (T = draft_max + 1). Runs the token recurrence on the recurrent kernel.
 * ---------------------------------------------------------------------- */
typedef struct {
  int n_seqs;         /* N >= 0 independent sequences */
  int T;              /* tokens per sequence, >= 0 */
  int H;              /* value heads (v, g, beta, out and the state have H heads) */
  int D_k, D_v;       /* head sizes, each 64 or 128 */
  gdn_dtype in_dtype; /* dtype of q, k, v; g and beta are always fp32 */
  float scale;        /* output scale; 0 means 1/sqrt(D_k) */
  int H_qk;           /* heads of q and k; 0 means H; must divide H */
  gdn_qk_map qk_map;  /* value head -> q/k head when H_qk < H */
} gdn_shape;

/*
 * q, k        device [N*T][H_qk][D_k]  in_dtype (token n*T+t is token t of seq n)
 * v           device [N*T][H][D_v]  in_dtype
 * g           device fp32 [N*T][H] (GDA) or [N*T][H][D_k] (KDA)
 * beta        device fp32 [N*T][H]
 * state_in    device array of N device pointers; state_in[s] -> fp32
 *             [H][D_k][D_v], the state before this call (any slot a rollback
 *             chose). A NULL entry means a zero state. Read only.
 * state_slots device fp32 [N][n_slots][H][D_k][D_v]; slot j of sequence s
 *             receives the state after token T-n_slots+j. No state_in[s] may
 *             point into it: the kernel checks each pointer, leaves that
 *             sequence unwritten and reports GDN_ERR_DEVICE_ARG through
 *             gdn_check_device_error.
 * out         device fp32 [N*T][H][D_v]
 * n_slots     K >= 1
 * Returns GDN_OK once the kernel is enqueued on `stream`.
 * The kernel is a programmatic dependent launch: its blocks may be scheduled
 * while the previous kernel of `stream` is still running, but they read and
 * write no memory until that kernel has completed, so stream order holds for
 * every argument as for an ordinary launch.
 */
gdn_status gdn_forward(const gdn_shape *shape, const void *q, const void *k,
                       const void *v, const float *g, const float *beta,
                       const float *const *state_in, float *state_slots,
                       float *out, int n_slots, gdn_mode mode,
                       gdn_stream_t stream);

/*
 * gdn_forward with the per-token buffers in host memory (no counterpart on
 * the pages): q, k, v, g, beta and out may each be page-locked host memory
 * (cudaMallocHost / cudaHostAlloc / cudaHostRegister, mapped into the
 * device's address space at the same address, as unified addressing does)
 * or device memory. The kernel reads the token rows and writes the outputs
 * over the host link itself, so no separate copy (and no event between a copy
 * stream and the launch stream) stands between consecutive calls; the state
 * pointers and slots stay device memory. Layouts, results (bit for bit) and
 * the programmatic launch are those of gdn_forward.
 * Errors: GDN_ERR_INVALID_ARG when one of the six pointers is pageable host
 * memory or unknown to CUDA (each is checked with cudaPointerGetAttributes
 * before anything is enqueued), otherwise as gdn_forward. The host memory
 * must stay valid and unmodified until the call has completed on `stream`.
 */
gdn_status gdn_forward_host(const gdn_shape *shape, const void *q, const void *k,
                            const void *v, const float *g, const float *beta,
                            const float *const *state_in, float *state_slots,
                            float *out, int n_slots, gdn_mode mode,
                            gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * Varlen chunked prefill ("llama : enable chunked fused GDN path", llama.cpp
 * commits, tag b9752). Sequence s covers packed tokens
 * [cu_seqlens[s], cu_seqlens[s+1]). Routing:
 *  - bf16 inputs with D_k = D_v = 128: tokens [0, L_s - n_slots) of each
 *    sequence run through the chunked (chunk 64, WY/UT-transform)
 *    tensor-core kernels, with the last partial chunk padded by no-op rows;
 *    the last n_slots tokens run through the recurrent kernel, which writes
 *    the slots. With n_slots = 1 the slot is the final state, so every token
 *    runs through the chunked kernels, which write it. The result equals the
 *    token recurrence up to rounding (bf16 tensor-core operands, fp32
 *    accumulation and fp32 state).
 *  - fp32 inputs (whose 1e-5 accuracy bf16 operands cannot meet) and head
 *    sizes of 64: every token runs through the recurrent kernel on the GPU,
 *    as the pages' chunked path also falls back to the token loop ("Enable
 *    GDN also for prefill, move TODO for chunked_GDN", llama.cpp commits).
 * ---------------------------------------------------------------------- */
typedef struct {
  int n_seqs;         /* N >= 1 */
  int total_tokens;   /* Ntok = cu_seqlens[N] */
  int H;              /* value heads */
  int D_k, D_v;       /* each 64 or 128 */
  gdn_dtype in_dtype; /* GDN_BF16 or GDN_F32 (see the routing note below) */
  float scale;        /* 0 means 1/sqrt(D_k) */
  int H_qk;           /* heads of q and k; 0 means H; must divide H */
  gdn_qk_map qk_map;  /* value head -> q/k head when H_qk < H */
} gdn_varlen_shape;

/* Bytes of device workspace gdn_forward_chunked needs for this shape in either
 * gate mode (the per-row gate mode needs more; this is its figure). */
size_t gdn_chunked_workspace_size(const gdn_varlen_shape *shape, int n_slots);

/*
 * cu_seqlens  device int32 [N+1], non-decreasing, cu_seqlens[0] = 0,
 *             cu_seqlens[N] = total_tokens (checked on the device)
 * q, k, v, g, beta, out: as gdn_forward with Ntok = total_tokens (q, k with
 *             H_qk heads)
 * state_in    device array of N device pointers (NULL entry = zero state)
 * state_slots device fp32 [N][n_slots][H][D_k][D_v]
 * workspace   device buffer of at least gdn_chunked_workspace_size bytes,
 *             256-byte aligned; its contents on entry do not matter.
 * Gate range: inside each 64-token chunk the cumulative log-gate from the
 * chunk's first token must stay within [-80, 80] for per-row gates. For
 * scalar gates only growth is limited (no interval of the chunk may grow by
 * more than e^80); any decay is computed, and a gate of -inf resets the state
 * exactly. The chunk form keeps its decay factors e^(+-gamma) in bf16/fp32,
 * whose range ends near e^88. A chunk outside the range (a NaN gate too)
 * leaves its outputs undefined and makes gdn_check_device_error return
 * GDN_ERR_DEVICE_ARG; gdn_forward (the token loop) has no such limit, and
 * the last n_slots tokens of each sequence, which run through it, neither.
 */
gdn_status gdn_forward_chunked(const gdn_varlen_shape *shape,
                               const int32_t *cu_seqlens, const void *q,
                               const void *k, const void *v, const float *g,
                               const float *beta, const float *const *state_in,
                               float *state_slots, float *out, int n_slots,
                               gdn_mode mode, void *workspace,
                               size_t workspace_bytes, gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * Allocation-free chunked prefill. The pages describe no counterpart: this is
 * a convenience of this library. Some callers cannot give the chunked call a
 * workspace because they may not allocate device memory at all: a host
 * application that owns every device byte through its own pool, or a loop
 * that must never pay for a device allocation (cudaMalloc can synchronise the
 * whole device). This entry point computes exactly what gdn_forward_chunked
 * computes, with the same arguments minus the workspace; its scratch is a
 * fixed 256 MiB device array inside the library, which every GPU that loads
 * the chunked kernels holds until the process exits.
 *  - Limit: shapes whose workspace for the given mode exceeds
 *    gdn_noalloc_scratch_bytes() are rejected with GDN_ERR_UNSUPPORTED and a
 *    message naming both sizes. The scalar-gate mode needs about 33 KB per
 *    (chunk of 64 tokens, head), the per-row mode about 65 KB, plus 64 KB of
 *    fp32 state per (sequence, head): 1 x 4096 tokens x 32 heads needs about
 *    140 MB per-row and fits; 8 x ~4k tokens x 16 heads does not.
 *  - The first call on a device looks up the array's device address with
 *    that device current and keeps it for the life of the process; make that
 *    first call before any stream capture. A cudaDeviceReset invalidates the
 *    kept address (as it does the error word's): do not call this entry
 *    point after resetting a device it was used on.
 *  - Every call on a device shares the one array and it keeps the previous
 *    call's contents; nothing in it needs to start at zero (the work list
 *    rewrites what the later kernels read). Calls that can overlap on the
 *    GPU (different streams without ordering) race on it: serialise them.
 *  - It calls no cudaMalloc, cudaFree or other allocating routine.
 * ---------------------------------------------------------------------- */
gdn_status gdn_forward_chunked_noalloc(const gdn_varlen_shape *shape,
                                       const int32_t *cu_seqlens, const void *q,
                                       const void *k, const void *v, const float *g,
                                       const float *beta, const float *const *state_in,
                                       float *state_slots, float *out, int n_slots,
                                       gdn_mode mode, gdn_stream_t stream);

/* Size in bytes of the built-in scratch array of gdn_forward_chunked_noalloc. */
size_t gdn_noalloc_scratch_bytes(void);

/* ------------------------------------------------------------------------
 * Chunked prefill with state checkpoints ("llama-memory: enable
 * checkpointing with partial rollback", koboldcpp commits page, tag
 * v1.113.1): the slots keep only the last n_slots states of a call, so a
 * caller that may later keep fewer tokens (a shared prompt prefix, a
 * rejected continuation) also wants states at regular positions. Computes
 * exactly what gdn_forward_chunked computes and in addition stores
 *   checkpoints[s][m] = state after token (m+1)*ckpt_every - 1 of sequence s
 * (0-based within the sequence) for every m < max_ckpts with
 * (m+1)*ckpt_every <= L_s. Entries a sequence does not reach are not
 * written.
 * checkpoints  device fp32 [N][max_ckpts][H][D_k][D_v], 16-byte aligned;
 *              must not overlap state_in, state_slots or out
 * ckpt_every   positive multiple of 64 (a chunk boundary)
 * max_ckpts    >= 1
 * The other arguments are those of gdn_forward_chunked.
 * ---------------------------------------------------------------------- */
gdn_status gdn_forward_chunked_checkpointed(
    const gdn_varlen_shape *shape, const int32_t *cu_seqlens, const void *q, const void *k,
    const void *v, const float *g, const float *beta, const float *const *state_in,
    float *state_slots, float *out, int n_slots, gdn_mode mode, float *checkpoints,
    int ckpt_every, int max_ckpts, void *workspace, size_t workspace_bytes,
    gdn_stream_t stream);

/*
 * Where to restart a sequence of L tokens, last run with n_slots slots and
 * checkpoints every ckpt_every tokens (max_ckpts of them), that keeps only
 * its first n_keep tokens (0 <= n_keep <= L):
 *   *source = 0: start from that call's state_in and replay tokens
 *                [0, n_keep) (*index = -1, *replay_from = 0);
 *   *source = 1: start from checkpoint *index and replay tokens
 *                [*replay_from, n_keep);
 *   *source = 2: the state is slot *index, nothing to replay
 *                (*replay_from = n_keep).
 * A slot is chosen whenever one holds the state; otherwise the latest
 * checkpoint at or before n_keep. GDN_ERR_INVALID_ARG for bad arguments.
 * Host only.
 */
gdn_status gdn_checkpoint_select(int n_keep, int L, int n_slots, int ckpt_every,
                                 int max_ckpts, int *source, int *index,
                                 int *replay_from);

/* ------------------------------------------------------------------------
 * The attention layer between the recurrent ones. A hybrid model runs full
 * attention every few layers, and a norm and projections around every layer;
 * the calls below are that layer's work for the two shapes gdn_forward serves
 * (T = 1 and T = draft_max + 1). "Every buffer" conventions above hold:
 * dense unless a stride is given, 16-byte aligned, nothing allocated, no
 * synchronisation. Each kernel is a programmatic dependent launch like
 * gdn_forward's: stream order holds as usual.
 * ---------------------------------------------------------------------- */

/*
 * Root-mean-square norm with the residual's addition and an 8-bit output.
 * Per row (all arithmetic and sums in fp32):
 *   h = x + residual                      (residual NULL: h = x)
 *   y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight)
 *                                         (weight NULL: without that factor;
 *                                          normalize = 0: y = h)
 *   scale[b] = max(max |y| over columns [128 b, 128 b + 128) / 448, 2^-100)
 *   fp8      = y / scale[b], rounded to e4m3 (to nearest even, saturating)
 * so y is about fp8 * scale; each of the two quotients is rounded once to fp32.
 * NaNs take no part in the maximum and stay NaN.
 */
typedef struct {
  int rows, cols;      /* rows >= 0, 1 <= cols <= 2^31 - 1024 */
  gdn_dtype dtype;     /* of x, residual, weight, residual_out and out */
  int normalize;       /* 1: as above; 0: y = h (a plain quantiser) */
  float eps;           /* finite, >= 0 */
  float weight_offset; /* 0, or 1 for weights stored around zero */
} gdn_norm_shape;

/*
 * x, residual   device [rows][cols] dtype (residual may be NULL)
 * weight        device [cols] dtype (may be NULL; must be with normalize = 0)
 * residual_out  device [rows][cols] dtype, receives h; may be NULL
 * out           device [rows][cols] dtype, receives y; may be NULL
 * out_fp8       device e4m3 [rows][cols], one byte each
 * out_scale     device fp32 [rows][ceil(cols / 128)]
 *               (both NULL when only `out` is wanted, never one alone)
 * residual_out and out may each be x or residual itself (in place); any
 * other overlap of an output with another buffer is refused.
 */
gdn_status gdn_rmsnorm_fp8(const gdn_norm_shape *shape, const void *x, const void *residual,
                           const void *weight, void *residual_out, void *out, void *out_fp8,
                           float *out_scale, gdn_stream_t stream);

/*
 * Product of two 8-bit matrices with block scales, for example of
 * gdn_rmsnorm_fp8's output and a projection's weights:
 *   out[m][n] = sum_b a_scale[m][b] b_scale[n / 128][b]
 *                     sum_{k in [128 b, 128 b + 128)} a[m][k] b[n][k]
 * on the tensor cores, sums in fp32 (each block's products exactly as the
 * tensor cores add them in fp32, then in fp32 over the blocks), rounded once
 * to out_dtype. Nothing but the order of those sums depends on the sizes.
 */
typedef struct {
  int M, N;            /* >= 0 */
  int K;               /* >= 1, a multiple of 16 (a row starts on 16 bytes) */
  gdn_dtype out_dtype;
} gdn_gemm_shape;

/*
 * a        device e4m3 [M][K];  a_scale  device fp32 [M][ceil(K / 128)]
 * b        device e4m3 [N][K];  b_scale  device fp32 [ceil(N / 128)][ceil(K / 128)]
 * out      device [M][N] out_dtype; overlaps no other buffer
 * The last blocks of N and K may be partial. GDN_ERR_UNSUPPORTED for another K
 * and for sizes above 2^21.
 */
gdn_status gdn_gemm_fp8(const gdn_gemm_shape *shape, const void *a, const float *a_scale,
                        const void *b, const float *b_scale, void *out, gdn_stream_t stream);

/* A key-value cache in pages: token j of a page's page_size tokens, head h:
 *   element p * page_stride + j * token_stride + h * head_stride + d
 * of the k (or v) buffer, for page p. Strides are in elements and multiples
 * of 16 bytes; all three 0 means dense [n_pages][page_size][H_kv][D]. The k
 * and the v buffer share one layout. */
typedef struct {
  int n_pages, page_size; /* >= 0, >= 1 */
  int H_kv;               /* key-value heads */
  int D;                  /* head size: 64, 128 or 256 */
  gdn_dtype dtype;        /* of the cache, and of q, k, v and out with it */
  long long page_stride, token_stride, head_stride;
} gdn_kv_cache;

/* Which elements of a head form the pairs that are rotated: (i, i + rot/2),
 * or the neighbours (2i, 2i + 1). */
typedef enum { GDN_ROPE_HALVES = 0, GDN_ROPE_NEIGHBOURS = 1 } gdn_rope_pairs;

/* Which axis turns frequency i of rot_dim/2, with n_i = section[] frequencies
 * for each axis: one run for each axis in turn, or the axes taking turns
 * (axis a = i % n_axes while i / n_axes < section[a], axis 0 otherwise). */
typedef enum { GDN_ROPE_AXES_SECTIONED = 0, GDN_ROPE_AXES_INTERLEAVED = 1 } gdn_rope_axes;

/*
 * Rotary positions with several axes (time, height, width), and the cache
 * append. For token t, pair i of the first rot_dim elements of every q and k
 * head turns by the angle positions[axis(i)][t] * inv_freq[i]:
 *   (a, b) -> (a cos - b sin, a sin + b cos)
 * and the other elements pass unchanged. The angle is reduced to one turn
 * beyond fp32 (inv_freq up to 1: error below 2e-6 for positions up to 2^24, in
 * proportion to the position beyond), so long positions lose nothing. The
 * rotated q goes to q_out; the rotated k and v go to slot slots[t] of the cache
 * (page slot / page_size, token slot % page_size).
 * A negative slot (padding) writes no cache entry; one beyond the cache is
 * skipped and reported as GDN_ERR_DEVICE_ARG by gdn_check_device_error. Of
 * two tokens with one slot, each element that stays may be either's.
 */
typedef struct {
  int n_tokens;             /* >= 0 */
  int H;                    /* query heads (the cache has the key-value heads) */
  int rot_dim;              /* even, 0 .. D */
  gdn_rope_pairs pairs;
  int n_axes;               /* 1 .. 4 */
  int section[4];           /* frequencies of each axis; they sum to rot_dim / 2 */
  gdn_rope_axes axes;
  long long q_stride, k_stride, v_stride; /* elements between tokens, multiples of 16
                                             bytes; 0 = dense (heads * D) */
} gdn_rope_shape;

/*
 * q          device [n_tokens] rows of [H][D], q_stride apart (k, v: [H_kv][D]),
 *            for example column ranges of one projection's output
 * positions  device int32 [n_axes][n_tokens]
 * inv_freq   device fp32 [rot_dim / 2]
 * slots      device int64 [n_tokens]
 * q_out      device [n_tokens][H][D]; overlaps no other buffer
 * k_cache, v_cache  device buffers of the layout `cache`; no row of one shares
 *            bytes with a row of the other (k and v may alternate in one buffer)
 */
gdn_status gdn_rope_append(const gdn_rope_shape *shape, const gdn_kv_cache *cache, const void *q,
                           const void *k, const void *v, const int32_t *positions,
                           const float *inv_freq, const int64_t *slots, void *q_out,
                           void *k_cache, void *v_cache, gdn_stream_t stream);

/*
 * gdn_rope_append for models that norm every q and k head before the
 * rotation. Per token and head (all arithmetic and sums in fp32, one rounding
 * at the end):
 *   y = x / sqrt(mean(x^2) + eps) * (weight_offset + weight)
 * over the head's D elements; the first rot_dim elements of y are then
 * rotated, the others are written as they are. v is copied.
 */
typedef struct {
  float eps;           /* finite, >= 0 */
  float weight_offset; /* 0, or 1 for weights stored around zero */
} gdn_qk_norm;

/*
 * q_weight, k_weight  device [D], dtype of the cache, for all q and all k
 *            heads; each may be NULL (without that factor)
 * The other arguments are those of gdn_rope_append.
 */
gdn_status gdn_qknorm_rope_append(const gdn_rope_shape *shape, const gdn_kv_cache *cache,
                                  const gdn_qk_norm *norm, const void *q, const void *k,
                                  const void *v, const void *q_weight, const void *k_weight,
                                  const int32_t *positions, const float *inv_freq,
                                  const int64_t *slots, void *q_out, void *k_cache,
                                  void *v_cache, gdn_stream_t stream);

/*
 * Attention of the last T tokens of each sequence over its pages (T = 1:
 * decode; T = draft_max + 1: verify). Sequence s has lens[s] tokens in the
 * cache, the new ones included; its token j is at page
 * page_table[s][j / page_size], token j % page_size. Row t of its T rows
 * stands at position lens[s] - T + t and sees the keys 0 up to itself:
 *   out = sum_j softmax_j(scale q . k_j) v_j
 * with statistics and sums in fp32 (bf16: the probabilities are rounded to
 * bf16 before the product with v). A row that sees no key (lens[s] = 0, or
 * lens[s] < T) is 0. What pages hold beyond lens[s] is not used, whatever it
 * is; a NaN or infinity in v of one of the last T tokens reaches all T rows.
 * Query head h reads kv head h / (H / H_kv) (GDN_QK_GROUPED) or h % H_kv
 * (GDN_QK_TILED).
 * The result does not depend on what ran before, bit for bit: the cache is
 * cut by the lengths alone and the parts are joined in order.
 */
typedef struct {
  int n_seqs;        /* >= 0 */
  int T;             /* new tokens of each sequence, >= 0 */
  int H;             /* query heads, a multiple of the cache's H_kv */
  int max_pages;     /* columns of page_table, >= 0 */
  float scale;       /* 0 means 1/sqrt(D) */
  gdn_qk_map kv_map; /* query head -> kv head */
} gdn_attn_shape;

/* max_pages is also what the call's kernel is chosen by (the lengths are known
 * on the device only): with a table much wider than the longest sequence a short
 * batch takes the form for long ones, which starts some 4 us later. */

/* Bytes of device workspace gdn_paged_attention needs (at most 64 MiB); 0 for
 * arguments that it refuses. Depends on the shapes alone, not on lens. */
size_t gdn_paged_attention_workspace_size(const gdn_attn_shape *shape, const gdn_kv_cache *cache);

/*
 * q           device [n_seqs*T][H][D] (token s*T+t is token t of sequence s)
 * k_cache, v_cache  device buffers of the layout `cache`
 * page_table  device int32 [n_seqs][max_pages]; entries that no token needs
 *             are not read
 * lens        device int32 [n_seqs], 0 <= lens[s] <= max_pages * page_size
 *             and at most 2^30 (a longer one is cut to that, a negative one
 *             is 0)
 * out         device [n_seqs*T][H][D]; overlaps no other buffer
 * workspace   device buffer of at least gdn_paged_attention_workspace_size
 *             bytes, 256-byte aligned; its contents on entry do not matter.
 *             Calls that can overlap on the GPU need one each.
 * A page table entry outside the cache, or a length that was cut, is reported
 * as GDN_ERR_DEVICE_ARG by gdn_check_device_error; nothing out of range is
 * read, and that sequence's output is undefined.
 */
gdn_status gdn_paged_attention(const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                               const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *page_table, const int32_t *lens, void *out,
                               void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * Trees of drafted tokens. A verify step may score several continuations of a
 * sequence at once: its T tokens are the nodes of a tree (of several, if
 * several follow the last accepted token), numbered so that a node comes
 * after its parent. The tree of sequence s is T words of 64 bits:
 *   bit j of tree[s][t]: node j is an ancestor of node t, or t itself
 * so T is at most 64. n_nodes[s] (0 .. T) says how many of the T nodes the
 * sequence has; rows of the others are padding. n_nodes = NULL: all have T.
 * ---------------------------------------------------------------------- */

/* Bytes of device workspace gdn_tree_attention needs (at most 64 MiB); 0 for
 * arguments that it refuses. Depends on the shapes alone. */
size_t gdn_tree_attention_workspace_size(const gdn_attn_shape *shape, const gdn_kv_cache *cache);

/*
 * Attention of the nodes over the sequence's pages. The sequence has lens[s]
 * tokens in the cache, its m = n_nodes[s] nodes being the last of them (node j is
 * token lens[s] - m + j: appended by gdn_rope_append or gdn_qknorm_rope_append
 * with the positions that the nodes' depths give). Node t sees all tokens
 * before the nodes, and those nodes that its word names:
 *   out = sum_j softmax_j(scale q . k_j) v_j
 * Any words are taken, a node without its own bit among them; a row that sees
 * no key is 0, as are the rows of padding, whose q and words are not used.
 * Bits from m on are ignored. With lens[s] < m the first m - lens[s] nodes have
 * no key. Statistics, sums and the use of a NaN or infinity
 * in v of one of the nodes (it reaches all rows of its sequence) are as in
 * gdn_paged_attention, and so are all arguments but
 * n_nodes     device int32 [n_seqs] (0 .. T), or NULL
 * tree        device uint64 [n_seqs][T]
 * shape->T    nodes of each sequence, at most 64
 * n_nodes out of range is cut to it and reported as GDN_ERR_DEVICE_ARG by
 * gdn_check_device_error.
 * Any page size is taken; for bf16 and more than 64 rows of a kv head (T x H / H_kv),
 * pages of 8, 16, 32 or a multiple of 64 tokens are some 3 times as fast as others.
 */
gdn_status gdn_tree_attention(const gdn_attn_shape *shape, const gdn_kv_cache *cache,
                              const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *page_table, const int32_t *lens,
                              const int32_t *n_nodes, const uint64_t *tree, void *out,
                              void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * The gated delta rule along every branch: with S_p the state after node t's
 * parent (state_in for a node without one), node t has
 *   S = decay(S_p), d = beta (v - S^T k), S <- S + k d^T, o = scale S^T q
 * (decay as gdn_forward). No state is written: o and d follow from state_in,
 * the keys of the ancestors and their d, and gdn_tree_commit forms the one
 * state that is wanted from the d once a branch is accepted. All products and
 * sums are as exact as fp32 ones, for bf16 inputs too, whatever the size of the
 * state's other elements; any gate is computed, -inf included. An element of the
 * state, or of a key or query times its decays, that is not finite or above 3.38e38
 * makes the sums that it enters NaN.
 * shape       as gdn_forward, T = nodes of each sequence, at most 64
 * q, k, v, g, beta, state_in  as gdn_forward (token s*T+t is node t)
 * n_nodes     device int32 [n_seqs], or NULL
 * tree        device uint64 [n_seqs][T]; words of padding are not read
 * out         device fp32 [n_seqs*T][H][D_v]: o
 * updates     device fp32 [n_seqs*T][H][D_v]: d
 * Padding rows of out and updates are 0; their inputs are not used. n_nodes
 * outside 0 .. T, or words that are no tree (bit t missing in word t, a later
 * node's bit, an ancestor whose own ancestors differ) are reported as
 * GDN_ERR_DEVICE_ARG by gdn_check_device_error, and that sequence's rows are
 * not written. out and updates overlap each other and the inputs nowhere, nor any
 * state_in[s] (not checked). With n_seqs = 0 or T = 0 this call and the next
 * do nothing.
 */
gdn_status gdn_tree_forward(const gdn_shape *shape, const void *q, const void *k, const void *v,
                            const float *g, const float *beta, const float *const *state_in,
                            const int32_t *n_nodes, const uint64_t *tree, float *out,
                            float *updates, gdn_mode mode, gdn_stream_t stream);

/*
 * The state after node leaf[s] of each sequence, from the same k, g, state_in
 * and tree as gdn_tree_forward's and the updates that it wrote:
 *   S = state_in, then for each ancestor of the leaf and the leaf in turn
 *   S = decay(S) + k d^T
 * leaf        device int32 [n_seqs], one of the nodes that the sequence has; -1: no
 *             node, the state is state_in. (n_nodes is not given: a leaf in the
 *             padding is reported only where its word could be no node's.)
 * state_out   device fp32 [n_seqs][H][D_k][D_v]. state_in[s] may be the place
 *             of sequence s in it (in place); any other overlap is reported as
 *             GDN_ERR_DEVICE_ARG and that sequence's state is not written.
 * A leaf outside -1 .. T-1, or whose word lacks its own bit or has a later
 * node's, is reported likewise. The scale of `shape` is not used.
 */
gdn_status gdn_tree_commit(const gdn_shape *shape, const void *k, const float *g,
                           const float *updates, const float *const *state_in,
                           const uint64_t *tree, const int32_t *leaf, float *state_out,
                           gdn_mode mode, gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * One token of each row of logits (a decode step's sequences, or every
 * drafted token that a verify step scored), from a random number that the
 * caller gives. Per row, with its own settings:
 *   w[i]  = exp((x[i] - max x) / temperature)
 *   order = by logit, largest first, equal ones by index, lowest first
 *   kept  = the first n of that order, n the least of
 *             top_k;
 *             the fewest whose mass (sum of w) is at least top_p times that of
 *             the first top_k;
 *             those with w[i] >= min_p;
 *           but one at least
 *   token = the first kept index, counting up, whose running mass is above
 *           uniform * (mass of all kept)
 *   prob  = w[token] / (mass of all kept)
 * temperature <= 0 (or NaN) takes the first token of the order (prob 1). A
 * NaN logit counts as -infinity. Tokens at +infinity have weight 1 and all
 * others 0. A row with nothing above -infinity gives token -1, prob 0.
 * top_k <= 0, top_p >= 1, min_p <= 0 or NaN: no such limit.
 * Weights and masses are whole numbers of 2^-44 of the largest weight (a
 * weight is off by some 2^-30 of itself; below 2^-44.9 it is 0), so the result is
 * the same bits every time and its place between two tokens is that of exact
 * sums. Temperatures below 1e-30 count as 1e-30, those above 3e33 as 3e33.
 * ---------------------------------------------------------------------- */
typedef struct {
  int rows;             /* >= 0, at most 2^24 */
  int vocab;            /* 1 .. 2^18 */
  gdn_dtype dtype;      /* of the logits */
  long long row_stride; /* elements between rows, any from vocab on; 0 = vocab */
} gdn_sample_shape;

/*
 * logits       device [rows] rows of [vocab], row_stride apart
 * temperature, top_p, min_p  device fp32 [rows]; top_k device int32 [rows];
 *              each may be NULL (temperature 1; no limit)
 * uniform      device fp32 [rows], 0 <= uniform < 1 (outside: the first or
 *              the last kept token; NaN: the first)
 * tokens       device int32 [rows]
 * probs        device fp32 [rows], or NULL
 */
gdn_status gdn_sample(const gdn_sample_shape *shape, const void *logits, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p,
                      const float *uniform, int32_t *tokens, float *probs, gdn_stream_t stream);

/* ------------------------------------------------------------------------
 * Rollback bookkeeping: a host-side table with one entry per sequence (the
 * recurrent memory's per-sequence record of which stored state is live,
 * "llama-memory-recurrent: clear rs_idx in clear", koboldcpp commits, tag
 * v1.113.1). No device work.
 * ---------------------------------------------------------------------- */
typedef struct gdn_seq_table gdn_seq_table;

gdn_status gdn_seq_table_create(int n_seqs, int n_slots, gdn_seq_table **out);
void gdn_seq_table_destroy(gdn_seq_table *table);

/* Records that the last forward ran T_last tokens of sequence `seq`. */
gdn_status gdn_seq_table_record(gdn_seq_table *table, int seq, int T_last);

/* Forgets the last forward of `seq` (only n_accepted = 0 is valid after). */
gdn_status gdn_seq_table_clear(gdn_seq_table *table, int seq);

/*
 * Which state holds sequence `seq` after accepting the first n_accepted
 * tokens of its last forward: *slot = -1 means "the state_in of that forward
 * is unchanged"; otherwise the slot index. GDN_ERR_ROLLBACK_RANGE when
 * n_accepted is outside [0, T_last] or the token was not snapshotted (the
 * caller must recompute). The table is not modified.
 */
gdn_status gdn_rollback(const gdn_seq_table *table, int seq, int n_accepted,
                        int *slot);

/*
 * Device address of slot `slot` of sequence `seq` in a state_slots buffer of
 * the layout above, for building the next call's state_in array. Pure
 * address arithmetic; *out = NULL for slot = -1.
 */
gdn_status gdn_slot_state_ptr(const float *state_slots, int seq, int slot,
                              int n_slots, int H, int D_k, int D_v,
                              const float **out);

/* ------------------------------------------------------------------------
 * Device error word of the current device: synchronises `stream`, then
 * reads and clears the word. GDN_OK if no kernel reported a problem since
 * the last check; else GDN_ERR_TIMEOUT or GDN_ERR_DEVICE_ARG with a message.
 * ---------------------------------------------------------------------- */
gdn_status gdn_check_device_error(gdn_stream_t stream);

/*
 * Maps a value of the device error word to the status gdn_check_device_error
 * returns for it, and sets the calling thread's gdn_last_error message to the
 * text it would give: GDN_OK for 0; GDN_ERR_TIMEOUT for a bounded wait that
 * ran out (the message names the wait site, bits 8..15, and the chunk, bits
 * 16..30); GDN_ERR_DEVICE_ARG for the argument conditions above. Host only,
 * no device access.
 */
gdn_status gdn_decode_device_error(int word);

/*
 * Device address of the current device's error word (one int), for a
 * caller's own kernels that want to report through gdn_check_device_error:
 * they set it with atomicCAS(word, 0, value) so that the first condition
 * wins, as the library's kernels do. The address is looked up once per
 * device and is not valid after cudaDeviceReset.
 */
gdn_status gdn_device_error_word(int **word);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
