"""Thin ctypes binding of libgdn (include/gdn.h): same names, argument
marshalling only. Every step of the op runs in the library's CUDA kernels.

Device buffers may be passed as torch tensors (their data_ptr is used) or as
integer addresses. A non-OK status raises GDNError carrying the status code
and the library's message. If the library is missing this module raises at
import time: there is no fallback.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = 1
GDN_ERR_UNSUPPORTED = 2
GDN_ERR_ROLLBACK_RANGE = 3
GDN_ERR_CUDA = 4
GDN_ERR_TIMEOUT = 5
GDN_ERR_DEVICE_ARG = 6

GDN_MODE_GDA = 0
GDN_MODE_KDA = 1
GDN_F32 = 0
GDN_BF16 = 1

_MODES = {"gda": GDN_MODE_GDA, "kda": GDN_MODE_KDA,
          GDN_MODE_GDA: GDN_MODE_GDA, GDN_MODE_KDA: GDN_MODE_KDA}


class GDNError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"[gdn status {status}] {message}")
        self.status = status


GDN_QK_TILED, GDN_QK_GROUPED = 0, 1
QK_MAPS = {"tiled": GDN_QK_TILED, "grouped": GDN_QK_GROUPED}


class gdn_shape(ctypes.Structure):
    # H_qk = 0 (the default) means q and k have H heads
    _fields_ = [("n_seqs", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("D_k", ctypes.c_int), ("D_v", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("H_qk", ctypes.c_int), ("qk_map", ctypes.c_int)]


class gdn_varlen_shape(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("total_tokens", ctypes.c_int),
                ("H", ctypes.c_int), ("D_k", ctypes.c_int), ("D_v", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("H_qk", ctypes.c_int), ("qk_map", ctypes.c_int)]


class gdn_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("dtype", ctypes.c_int),
                ("normalize", ctypes.c_int), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float)]


class gdn_gemm_shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("out_dtype", ctypes.c_int)]


GDN_ROPE_HALVES, GDN_ROPE_NEIGHBOURS = 0, 1
GDN_ROPE_AXES_SECTIONED, GDN_ROPE_AXES_INTERLEAVED = 0, 1
c_int = ctypes.c_int    # (c_int * 4)(...) builds gdn_rope_shape's sections


class gdn_kv_cache(ctypes.Structure):
    # all three strides 0 (the default) means dense [n_pages][page_size][H_kv][D]
    _fields_ = [("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("H_kv", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int),
                ("page_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong)]


class gdn_rope_shape(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int), ("H", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("pairs", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("section", ctypes.c_int * 4), ("axes", ctypes.c_int),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong)]


class gdn_qk_norm(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class gdn_attn_shape(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("scale", ctypes.c_float),
                ("kv_map", ctypes.c_int)]


class gdn_sample_shape(ctypes.Structure):
    # row_stride = 0 (the default) means rows of vocab elements, packed
    _fields_ = [("rows", ctypes.c_int), ("vocab", ctypes.c_int), ("dtype", ctypes.c_int),
                ("row_stride", ctypes.c_longlong)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libgdn.so is not built ({LIB_PATH}); run "
                      "gated_delta_net_02_gb300/build.py or __graft_entry__.build()")
lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i = ctypes.c_int
_st = ctypes.c_int

lib.gdn_last_error.restype = ctypes.c_char_p
lib.gdn_version.restype = ctypes.c_char_p
lib.gdn_forward.restype = _st
lib.gdn_forward.argtypes = [ctypes.POINTER(gdn_shape), _vp, _vp, _vp, _vp, _vp, _vp,
                            _vp, _vp, _i, _i, _vp]
lib.gdn_forward_host.restype = _st
lib.gdn_forward_host.argtypes = lib.gdn_forward.argtypes
lib.gdn_chunked_workspace_size.restype = ctypes.c_size_t
lib.gdn_chunked_workspace_size.argtypes = [ctypes.POINTER(gdn_varlen_shape), _i]
lib.gdn_forward_chunked.restype = _st
lib.gdn_forward_chunked.argtypes = [ctypes.POINTER(gdn_varlen_shape), _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, ctypes.c_size_t,
                                    _vp]
lib.gdn_forward_chunked_noalloc.restype = _st
lib.gdn_forward_chunked_noalloc.argtypes = [ctypes.POINTER(gdn_varlen_shape), _vp, _vp, _vp,
                                            _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp]
lib.gdn_forward_chunked_checkpointed.restype = _st
lib.gdn_forward_chunked_checkpointed.argtypes = [
    ctypes.POINTER(gdn_varlen_shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
    _vp, _i, _i, _vp, ctypes.c_size_t, _vp]
lib.gdn_checkpoint_select.restype = _st
lib.gdn_checkpoint_select.argtypes = [_i, _i, _i, _i, _i, ctypes.POINTER(_i),
                                      ctypes.POINTER(_i), ctypes.POINTER(_i)]
lib.gdn_noalloc_scratch_bytes.restype = ctypes.c_size_t
lib.gdn_noalloc_scratch_bytes.argtypes = []
lib.gdn_rmsnorm_fp8.restype = _st
lib.gdn_rmsnorm_fp8.argtypes = [ctypes.POINTER(gdn_norm_shape), _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp]
lib.gdn_gemm_fp8.restype = _st
lib.gdn_gemm_fp8.argtypes = [ctypes.POINTER(gdn_gemm_shape), _vp, _vp, _vp, _vp, _vp, _vp]
lib.gdn_rope_append.restype = _st
lib.gdn_rope_append.argtypes = [ctypes.POINTER(gdn_rope_shape), ctypes.POINTER(gdn_kv_cache),
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.gdn_qknorm_rope_append.restype = _st
lib.gdn_qknorm_rope_append.argtypes = [
    ctypes.POINTER(gdn_rope_shape), ctypes.POINTER(gdn_kv_cache), ctypes.POINTER(gdn_qk_norm),
    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.gdn_paged_attention_workspace_size.restype = ctypes.c_size_t
lib.gdn_paged_attention_workspace_size.argtypes = [ctypes.POINTER(gdn_attn_shape),
                                                   ctypes.POINTER(gdn_kv_cache)]
lib.gdn_paged_attention.restype = _st
lib.gdn_paged_attention.argtypes = [ctypes.POINTER(gdn_attn_shape),
                                    ctypes.POINTER(gdn_kv_cache), _vp, _vp, _vp, _vp, _vp, _vp,
                                    _vp, ctypes.c_size_t, _vp]
lib.gdn_tree_attention_workspace_size.restype = ctypes.c_size_t
lib.gdn_tree_attention_workspace_size.argtypes = lib.gdn_paged_attention_workspace_size.argtypes
lib.gdn_tree_attention.restype = _st
lib.gdn_tree_attention.argtypes = [ctypes.POINTER(gdn_attn_shape), ctypes.POINTER(gdn_kv_cache),
                                   _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                   _vp]
lib.gdn_tree_forward.restype = _st
lib.gdn_tree_forward.argtypes = [ctypes.POINTER(gdn_shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _i, _vp]
lib.gdn_tree_commit.restype = _st
lib.gdn_tree_commit.argtypes = [ctypes.POINTER(gdn_shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i,
                                _vp]
lib.gdn_sample.restype = _st
lib.gdn_sample.argtypes = [ctypes.POINTER(gdn_sample_shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _vp, _vp]
lib.gdn_seq_table_create.restype = _st
lib.gdn_seq_table_create.argtypes = [_i, _i, ctypes.POINTER(_vp)]
lib.gdn_seq_table_destroy.restype = None
lib.gdn_seq_table_destroy.argtypes = [_vp]
lib.gdn_seq_table_record.restype = _st
lib.gdn_seq_table_record.argtypes = [_vp, _i, _i]
lib.gdn_seq_table_clear.restype = _st
lib.gdn_seq_table_clear.argtypes = [_vp, _i]
lib.gdn_rollback.restype = _st
lib.gdn_rollback.argtypes = [_vp, _i, _i, ctypes.POINTER(_i)]
lib.gdn_slot_state_ptr.restype = _st
lib.gdn_slot_state_ptr.argtypes = [_vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_vp)]
lib.gdn_check_device_error.restype = _st
lib.gdn_check_device_error.argtypes = [_vp]
lib.gdn_decode_device_error.restype = _st
lib.gdn_decode_device_error.argtypes = [_i]
lib.gdn_device_error_word.restype = _st
lib.gdn_device_error_word.argtypes = [ctypes.POINTER(_vp)]


def _addr(x):
    """Device address of a tensor argument (or a raw integer address). The C
    ABI takes packed row-major buffers, so a strided view is refused here
    rather than read as if it were packed."""
    if x is None or x.__class__ is int:   # the common cases first: this runs for
        return x                          # every buffer of every call
    try:
        packed = x.is_contiguous()
    except AttributeError:
        if isinstance(x, int):            # an int of another class
            return int(x)
        raise
    if not packed:
        raise ValueError("gdn: tensor arguments must be contiguous (packed row-major)")
    return x.data_ptr()


def _rows_addr(x, n, stride, width, D):
    """Device address of n rows [heads][D] that lie `stride` elements apart
    (0 = dense, `width`): a column range of a wider matrix is such a view."""
    if x is None or x.__class__ is int:
        return x
    try:
        st = x.stride()
    except AttributeError:
        if isinstance(x, int):
            return int(x)
        raise
    if (len(st) != 3 or st[2] != 1 or st[1] != D and width != D
            or n > 1 and st[0] != (stride or width)):
        raise ValueError("gdn: rows must be packed, and apart by the shape's stride")
    return x.data_ptr()


def _cache_addr(x, cache):
    """Device address of a cache tensor; a strided one must say so in `cache`."""
    if x is None or x.__class__ is int:
        return x
    try:
        address = x.data_ptr()
    except AttributeError:
        if isinstance(x, int):
            return int(x)
        raise
    if not cache.token_stride:
        if not x.is_contiguous():
            raise ValueError("gdn: a strided cache needs its strides in gdn_kv_cache")
    elif (x.stride() != (cache.page_stride, cache.token_stride, cache.head_stride, 1)
          and not _cache_matches(x, cache)):
        raise ValueError("gdn: the cache's strides are not those in gdn_kv_cache")
    return address


def _cache_matches(x, cache):
    """Whether tensor x, in another form than [n_pages, page_size, H_kv, D],
    has the elements that `cache` names: its dimensions in another order, or
    pages and tokens in one. A packed tensor is memory from its start on."""
    levels = [(stride, n) for stride, n in (
        (cache.page_stride, cache.n_pages), (cache.token_stride, cache.page_size),
        (cache.head_stride, cache.H_kv), (1, cache.D)) if n > 1]
    if x.is_contiguous():
        held = x.untyped_storage().nbytes() // x.element_size() - x.storage_offset()
        return cache.n_pages == 0 or sum(stride * (n - 1) for stride, n in levels) < held
    dims = {stride: n for stride, n in zip(x.stride(), x.shape) if n > 1 and stride > 0}
    last = dict.fromkeys(dims, 0)      # index of the cache's last element
    for stride, n in levels:
        along = max((d for d in dims if stride % d == 0), default=None)
        if along is None:
            return False
        last[along] += (n - 1) * (stride // along)
    return all(last[d] < n for d, n in dims.items())


def _check(status):
    if status != GDN_OK:
        raise GDNError(status, lib.gdn_last_error().decode(errors="replace"))


def _stream(stream):
    if stream is None or stream.__class__ is int:
        return stream
    try:
        return stream.cuda_stream  # torch.cuda.Stream
    except AttributeError:
        if isinstance(stream, int):
            return int(stream)
        raise


def gdn_version() -> str:
    return lib.gdn_version().decode()


def gdn_last_error() -> str:
    return lib.gdn_last_error().decode(errors="replace")


def gdn_forward(shape: gdn_shape, q, k, v, g, beta, state_in, state_slots, out,
                n_slots: int, mode, stream=None) -> None:
    """state_in: device array of n_seqs state pointers (e.g. an int64 tensor
    built with state_ptr_array)."""
    _check(lib.gdn_forward(ctypes.byref(shape), _addr(q), _addr(k), _addr(v), _addr(g),
                           _addr(beta), _addr(state_in), _addr(state_slots), _addr(out),
                           int(n_slots), _MODES[mode], _stream(stream)))


def gdn_forward_host(shape: gdn_shape, q, k, v, g, beta, state_in, state_slots, out,
                     n_slots: int, mode, stream=None) -> None:
    """gdn_forward whose q, k, v, g, beta and out may be pinned host tensors
    (or device tensors): the kernel reads and writes them over the host link."""
    _check(lib.gdn_forward_host(ctypes.byref(shape), _addr(q), _addr(k), _addr(v), _addr(g),
                                _addr(beta), _addr(state_in), _addr(state_slots), _addr(out),
                                int(n_slots), _MODES[mode], _stream(stream)))


def gdn_chunked_workspace_size(shape: gdn_varlen_shape, n_slots: int) -> int:
    return int(lib.gdn_chunked_workspace_size(ctypes.byref(shape), int(n_slots)))


def gdn_forward_chunked(shape: gdn_varlen_shape, cu_seqlens, q, k, v, g, beta, state_in,
                        state_slots, out, n_slots: int, mode, workspace,
                        workspace_bytes: int, stream=None) -> None:
    _check(lib.gdn_forward_chunked(ctypes.byref(shape), _addr(cu_seqlens), _addr(q),
                                   _addr(k), _addr(v), _addr(g), _addr(beta),
                                   _addr(state_in), _addr(state_slots), _addr(out),
                                   int(n_slots), _MODES[mode], _addr(workspace),
                                   int(workspace_bytes), _stream(stream)))


def gdn_forward_chunked_noalloc(shape: gdn_varlen_shape, cu_seqlens, q, k, v, g, beta,
                                state_in, state_slots, out, n_slots: int, mode,
                                stream=None) -> None:
    """gdn_forward_chunked without a workspace: the library's built-in
    scratch array is used (for callers that cannot allocate device memory)."""
    _check(lib.gdn_forward_chunked_noalloc(ctypes.byref(shape), _addr(cu_seqlens), _addr(q),
                                           _addr(k), _addr(v), _addr(g), _addr(beta),
                                           _addr(state_in), _addr(state_slots), _addr(out),
                                           int(n_slots), _MODES[mode], _stream(stream)))


def gdn_forward_chunked_checkpointed(shape: gdn_varlen_shape, cu_seqlens, q, k, v, g, beta,
                                     state_in, state_slots, out, n_slots: int, mode,
                                     checkpoints, ckpt_every: int, max_ckpts: int,
                                     workspace, workspace_bytes: int, stream=None) -> None:
    """gdn_forward_chunked that also stores checkpoints[s][m], the state
    after (m+1)*ckpt_every tokens of sequence s (fp32 [N][max_ckpts][H][D_k][D_v])."""
    _check(lib.gdn_forward_chunked_checkpointed(
        ctypes.byref(shape), _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(g),
        _addr(beta), _addr(state_in), _addr(state_slots), _addr(out), int(n_slots),
        _MODES[mode], _addr(checkpoints), int(ckpt_every), int(max_ckpts), _addr(workspace),
        int(workspace_bytes), _stream(stream)))


CKPT_SOURCES = ("state_in", "checkpoint", "slot")


def gdn_checkpoint_select(n_keep: int, L: int, n_slots: int, ckpt_every: int,
                          max_ckpts: int):
    """(source, index, replay_from) for keeping the first n_keep of L tokens;
    source is one of CKPT_SOURCES."""
    src, idx, rep = _i(), _i(), _i()
    _check(lib.gdn_checkpoint_select(int(n_keep), int(L), int(n_slots), int(ckpt_every),
                                     int(max_ckpts), ctypes.byref(src), ctypes.byref(idx),
                                     ctypes.byref(rep)))
    return CKPT_SOURCES[src.value], idx.value, rep.value


def gdn_noalloc_scratch_bytes() -> int:
    return int(lib.gdn_noalloc_scratch_bytes())


def gdn_rmsnorm_fp8(shape: gdn_norm_shape, x, residual, weight, residual_out, out, out_fp8,
                    out_scale, stream=None) -> None:
    """residual, weight, residual_out and out may be None, and out_fp8 with
    out_scale when out is given. out_fp8: a float8_e4m3fn (or uint8) tensor."""
    _check(lib.gdn_rmsnorm_fp8(ctypes.byref(shape), _addr(x), _addr(residual), _addr(weight),
                               _addr(residual_out), _addr(out), _addr(out_fp8),
                               _addr(out_scale), _stream(stream)))


def gdn_gemm_fp8(shape: gdn_gemm_shape, a, a_scale, b, b_scale, out, stream=None) -> None:
    """out = A B^T of e4m3 matrices (float8_e4m3fn or uint8 tensors) with a
    scale for each row and 128 columns of A and each 128 x 128 block of B."""
    _check(lib.gdn_gemm_fp8(ctypes.byref(shape), _addr(a), _addr(a_scale), _addr(b),
                            _addr(b_scale), _addr(out), _stream(stream)))


def gdn_rope_append(shape: gdn_rope_shape, cache: gdn_kv_cache, q, k, v, positions, inv_freq,
                    slots, q_out, k_cache, v_cache, stream=None) -> None:
    """q, k and v may be column ranges of one wider matrix (the shape's
    strides); k_cache and v_cache have the layout of `cache`."""
    n, D = shape.n_tokens, cache.D
    kv = cache.H_kv * D
    _check(lib.gdn_rope_append(
        ctypes.byref(shape), ctypes.byref(cache),
        _rows_addr(q, n, shape.q_stride, shape.H * D, D), _rows_addr(k, n, shape.k_stride, kv, D),
        _rows_addr(v, n, shape.v_stride, kv, D), _addr(positions), _addr(inv_freq), _addr(slots),
        _addr(q_out), _cache_addr(k_cache, cache), _cache_addr(v_cache, cache),
        _stream(stream)))


def gdn_qknorm_rope_append(shape: gdn_rope_shape, cache: gdn_kv_cache, norm: gdn_qk_norm, q, k, v,
                           q_weight, k_weight, positions, inv_freq, slots, q_out, k_cache, v_cache,
                           stream=None) -> None:
    """gdn_rope_append with an RMS norm of every q and k head before the
    rotation; q_weight and k_weight may be None."""
    n, D = shape.n_tokens, cache.D
    kv = cache.H_kv * D
    _check(lib.gdn_qknorm_rope_append(
        ctypes.byref(shape), ctypes.byref(cache), ctypes.byref(norm),
        _rows_addr(q, n, shape.q_stride, shape.H * D, D), _rows_addr(k, n, shape.k_stride, kv, D),
        _rows_addr(v, n, shape.v_stride, kv, D), _addr(q_weight), _addr(k_weight),
        _addr(positions), _addr(inv_freq), _addr(slots), _addr(q_out),
        _cache_addr(k_cache, cache), _cache_addr(v_cache, cache), _stream(stream)))


def gdn_paged_attention_workspace_size(shape: gdn_attn_shape, cache: gdn_kv_cache) -> int:
    return int(lib.gdn_paged_attention_workspace_size(ctypes.byref(shape), ctypes.byref(cache)))


def gdn_paged_attention(shape: gdn_attn_shape, cache: gdn_kv_cache, q, k_cache, v_cache,
                        page_table, lens, out, workspace, workspace_bytes: int,
                        stream=None) -> None:
    """Attention of the last T tokens of each sequence over its pages."""
    _check(lib.gdn_paged_attention(
        ctypes.byref(shape), ctypes.byref(cache), _addr(q), _cache_addr(k_cache, cache),
        _cache_addr(v_cache, cache), _addr(page_table), _addr(lens), _addr(out),
        _addr(workspace), int(workspace_bytes), _stream(stream)))


def gdn_tree_attention_workspace_size(shape: gdn_attn_shape, cache: gdn_kv_cache) -> int:
    return int(lib.gdn_tree_attention_workspace_size(ctypes.byref(shape), ctypes.byref(cache)))


def gdn_tree_attention(shape: gdn_attn_shape, cache: gdn_kv_cache, q, k_cache, v_cache, page_table,
                       lens, n_nodes, tree, out, workspace, workspace_bytes: int,
                       stream=None) -> None:
    """Attention of a tree of drafted tokens of each sequence over its pages;
    `tree`: an int64 (or uint64) tensor of the words, n_nodes may be None."""
    _check(lib.gdn_tree_attention(
        ctypes.byref(shape), ctypes.byref(cache), _addr(q), _cache_addr(k_cache, cache),
        _cache_addr(v_cache, cache), _addr(page_table), _addr(lens), _addr(n_nodes), _addr(tree),
        _addr(out), _addr(workspace), int(workspace_bytes), _stream(stream)))


def gdn_tree_forward(shape: gdn_shape, q, k, v, g, beta, state_in, n_nodes, tree, out, updates,
                     mode, stream=None) -> None:
    """The delta rule along every branch of a tree of drafted tokens; `tree`:
    an int64 (or uint64) tensor of the words, n_nodes may be None."""
    _check(lib.gdn_tree_forward(ctypes.byref(shape), _addr(q), _addr(k), _addr(v), _addr(g),
                                _addr(beta), _addr(state_in), _addr(n_nodes), _addr(tree),
                                _addr(out), _addr(updates), _MODES[mode], _stream(stream)))


def gdn_tree_commit(shape: gdn_shape, k, g, updates, state_in, tree, leaf, state_out, mode,
                    stream=None) -> None:
    """The state after node leaf[s] of each sequence, from gdn_tree_forward's updates."""
    _check(lib.gdn_tree_commit(ctypes.byref(shape), _addr(k), _addr(g), _addr(updates),
                               _addr(state_in), _addr(tree), _addr(leaf), _addr(state_out),
                               _MODES[mode], _stream(stream)))


def _matrix_addr(x, rows, cols, stride):
    """Device address of `rows` rows of `cols` elements, `stride` apart (0 = packed)."""
    if x is None or x.__class__ is int:
        return x
    try:
        st = x.stride()
    except AttributeError:
        if isinstance(x, int):
            return int(x)
        raise
    if st[-1] != 1 and cols > 1 or rows > 1 and (
            not x.is_contiguous() if not stride or stride == cols else st[:-1] != (stride,)):
        raise ValueError("gdn: rows must be packed, and apart by the shape's stride")
    return x.data_ptr()


def gdn_sample(shape: gdn_sample_shape, logits, temperature, top_k, top_p, min_p, uniform, tokens,
               probs=None, stream=None) -> None:
    """One token of each row of logits from given random numbers; temperature,
    top_k, top_p, min_p and probs may be None."""
    _check(lib.gdn_sample(
        ctypes.byref(shape), _matrix_addr(logits, shape.rows, shape.vocab, shape.row_stride),
        _addr(temperature), _addr(top_k), _addr(top_p), _addr(min_p), _addr(uniform),
        _addr(tokens), _addr(probs), _stream(stream)))


def gdn_check_device_error(stream=None) -> None:
    _check(lib.gdn_check_device_error(_stream(stream)))


def gdn_decode_device_error(word: int):
    """(status, message) the library gives for a device error-word value."""
    st = int(lib.gdn_decode_device_error(int(word)))
    return st, (lib.gdn_last_error().decode(errors="replace") if st != GDN_OK else "")


def gdn_device_error_word() -> int:
    """Device address of the current device's error word."""
    out = _vp()
    _check(lib.gdn_device_error_word(ctypes.byref(out)))
    return out.value or 0


class SeqTable:
    """Owner of a gdn_seq_table (host-side rollback bookkeeping)."""

    def __init__(self, n_seqs: int, n_slots: int):
        h = _vp()
        _check(lib.gdn_seq_table_create(int(n_seqs), int(n_slots), ctypes.byref(h)))
        self._h = h
        self.n_seqs, self.n_slots = n_seqs, n_slots

    def record(self, seq: int, T_last: int) -> None:
        _check(lib.gdn_seq_table_record(self._h, int(seq), int(T_last)))

    def clear(self, seq: int) -> None:
        _check(lib.gdn_seq_table_clear(self._h, int(seq)))

    def rollback(self, seq: int, n_accepted: int) -> int:
        """gdn_rollback: slot index, or -1 for "input state unchanged"."""
        slot = _i(-2)
        _check(lib.gdn_rollback(self._h, int(seq), int(n_accepted), ctypes.byref(slot)))
        return slot.value

    def close(self):
        if self._h:
            lib.gdn_seq_table_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_slot_state_ptr(state_slots, seq: int, slot: int, n_slots: int, H: int, D_k: int,
                       D_v: int) -> int:
    out = _vp()
    _check(lib.gdn_slot_state_ptr(_addr(state_slots), int(seq), int(slot), int(n_slots),
                                  int(H), int(D_k), int(D_v), ctypes.byref(out)))
    return out.value or 0


def state_ptr_array(ptrs, device):
    """Device int64 tensor holding the given state addresses (0 = zero state)."""
    import torch
    return torch.tensor([int(p) if p else 0 for p in ptrs], dtype=torch.int64, device=device)


def per_seq_state_ptrs(state, n_seqs: int):
    """Addresses of state[s] for a contiguous [N, H, D_k, D_v] fp32 tensor."""
    per = state[0].numel() * state.element_size()
    base = state.data_ptr()
    return [base + s * per for s in range(n_seqs)]


def dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.bfloat16:
        return GDN_BF16
    if torch_dtype == torch.float32:
        return GDN_F32
    raise ValueError(f"unsupported input dtype {torch_dtype}")
