"""Refusals of the attention layer's entry points, all made before the device
is touched (no GPU needed)."""
import ctypes

import pytest

FAKE = 1 << 24   # aligned addresses, far apart; never dereferenced here
STEP = 1 << 24


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    return mod


def refused(gdn, call):
    with pytest.raises(gdn.GDNError) as e:
        call()
    return e.value.status, str(e.value)


def norm(gdn, shape=None, **kw):
    sh = dict(rows=4, cols=256, dtype=gdn.GDN_BF16, normalize=1, eps=1e-6, weight_offset=0.0)
    sh.update(shape or {})
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("x", "residual", "weight", "residual_out", "out", "out_fp8", "out_scale"))}
    p.update(kw)
    gdn.gdn_rmsnorm_fp8(gdn.gdn_norm_shape(*(sh[f[0]] for f in gdn.gdn_norm_shape._fields_)),
                        *p.values())


@pytest.mark.parametrize("shape", [
    dict(rows=-1), dict(cols=0), dict(dtype=7), dict(normalize=2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(weight_offset=float("inf")), dict(normalize=0)])
def test_norm_refuses_shapes(gdn, shape):
    st, msg = refused(gdn, lambda: norm(gdn, shape))
    assert st == gdn.GDN_ERR_INVALID_ARG and "gdn_rmsnorm_fp8" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(x=0), "x is NULL"), (dict(x=FAKE + 2), "x is not 16-byte aligned"),
    (dict(out_fp8=0), "come together"), (dict(out_scale=0), "come together"),
    (dict(out=0, out_fp8=0, out_scale=0), "both NULL"),
    (dict(out=FAKE + 16), "out overlaps x"), (dict(out_fp8=FAKE), "out_fp8 overlaps x"),
    (dict(residual_out=FAKE + 2 * STEP), "residual_out overlaps weight"),
    (dict(out=FAKE + 3 * STEP), "out overlaps residual_out"),
    (dict(out_scale=FAKE + 5 * STEP + 1008), "out_scale overlaps out_fp8")])
def test_norm_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: norm(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_norm_of_no_rows(gdn):
    norm(gdn, dict(rows=0), x=0)
    assert gdn.lib.gdn_rmsnorm_fp8(None, *[0] * 8) == gdn.GDN_ERR_INVALID_ARG


def kv(gdn, **kw):
    c = dict(n_pages=10, page_size=16, H_kv=2, D=128, dtype=gdn.GDN_BF16, page_stride=0,
             token_stride=0, head_stride=0)
    c.update(kw)
    return gdn.gdn_kv_cache(*(c[f[0]] for f in gdn.gdn_kv_cache._fields_))


BAD_CACHES = [
    (dict(n_pages=-1), 1), (dict(page_size=0), 1), (dict(H_kv=0), 1), (dict(dtype=5), 1),
    (dict(D=0), 1), (dict(D=96), 2), (dict(D=512), 2),
    (dict(page_stride=4096), 1), (dict(page_stride=4096, token_stride=256, head_stride=129), 1),
    (dict(page_stride=4096, token_stride=256, head_stride=120), 1),   # heads overlap
    (dict(page_stride=4088, token_stride=256, head_stride=128), 1),   # pages overlap
    (dict(page_stride=1 << 59, token_stride=256, head_stride=128), 2)]


def rope(gdn, shape=None, cache=None, **kw):
    sh = dict(n_tokens=5, H=4, rot_dim=128, pairs=0, n_axes=3, section=(32, 16, 16), axes=0,
              q_stride=0, k_stride=0, v_stride=0)
    sh.update(shape or {})
    sh["section"] = (ctypes.c_int * 4)(*sh["section"])
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("q", "k", "v", "positions", "inv_freq", "slots", "q_out", "k_cache", "v_cache"))}
    p.update(kw)
    gdn.gdn_rope_append(gdn.gdn_rope_shape(*(sh[f[0]] for f in gdn.gdn_rope_shape._fields_)),
                        kv(gdn, **(cache or {})), *p.values())


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_rope_refuses_caches(gdn, cache, status):
    st, msg = refused(gdn, lambda: rope(gdn, cache=cache))
    assert st == status and "gdn_rope_append" in msg


@pytest.mark.parametrize("shape", [
    dict(n_tokens=-1), dict(H=0), dict(rot_dim=127), dict(rot_dim=130), dict(rot_dim=-2),
    dict(pairs=2), dict(axes=2), dict(n_axes=0), dict(n_axes=5), dict(section=(32, 16, 15)),
    dict(section=(65, 0, 0)), dict(section=(65, -1, 0)), dict(axes=1, section=(10, 22, 32)),
    dict(q_stride=512 - 8), dict(k_stride=260), dict(v_stride=(1 << 28) + 8)])
def test_rope_refuses_shapes(gdn, shape):
    st, msg = refused(gdn, lambda: rope(gdn, shape))
    assert st == gdn.GDN_ERR_INVALID_ARG and "gdn_rope_append" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(q=0), "q is NULL"), (dict(v_cache=0), "v_cache is NULL"),
    (dict(inv_freq=0), "inv_freq is NULL"), (dict(slots=FAKE + 8), "slots is not 16-byte"),
    (dict(q_out=FAKE), "q_out overlaps q"), (dict(k_cache=FAKE + STEP), "k_cache overlaps k"),
    (dict(v_cache=FAKE + 7 * STEP), "are the same"),
    (dict(q_out=FAKE + 8 * STEP), "q_out overlaps v_cache")])
def test_rope_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: rope(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_rope_of_no_tokens_and_null_structs(gdn):
    rope(gdn, dict(n_tokens=0), q=0)
    assert gdn.lib.gdn_rope_append(None, None, *[0] * 10) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.lib.gdn_rope_append(ctypes.byref(gdn.gdn_rope_shape()), None,
                                   *[0] * 10) == gdn.GDN_ERR_INVALID_ARG


def attend(gdn, shape=None, cache=None, nbytes=1 << 23, **kw):
    sh = dict(n_seqs=3, T=2, H=8, max_pages=4, scale=0.0, kv_map=1)
    sh.update(shape or {})
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("q", "k_cache", "v_cache", "page_table", "lens", "out", "workspace"))}
    p.update(kw)
    gdn.gdn_paged_attention(gdn.gdn_attn_shape(*(sh[f[0]] for f in gdn.gdn_attn_shape._fields_)),
                            kv(gdn, **(cache or {})), *p.values(), nbytes)


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_attention_refuses_caches(gdn, cache, status):
    st, msg = refused(gdn, lambda: attend(gdn, cache=cache))
    assert st == status and "gdn_paged_attention" in msg
    assert gdn.gdn_paged_attention_workspace_size(gdn.gdn_attn_shape(3, 2, 8, 4, 0.0, 1),
                                                  kv(gdn, **cache)) == 0


@pytest.mark.parametrize("shape,status", [
    (dict(n_seqs=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(max_pages=-1), 1),
    (dict(kv_map=2), 1), (dict(scale=float("inf")), 1), (dict(n_seqs=1 << 28), 2)])
def test_attention_refuses_shapes(gdn, shape, status):
    st, msg = refused(gdn, lambda: attend(gdn, shape))
    assert st == status and "gdn_paged_attention" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(q=0), "q is NULL"), (dict(lens=0), "lens is NULL"), (dict(workspace=0), "workspace is"),
    (dict(k_cache=FAKE + STEP + 4), "k_cache is not 16-byte"), (dict(out=FAKE), "out overlaps q"),
    (dict(workspace=FAKE + 6 * STEP + 16), "256-byte"),
    (dict(workspace=FAKE + STEP), "workspace overlaps k_cache"), (dict(nbytes=1000), "needed")])
def test_attention_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: attend(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_attention_of_nothing(gdn):
    attend(gdn, dict(n_seqs=0), q=0)
    attend(gdn, dict(T=0), q=0)
    assert gdn.lib.gdn_paged_attention(None, None, *[0] * 9) == gdn.GDN_ERR_INVALID_ARG


def test_attention_workspace_goes_by_the_shapes(gdn):
    size = gdn.gdn_paged_attention_workspace_size
    small = size(gdn.gdn_attn_shape(1, 1, 8, 1, 0.0, 1), kv(gdn))
    large = size(gdn.gdn_attn_shape(64, 8, 16, 512, 0.0, 1), kv(gdn))
    assert 0 < small < large <= 64 << 20


def gemm(gdn, shape=None, **kw):
    sh = dict(M=40, N=300, K=512, out_dtype=gdn.GDN_BF16)
    sh.update(shape or {})
    p = {n: FAKE + i * STEP for i, n in enumerate(("a", "a_scale", "b", "b_scale", "out"))}
    p.update(kw)
    gdn.gdn_gemm_fp8(gdn.gdn_gemm_shape(*(sh[f[0]] for f in gdn.gdn_gemm_shape._fields_)),
                     *p.values())


@pytest.mark.parametrize("shape,status", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=0), 1), (dict(out_dtype=3), 1), (dict(K=520), 2),
    (dict(K=8), 2), (dict(M=(1 << 21) + 1), 2), (dict(K=(1 << 21) + 16), 2)])
def test_gemm_refuses_shapes(gdn, shape, status):
    st, msg = refused(gdn, lambda: gemm(gdn, shape))
    assert st == status and "gdn_gemm_fp8" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(a=0), "a is NULL"), (dict(b_scale=0), "b_scale is NULL"), (dict(out=0), "out is NULL"),
    (dict(b=FAKE + 2 * STEP + 8), "b is not 16-byte"), (dict(out=FAKE + 4 * STEP + 2), "out is not"),
    (dict(out=FAKE), "out overlaps a"), (dict(out=FAKE + 3 * STEP - 32), "out overlaps b_scale")])
def test_gemm_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: gemm(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_gemm_of_nothing(gdn):
    gemm(gdn, dict(M=0), a=0)
    gemm(gdn, dict(N=0), b=0)
    assert gdn.lib.gdn_gemm_fp8(None, *[0] * 6) == gdn.GDN_ERR_INVALID_ARG


def test_binding_refuses_views_that_do_not_match_their_shape(gdn):
    import torch
    qkv = torch.zeros(5, 8 * 128)
    q = qkv[:, :512].unflatten(1, (4, 128))
    out = torch.zeros(5, 4, 128)
    for stride, view in ((0, q), (1024, out), (1024, q.transpose(1, 2))):
        with pytest.raises(ValueError, match="rows must be packed"):
            rope(gdn, dict(q_stride=stride), q=view)
    with pytest.raises(ValueError, match="contiguous"):
        rope(gdn, q_out=qkv[:, ::2])
    with pytest.raises(ValueError, match="needs its strides"):
        rope(gdn, k_cache=torch.zeros(10, 2, 16, 128).transpose(1, 2))
