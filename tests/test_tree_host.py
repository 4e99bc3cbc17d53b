"""Refusals of the entry points that verify a tree of drafts, all made before
the device is touched (no GPU needed)."""
import ctypes

import pytest

from test_layer_host import BAD_CACHES, FAKE, STEP, gdn, kv, refused  # noqa: F401


def qknorm(gdn, shape=None, cache=None, eps=1e-6, offset=0.0, **kw):
    sh = dict(n_tokens=5, H=4, rot_dim=128, pairs=0, n_axes=3, section=(32, 16, 16), axes=0,
              q_stride=0, k_stride=0, v_stride=0)
    sh.update(shape or {})
    sh["section"] = (ctypes.c_int * 4)(*sh["section"])
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("q", "k", "v", "q_weight", "k_weight", "positions", "inv_freq", "slots", "q_out",
         "k_cache", "v_cache"))}
    p.update(kw)
    gdn.gdn_qknorm_rope_append(
        gdn.gdn_rope_shape(*(sh[f[0]] for f in gdn.gdn_rope_shape._fields_)),
        kv(gdn, **(cache or {})), gdn.gdn_qk_norm(eps, offset), *p.values())


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_qknorm_refuses_caches(gdn, cache, status):
    st, msg = refused(gdn, lambda: qknorm(gdn, cache=cache))
    assert st == status and "gdn_qknorm_rope_append" in msg


@pytest.mark.parametrize("args", [
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(offset=float("nan")),
    dict(shape=dict(n_tokens=-1)), dict(shape=dict(H=0)), dict(shape=dict(rot_dim=130)),
    dict(shape=dict(section=(32, 16, 15))), dict(shape=dict(q_stride=512 - 8))])
def test_qknorm_refuses_shapes(gdn, args):
    st, msg = refused(gdn, lambda: qknorm(gdn, **args))
    assert st == gdn.GDN_ERR_INVALID_ARG and "gdn_qknorm_rope_append" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(q=0), "q is NULL"), (dict(inv_freq=0), "inv_freq is NULL"),
    (dict(q_weight=FAKE + 3 * STEP + 8), "q_weight is not 16-byte"),
    (dict(k_weight=FAKE + 4 * STEP + 2), "k_weight is not 16-byte"),
    (dict(q_out=FAKE + 3 * STEP), "q_out overlaps q_weight"),
    (dict(k_cache=FAKE + 4 * STEP), "k_cache overlaps k_weight"),
    (dict(v_cache=FAKE + 9 * STEP), "are the same")])
def test_qknorm_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: qknorm(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_qknorm_of_no_tokens_and_null_structs(gdn):
    qknorm(gdn, dict(n_tokens=0), q=0)
    qknorm(gdn, dict(n_tokens=0), q_weight=0, k_weight=0)
    null = gdn.lib.gdn_qknorm_rope_append
    shape, norm = ctypes.byref(gdn.gdn_rope_shape()), ctypes.byref(gdn.gdn_qk_norm())
    for args in ((None, None, norm), (shape, None, norm), (shape, None, None)):
        assert null(*args, *[0] * 12) == gdn.GDN_ERR_INVALID_ARG


def sample(gdn, shape=None, **kw):
    sh = dict(rows=4, vocab=1000, dtype=gdn.GDN_BF16, row_stride=0)
    sh.update(shape or {})
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("logits", "temperature", "top_k", "top_p", "min_p", "uniform", "tokens", "probs"))}
    p.update(kw)
    gdn.gdn_sample(gdn.gdn_sample_shape(*(sh[f[0]] for f in gdn.gdn_sample_shape._fields_)),
                   *p.values())


@pytest.mark.parametrize("shape,status", [
    (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(dtype=2), 1), (dict(row_stride=999), 1),
    (dict(row_stride=-1000), 1), (dict(vocab=(1 << 18) + 1), 2), (dict(rows=(1 << 24) + 1), 2),
    (dict(row_stride=(1 << 32) + 1), 2)])
def test_sample_refuses_shapes(gdn, shape, status):
    st, msg = refused(gdn, lambda: sample(gdn, shape))
    assert st == status and "gdn_sample" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(logits=0), "logits is NULL"), (dict(uniform=0), "uniform is NULL"),
    (dict(tokens=0), "tokens is NULL"), (dict(logits=FAKE + 2), "logits is not 16-byte"),
    (dict(top_k=FAKE + 2 * STEP + 4), "top_k is not 16-byte"),
    (dict(probs=FAKE + 7 * STEP + 8), "probs is not 16-byte"), (dict(tokens=FAKE), "tokens overlaps"),
    (dict(probs=FAKE + 6 * STEP), "overlaps"), (dict(probs=FAKE + 5 * STEP), "probs overlaps uniform")])
def test_sample_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: sample(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_sample_of_no_rows(gdn):
    sample(gdn, dict(rows=0), logits=0, tokens=0, uniform=0)
    assert gdn.lib.gdn_sample(None, *[0] * 9) == gdn.GDN_ERR_INVALID_ARG


def test_sample_binding_refuses_views_that_do_not_match_their_shape(gdn):
    import torch
    base = torch.zeros(4, 1008, dtype=torch.bfloat16)
    for stride, view in ((0, base[:, :1000]), (1009, base[:, :1000]), (1008, base.t()[:1000].t()[:, ::2])):
        with pytest.raises(ValueError, match="rows must be packed"):
            sample(gdn, dict(row_stride=stride), logits=view)


def delta(gdn, call, shape=None, mode="gda", **kw):
    sh = dict(n_seqs=3, T=8, H=4, D_k=128, D_v=128, in_dtype=gdn.GDN_BF16, scale=0.0, H_qk=2,
              qk_map=0)
    sh.update(shape or {})
    names = {"forward": ("q", "k", "v", "g", "beta", "state_in", "n_nodes", "tree", "out", "updates"),
             "commit": ("k", "g", "updates", "state_in", "tree", "leaf", "state_out")}[call]
    p = {n: FAKE + i * STEP for i, n in enumerate(names)}
    p.update(kw)
    f = gdn.gdn_tree_forward if call == "forward" else gdn.gdn_tree_commit
    f(gdn.gdn_shape(*(sh[f[0]] for f in gdn.gdn_shape._fields_)), *p.values(), mode)


@pytest.mark.parametrize("call", ["forward", "commit"])
@pytest.mark.parametrize("shape,status", [
    (dict(n_seqs=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(D_k=0), 1), (dict(D_v=-1), 1),
    (dict(in_dtype=2), 1), (dict(scale=float("nan")), 1), (dict(H_qk=3), 1), (dict(qk_map=2), 1),
    (dict(D_k=256), 2), (dict(D_v=32), 2), (dict(T=65), 2), (dict(n_seqs=1 << 23), 2)])
def test_tree_calls_refuse_shapes(gdn, call, shape, status):
    st, msg = refused(gdn, lambda: delta(gdn, call, shape))
    assert st == status and "gdn_tree_" + call in msg


@pytest.mark.parametrize("call,ptrs,word", [
    ("forward", dict(q=0), "q is NULL"), ("forward", dict(tree=0), "tree is NULL"),
    ("forward", dict(updates=0), "updates is NULL"), ("forward", dict(state_in=0), "state_in is NULL"),
    ("forward", dict(n_nodes=FAKE + 6 * STEP + 4), "n_nodes is not 16-byte"),
    ("forward", dict(out=FAKE + 2 * STEP), "out overlaps v"),
    ("forward", dict(out=FAKE + 6 * STEP), "out overlaps n_nodes"),
    ("forward", dict(updates=FAKE + 8 * STEP + 16), "updates overlaps out"),
    ("commit", dict(leaf=0), "leaf is NULL"), ("commit", dict(g=FAKE + STEP + 8), "g is not 16-byte"),
    ("commit", dict(state_out=0), "state_out is NULL"),
    ("commit", dict(state_out=FAKE + 2 * STEP), "state_out overlaps updates")])
def test_tree_calls_refuse_buffers(gdn, call, ptrs, word):
    st, msg = refused(gdn, lambda: delta(gdn, call, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_tree_calls_of_nothing(gdn):
    for call in ("forward", "commit"):
        for shape in (dict(n_seqs=0), dict(T=0)):
            delta(gdn, call, shape, k=0, tree=0)
    assert gdn.lib.gdn_tree_forward(None, *[0] * 12) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.lib.gdn_tree_commit(None, *[0] * 9) == gdn.GDN_ERR_INVALID_ARG
    with pytest.raises(KeyError):
        delta(gdn, "forward", mode="other")


def test_device_error_of_a_bad_tree(gdn):
    st, msg = gdn.gdn_decode_device_error(7)
    assert st == gdn.GDN_ERR_DEVICE_ARG and "tree" in msg


def tree_attend(gdn, shape=None, cache=None, nbytes=1 << 23, **kw):
    sh = dict(n_seqs=3, T=2, H=8, max_pages=4, scale=0.0, kv_map=1)
    sh.update(shape or {})
    p = {n: FAKE + i * STEP for i, n in enumerate(
        ("q", "k_cache", "v_cache", "page_table", "lens", "n_nodes", "tree", "out", "workspace"))}
    p.update(kw)
    gdn.gdn_tree_attention(gdn.gdn_attn_shape(*(sh[f[0]] for f in gdn.gdn_attn_shape._fields_)),
                           kv(gdn, **(cache or {})), *p.values(), nbytes)


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_tree_attention_refuses_caches(gdn, cache, status):
    st, msg = refused(gdn, lambda: tree_attend(gdn, cache=cache))
    assert st == status and "gdn_tree_attention" in msg
    assert gdn.gdn_tree_attention_workspace_size(gdn.gdn_attn_shape(3, 2, 8, 4, 0.0, 1),
                                                 kv(gdn, **cache)) == 0


@pytest.mark.parametrize("shape,status", [
    (dict(n_seqs=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(max_pages=-1), 1),
    (dict(kv_map=2), 1), (dict(scale=float("inf")), 1), (dict(n_seqs=1 << 28), 2), (dict(T=65), 2)])
def test_tree_attention_refuses_shapes(gdn, shape, status):
    st, msg = refused(gdn, lambda: tree_attend(gdn, shape))
    assert st == status and "gdn_tree_attention" in msg


@pytest.mark.parametrize("ptrs,word", [
    (dict(q=0), "q is NULL"), (dict(tree=0), "tree is NULL"), (dict(workspace=0), "workspace is"),
    (dict(tree=FAKE + 6 * STEP + 8), "tree is not 16-byte"),
    (dict(n_nodes=FAKE + 5 * STEP + 4), "n_nodes is not 16-byte"),
    (dict(out=FAKE + 6 * STEP), "out overlaps tree"), (dict(out=FAKE + 5 * STEP), "out overlaps n_nodes"),
    (dict(workspace=FAKE + 6 * STEP), "workspace overlaps tree"), (dict(nbytes=1000), "needed")])
def test_tree_attention_refuses_buffers(gdn, ptrs, word):
    st, msg = refused(gdn, lambda: tree_attend(gdn, **ptrs))
    assert st == gdn.GDN_ERR_INVALID_ARG and word in msg


def test_tree_attention_of_nothing(gdn):
    tree_attend(gdn, dict(n_seqs=0), q=0)
    tree_attend(gdn, dict(T=0), tree=0)
    assert gdn.lib.gdn_tree_attention(None, None, *[0] * 11) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.gdn_tree_attention_workspace_size(gdn.gdn_attn_shape(3, 65, 8, 4, 0.0, 1), kv(gdn)) == 0
