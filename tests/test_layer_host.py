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
