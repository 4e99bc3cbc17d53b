"""gdn_qknorm_rope_append against the norm and the rotation in 64 bits.

Tolerance of an element made from the normed pair (a, b): the sum of D <= 256
squares is off by at most 24 roundings of 2^-24 (a chain of 16 terms and 8
halvings), of which the root keeps half; quotient, root, weight's offset and
two products add six more: 18 x 2^-24 < 1.1e-6 of each of a and b. The rotation
adds 3e-6 (|a| + |b|) (the angle at most 2e-6, the rest a handful of 2^-24). An
element that is not rotated has 1.1e-6 of itself. 2^-8 of the value where it is
rounded to bf16. v and whatever no slot names: equal bits."""
import pytest
import torch

from test_gpu_rope_append import LAYOUTS, TYPES, axis_of_freq, gdn, make_cache, rotated  # noqa: F401

pytestmark = pytest.mark.gpu


def normed(x, w, offset, eps):
    x = x.double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * (offset + w.double())


def check(got, y, pos, inv, axis, rot, neighbours):
    want, size = rotated(y, pos, inv, axis, rot, neighbours)
    size = torch.where(size == 0, want.abs() * (1.1 / 4.1), size)
    tol = 4.1e-6 * size + (2.0 ** -8 * want.abs() if got.dtype == torch.bfloat16 else 0)
    assert bool(((got.double() - want).abs() <= tol).all())


def run(gdn, n, H, H_kv, D, rot, sec, interleaved, neighbours, page, dtype, layout="dense",
        max_pos=4096, fused=True, seed=0, slots=None, expect=None, stream=None, offset=0.0,
        eps=1e-6, weights="both", std=3.0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    wide = (H + 2 * H_kv) * D if fused else 0
    if fused:
        qkv = (std * torch.randn(n, wide, generator=g, device="cuda")).to(dtype)
        q = qkv[:, :H * D].unflatten(1, (H, D))
        k = qkv[:, H * D:(H + H_kv) * D].unflatten(1, (H_kv, D))
        v = qkv[:, (H + H_kv) * D:].unflatten(1, (H_kv, D))
    else:
        q, k, v = ((std * torch.randn(n, h, D, generator=g, device="cuda")).to(dtype)
                   for h in (H, H_kv, H_kv))
    qw = (torch.randn(D, generator=g, device="cuda")).to(dtype) if weights != "k" else None
    kw = (torch.randn(D, generator=g, device="cuda")).to(dtype) if weights != "q" else None
    half = rot // 2
    pos = torch.randint(0, max_pos, (len(sec), n), generator=g, device="cuda", dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()
    pages = -(-n // page) + 2
    cache, kc, vc = make_cache(gdn, layout, pages, page, H_kv, D, dtype)
    if slots is None:
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].contiguous()
    k0, v0 = kc.clone(), vc.clone()
    q_out = torch.full((n, H, D), float("nan"), device="cuda", dtype=dtype)
    shape = gdn.gdn_rope_shape(
        n, H, rot, int(neighbours), len(sec), (gdn.c_int * 4)(*sec), int(interleaved),
        wide, wide, wide)
    torch.cuda.synchronize()
    gdn.gdn_qknorm_rope_append(shape, cache, gdn.gdn_qk_norm(eps, offset), q, k, v, qw, kw, pos,
                               inv, slots, q_out, kc, vc, stream)
    torch.cuda.synchronize()
    if expect:
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_check_device_error()
        assert e.value.status == expect
    else:
        gdn.gdn_check_device_error()
    axis = axis_of_freq(sec, half, interleaved)
    check(q_out, normed(q, qw, offset, eps), pos, inv, axis, rot, neighbours)
    use = (slots >= 0) & (slots < pages * page)
    at = slots[use]
    check(kc[at // page, at % page], normed(k, kw, offset, eps)[use], pos[:, use], inv, axis, rot,
          neighbours)
    assert torch.equal(vc[at // page, at % page], v[use])
    keep = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    keep[at // page, at % page] = False
    assert torch.equal(kc[keep], k0[keep]) and torch.equal(vc[keep], v0[keep])
    return q_out, kc.clone()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot,sec,interleaved", [
    ("all", (1,), False), ("all", (2, 1, 1), True), (2, (1, 0), True), (50, (25,), False),
    (16, (8,), False), (36, (8, 6, 4), True), (32, (16,), False), (0, (0, 0), False)])
def test_norms_and_rotations(gdn, dtype, D, neighbours, rot, sec, interleaved):
    if rot == "all":
        rot = D
        sec = tuple(s * D // 2 // sum(sec) for s in sec)
        if interleaved:
            each = D // 2 // 3
            sec = (D // 2 - 2 * each, each, each)
    run(gdn, 37, 6, 3, D, rot, sec, interleaved, neighbours, 7, dtype, seed=rot + D)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weights,offset,eps", [("both", 1.0, 1e-6), ("q", 0.0, 1e-2), ("k", 1.0, 0.0)])
def test_cache_layouts_and_weights(gdn, layout, dtype, weights, offset, eps):
    run(gdn, 100, 4, 2, 128, 64, (16, 8, 8), False, False, 16, dtype, layout=layout,
        weights=weights, offset=offset, eps=eps)


@pytest.mark.parametrize("n", [1, 2, 9, 1000])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (16, 2), (8, 8), (40, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_counts_and_dense_rows(gdn, n, H, H_kv, D):
    run(gdn, n, H, H_kv, D, D, (D // 2,), False, False, 16, torch.bfloat16, fused=False, seed=n)


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot", [256, 90])
@pytest.mark.parametrize("n,H,H_kv,dtype", [(40, 70, 2, torch.float32), (3, 128, 64, torch.bfloat16)])
def test_rows_of_many_wide_heads(gdn, neighbours, rot, n, H, H_kv, dtype):
    run(gdn, n, H, H_kv, 256, rot, (rot // 2 - 9, 9), True, neighbours, 16, dtype, seed=n)


@pytest.mark.parametrize("std", [1e-12, 1e15])
@pytest.mark.parametrize("dtype", TYPES)
def test_tiny_and_huge_heads(gdn, std, dtype):
    # the squares stay inside fp32: 1e30 x 256, and 1e-24 beside an eps of 1e-6
    run(gdn, 50, 4, 2, 128, 128, (64,), False, False, 16, dtype, std=std)


def test_heads_of_zeros_stay_zero(gdn):
    q, kc = run(gdn, 5, 4, 2, 64, 64, (32,), False, False, 16, torch.bfloat16, std=0.0)
    assert not bool(q.any())


def test_padding_and_slots_beyond_the_cache(gdn):
    pages = -(-6 // 4) + 2
    slots = torch.tensor([3, -1, 0, -7, 8, 2], device="cuda")
    run(gdn, 6, 4, 2, 64, 64, (32,), False, False, 4, torch.bfloat16, slots=slots)
    slots = torch.tensor([3, 4 * pages, 0, 1 << 60, 8, 2], device="cuda")
    run(gdn, 6, 4, 2, 64, 64, (32,), False, False, 4, torch.bfloat16, slots=slots,
        expect=gdn.GDN_ERR_DEVICE_ARG)


def test_on_another_stream_and_again(gdn):
    a = run(gdn, 70, 4, 2, 128, 128, (64,), False, False, 16, torch.bfloat16, seed=4)
    b = run(gdn, 70, 4, 2, 128, 128, (64,), False, False, 16, torch.bfloat16, seed=4,
            stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,H,H_kv,D,rot,sec,neighbours,layout", [
    (1217, 2, 1, 64, 64, (32,), False, "dense"), (5003, 4, 1, 64, 64, (20, 12), True, "heads_first"),
    (5003, 6, 2, 128, 90, (45,), False, "k_and_v_in_one"), (4999, 1, 1, 256, 256, (128,), True, "dense"),
    (7001, 3, 1, 64, 2, (1,), False, "dense"), (4864, 2, 2, 64, 0, (0,), False, "heads_first")])
def test_many_short_rows(gdn, dtype, n, H, H_kv, D, rot, sec, neighbours, layout):
    slots = torch.randperm(n, device="cuda")
    slots[::7] = -1
    run(gdn, n, H, H_kv, D, rot, sec, False, neighbours, 16, dtype, layout=layout, seed=n,
        slots=slots)


def test_the_rotation_alone_is_gdn_rope_append(gdn):
    # heads whose mean square is 1 by construction: the norm changes nothing but
    # by its own rounding, so the two calls agree to the rotation's tolerance
    n, H, D = 64, 4, 64
    x = torch.randn(n, H + 4, D, device="cuda").sign()
    q, k, v = x[:, :H].contiguous(), x[:, H:H + 2].contiguous(), x[:, H + 2:].contiguous()
    pos = torch.randint(0, 4096, (1, n), device="cuda", dtype=torch.int32)
    inv = torch.rand(32, device="cuda")
    slots = torch.arange(n, device="cuda")
    cache = gdn.gdn_kv_cache(4, 16, 2, D, gdn.GDN_F32, 0, 0, 0)
    shape = gdn.gdn_rope_shape(n, H, D, 0, 1, (gdn.c_int * 4)(32), 0, 0, 0, 0)
    got = []
    for norm in (False, True):
        kc, vc = (torch.zeros(4, 16, 2, D, device="cuda") for _ in range(2))
        out = torch.empty_like(q)
        if norm:
            gdn.gdn_qknorm_rope_append(shape, cache, gdn.gdn_qk_norm(0.0, 1.0), q, k, v, None, None,
                                       pos, inv, slots, out, kc, vc)
        else:
            gdn.gdn_rope_append(shape, cache, q, k, v, pos, inv, slots, out, kc, vc)
        gdn.gdn_check_device_error()
        got.append((out, kc, vc))
    for a, b in zip(*got):
        assert bool(((a - b).abs() <= 2 * 4.1e-6 * 2).all())
