"""gdn_rope_append against the rotation in 64 bits.

Tolerance of an element rotated from (a, b): the angle is off by at most 2e-6
(a handful of fp32 roundings of a turn), sine and cosine by two units of 2^-24
and the two products and the sum by one each: (|a| + |b|) 3e-6, and 2^-8 of
the value where it is rounded to bf16. Elements that are not rotated are
copied: equal bits, and so is everything in the cache that no slot names."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def axis_of_freq(sec, half, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    n = len(sec)
    return [i % n if i // n < sec[i % n] else 0 for i in range(half)]


def rotated(x, pos, inv_freq, axis, rot, neighbours):
    """(value, |a| + |b|) in 64 bits."""
    x = x.double().clone()
    size = torch.zeros_like(x)
    half = rot // 2
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
    ang = (pos.double()[axis] * inv_freq.double()[:, None]).T[:, None]
    xa, xb = x[..., a], x[..., b]
    x[..., a], x[..., b] = xa * ang.cos() - xb * ang.sin(), xa * ang.sin() + xb * ang.cos()
    size[..., a] = size[..., b] = xa.abs() + xb.abs()
    return x, size


def check(got, want, size, rot):
    tol = 3e-6 * size + (2.0 ** -8 * want.abs() if got.dtype == torch.bfloat16 else 0)
    assert bool(((got.double() - want).abs() <= tol).all())


LAYOUTS = ["dense", "heads_first", "k_and_v_in_one"]


def make_cache(gdn, layout, pages, page, H_kv, D, dtype):
    """(struct, k, v) with k, v viewed as [pages, page, H_kv, D]."""
    code = gdn.dtype_code(dtype)
    if layout == "dense":
        k = torch.randn(pages, page, H_kv, D, device="cuda").to(dtype)
        v = torch.randn(pages, page, H_kv, D, device="cuda").to(dtype)
        return gdn.gdn_kv_cache(pages, page, H_kv, D, code, 0, 0, 0), k, v
    if layout == "heads_first":
        k = torch.randn(pages, H_kv, page, D, device="cuda").to(dtype)
        v = torch.randn(pages, H_kv, page, D, device="cuda").to(dtype)
        return (gdn.gdn_kv_cache(pages, page, H_kv, D, code, H_kv * page * D, D, page * D),
                k.transpose(1, 2), v.transpose(1, 2))
    kv = torch.randn(pages, 2, page, H_kv, D, device="cuda").to(dtype)
    return (gdn.gdn_kv_cache(pages, page, H_kv, D, code, 2 * page * H_kv * D, H_kv * D, D),
            kv[:, 0], kv[:, 1])


def run(gdn, n, H, H_kv, D, rot, sec, interleaved, neighbours, page, dtype, layout="dense",
        max_pos=4096, fused=True, seed=0, slots=None, expect=None, stream=None):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    wide = (H + 2 * H_kv) * D if fused else 0
    if fused:
        qkv = torch.randn(n, wide, generator=g, device="cuda").to(dtype)
        q = qkv[:, :H * D].unflatten(1, (H, D))
        k = qkv[:, H * D:(H + H_kv) * D].unflatten(1, (H_kv, D))
        v = qkv[:, (H + H_kv) * D:].unflatten(1, (H_kv, D))
    else:
        q = torch.randn(n, H, D, generator=g, device="cuda").to(dtype)
        k = torch.randn(n, H_kv, D, generator=g, device="cuda").to(dtype)
        v = torch.randn(n, H_kv, D, generator=g, device="cuda").to(dtype)
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
    gdn.gdn_rope_append(shape, cache, q, k, v, pos, inv, slots, q_out, kc, vc, stream)
    torch.cuda.synchronize()
    if expect:
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_check_device_error()
        assert e.value.status == expect
    else:
        gdn.gdn_check_device_error()
    axis = axis_of_freq(sec, half, interleaved)
    want, size = rotated(q, pos, inv, axis, rot, neighbours)
    check(q_out, want, size, rot)
    assert torch.equal(q_out[..., rot:], q[..., rot:])
    use = (slots >= 0) & (slots < pages * page)
    at = slots[use]
    want, size = rotated(k, pos, inv, axis, rot, neighbours)
    check(kc[at // page, at % page], want[use], size[use], rot)
    assert torch.equal(kc[at // page, at % page][..., rot:], k[use][..., rot:])
    assert torch.equal(vc[at // page, at % page], v[use])
    keep = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    keep[at // page, at % page] = False
    assert torch.equal(kc[keep], k0[keep]) and torch.equal(vc[keep], v0[keep])
    return q_out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot,sec,interleaved", [
    ("all", (1,), False), ("all", (2, 1, 1), False), ("all", (2, 1, 1), True), (2, (1, 0), True),
    (50, (25,), False), (30, (5, 4, 6), False), (36, (8, 6, 4), True), (0, (0, 0), False)])
def test_rotations(gdn, dtype, D, neighbours, rot, sec, interleaved):
    if rot == "all":
        rot = D
        sec = tuple(s * D // 2 // sum(sec) for s in sec)
        if interleaved:   # turns: no axis may have more than its places
            each = D // 2 // 3
            sec = (D // 2 - 2 * each, each, each)
    run(gdn, 37, 6, 3, D, rot, sec, interleaved, neighbours, 7, dtype, seed=rot + D)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 16, 33])
@pytest.mark.parametrize("dtype", TYPES)
def test_cache_layouts(gdn, layout, page, dtype):
    run(gdn, 100, 4, 2, 128, 64, (16, 8, 8), False, False, page, dtype, layout=layout, seed=page)


@pytest.mark.parametrize("n", [1, 2, 9, 1000])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (16, 2), (8, 8)])
def test_counts_and_dense_rows(gdn, n, H, H_kv):
    run(gdn, n, H, H_kv, 64, 64, (32,), False, False, 16, torch.bfloat16, fused=False, seed=n)


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot", [256, 90])
@pytest.mark.parametrize("n,H,H_kv,dtype", [(40, 70, 2, torch.float32), (3, 128, 64, torch.bfloat16)])
def test_rows_of_many_wide_heads(gdn, neighbours, rot, n, H, H_kv, dtype):
    run(gdn, n, H, H_kv, 256, rot, (rot // 2 - 9, 9), True, neighbours, 16, dtype, seed=n)


@pytest.mark.parametrize("max_pos", [131072, 1 << 24])
def test_long_positions_keep_their_angles(gdn, max_pos):
    run(gdn, 500, 2, 1, 128, 128, (64,), False, False, 16, torch.float32, max_pos=max_pos)


def test_padding_and_slots_beyond_the_cache(gdn):
    slots = torch.tensor([3, -1, 0, -7, 8, 2], device="cuda")
    run(gdn, 6, 4, 2, 64, 64, (32,), False, False, 4, torch.bfloat16, slots=slots)
    pages = -(-6 // 4) + 2
    slots = torch.tensor([3, 4 * pages, 0, 1 << 60, 8, 2], device="cuda")
    run(gdn, 6, 4, 2, 64, 64, (32,), False, False, 4, torch.bfloat16, slots=slots,
        expect=gdn.GDN_ERR_DEVICE_ARG)


def test_a_cache_beyond_32_bits_of_elements(gdn):
    # one page every 2^26 elements (128 MiB): page 39 starts past 2^31 elements
    pages, page, H_kv, D = 40, 16, 2, 64
    stride = 1 << 26
    store = torch.zeros(pages * stride, device="cuda", dtype=torch.bfloat16)
    size = (pages, page, H_kv, D)
    kc = store.as_strided(size, (stride, H_kv * D, D, 1))
    vc = store.as_strided(size, (stride, H_kv * D, D, 1), 1 << 20)
    cache = gdn.gdn_kv_cache(pages, page, H_kv, D, gdn.GDN_BF16, stride, H_kv * D, D)
    q = torch.randn(2, 2, D, device="cuda").bfloat16()
    k, v = torch.randn_like(q), torch.randn_like(q)
    slots = torch.tensor([39 * page + 5, 0], device="cuda")
    pos = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    inv = torch.ones(32, device="cuda")
    q_out = torch.empty_like(q)
    gdn.gdn_rope_append(gdn.gdn_rope_shape(2, 2, 64, 0, 1, (gdn.c_int * 4)(32), 0, 0, 0, 0), cache,
                        q, k, v, pos, inv, slots, q_out, kc, vc)
    gdn.gdn_check_device_error()
    assert torch.equal(kc[39, 5], k[0]) and torch.equal(vc[39, 5], v[0])
    assert torch.equal(kc[0, 0], k[1]) and torch.equal(vc[0, 0], v[1])
    assert torch.equal(q_out, q)     # position 0 turns nothing


def test_on_another_stream(gdn):
    a = run(gdn, 70, 4, 2, 128, 128, (64,), False, False, 16, torch.bfloat16, seed=4)
    b = run(gdn, 70, 4, 2, 128, 128, (64,), False, False, 16, torch.bfloat16, seed=4,
            stream=torch.cuda.Stream())
    assert torch.equal(a, b)


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
