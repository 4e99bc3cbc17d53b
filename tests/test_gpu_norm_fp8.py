"""gdn_rmsnorm_fp8 against the formula in 64 bits.

Tolerances, per element. fp32 arithmetic: at most 140 roundings of 2^-24 enter
a row's sum (chains of at most 129 products, then the reduction), which count
half in the root, and six more follow: 5e-6. An output in bf16 adds its own
rounding of 2^-8 (eight significant bits). e4m3 keeps four: half a unit is 2^-4 of the
value, and 2^-10 of the scale below the smallest normal number."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32 = 5e-6
OUT = {torch.float32: F32, torch.bfloat16: 2.0 ** -8 + F32}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def inputs_of(rows, cols, dtype, seed=0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * 3
    r = torch.randn(rows, cols, generator=g, device="cuda")
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    return x.to(dtype), r.to(dtype), w.to(dtype)


def call(gdn, x, r, w, normalize=1, eps=1e-6, w_off=0.0, res_out=None, out=None, fp8=True,
         stream=None):
    rows, cols = x.shape
    q = torch.full((rows, cols), 0x7f, device="cuda", dtype=torch.uint8) if fp8 else None
    s = torch.full((rows, -(-cols // 128)), -1.0, device="cuda") if fp8 else None
    shape = gdn.gdn_norm_shape(rows, cols, gdn.dtype_code(x.dtype), normalize, eps, w_off)
    torch.cuda.synchronize()
    gdn.gdn_rmsnorm_fp8(shape, x, r, w, res_out, out, q, s, stream)
    torch.cuda.synchronize()
    return (q.view(E4M3) if fp8 else None), s


def formula(x, r, w, normalize=1, eps=1e-6, w_off=0.0):
    h = x.double() + (0 if r is None else r.double())
    y = h
    if normalize:
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
        if w is not None:
            y = y * (w_off + w.double())
    return h, y


def close(got, want, tol):
    assert bool(((got.double() - want).abs() <= tol * want.abs() + 1e-30).all())


def check_fp8(q, s, y):
    rows, cols = y.shape
    blocks = torch.nn.functional.pad(y, (0, -cols % 128)).view(rows, -1, 128)
    want = (blocks.abs().amax(-1) / 448).clamp_min(2.0 ** -100)
    close(s, want, F32 + 2.0 ** -22)
    scale = s.double().repeat_interleave(128, 1)[:, :cols]
    v = y / scale
    err = (q.double() - v).abs()
    assert bool((err <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 1e-3)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [
    (1, 1), (1, 8), (3, 127), (2, 128), (5, 129), (7, 136), (64, 256), (33, 264), (9, 1000),
    (17, 2048), (3, 2056), (5, 4096), (4, 4104), (3, 8200), (2, 9999), (2, 16392), (2, 32768),
    (2, 32776)])
def test_against_the_formula(gdn, rows, cols, dtype):
    x, r, w = inputs_of(rows, cols, dtype, rows * cols)
    out, res = torch.empty_like(x), torch.empty_like(x)
    q, s = call(gdn, x, r, w, res_out=res, out=out)
    h, y = formula(x, r, w)
    close(res, h, OUT[dtype])
    close(out, y, OUT[dtype])
    check_fp8(q, s, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(40001, 16), (20001, 272), (5003, 2048), (3001, 2064),
                                       (2001, 4096), (1501, 8192), (700, 10000)])
def test_many_rows(gdn, rows, cols, residual, dtype):
    x, r, w = inputs_of(rows, cols, dtype, rows + cols)
    r = r if residual else None
    out = torch.empty_like(x)
    res = torch.empty_like(x) if residual else None
    q, s = call(gdn, x, r, w, res_out=res, out=out, w_off=0.5)
    h, y = formula(x, r, w, w_off=0.5)
    if residual:
        close(res, h, OUT[dtype])
    close(out, y, OUT[dtype])
    check_fp8(q, s, y)
    # in place, and outputs that start on 16 bytes only
    wide = torch.empty(rows * cols + 16, device="cuda", dtype=dtype)
    off = wide[16 // wide.element_size():][:rows * cols].view(rows, cols)
    call(gdn, x, r, w, res_out=r, out=off, w_off=0.5)
    assert torch.equal(off, out) and (not residual or torch.equal(r, res))


@pytest.mark.parametrize("cols", [1024, 1001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_options(gdn, dtype, cols):
    x, r, w = inputs_of(6, cols, dtype, 5)
    # weights around zero, no residual, only the unquantised output
    out = torch.empty_like(x)
    call(gdn, x, None, w, w_off=1.0, eps=0.1, out=out, fp8=False)
    close(out, formula(x, None, w, eps=0.1, w_off=1.0)[1], OUT[dtype])
    # no weight
    q, s = call(gdn, x, r, None)
    check_fp8(q, s, formula(x, r, None)[1])
    # the plain quantiser of a sum
    res = torch.empty_like(x)
    q, s = call(gdn, x, r, None, normalize=0, res_out=res)
    h, y = formula(x, r, None, normalize=0)
    close(res, h, OUT[dtype])
    check_fp8(q, s, y)


@pytest.mark.parametrize("cols", [512, 515, 40000])
def test_in_place(gdn, cols):
    x, r, w = inputs_of(9, cols, torch.bfloat16, 6)
    h, y = formula(x, r, w)
    q, s = call(gdn, x, r, w, res_out=r, out=x)
    close(r, h, OUT[torch.bfloat16])
    close(x, y, OUT[torch.bfloat16])
    check_fp8(q, s, y)


@pytest.mark.parametrize("cols", [384, 390])
def test_zeros_tiny_values_and_nans(gdn, cols):
    x, _, w = inputs_of(5, cols, torch.float32, 7)
    x[0] = 0                     # a row of zeros: rstd is finite through eps
    x[1, 128:256] = 0            # a block of zeros
    x[2] *= 1e-20                # h^2 underflows: the row stays near zero
    x[3, 5] = float("nan")
    w[:] = 1
    q, s = call(gdn, x, None, w)
    q, s = q.double(), s.double()
    assert bool((q[0] == 0).all()) and bool((s[0] == 2.0 ** -100).all())
    assert bool((q[1, 128:256] == 0).all()) and float(s[1, 1]) == 2.0 ** -100
    check_fp8(q[2:3], s[2:3], formula(x, None, w)[1][2:3])
    assert bool(q[3].isnan().all()) and bool(s[3].isfinite().all())
    check_fp8(q[4:], s[4:], formula(x, None, w)[1][4:])


def test_a_nan_stays_in_its_place_without_the_norm(gdn):
    x, _, _ = inputs_of(2, 256, torch.bfloat16, 8)
    x[0, 3] = float("nan")
    q, s = call(gdn, x, None, None, normalize=0)
    assert bool(q.double()[0, 3].isnan()) and int(q.double().isnan().sum()) == 1
    y = x.double().nan_to_num(0.0)
    check_fp8(q.double().nan_to_num(0.0), s, y)


def test_on_another_stream_and_in_a_graph(gdn):
    x, r, w = inputs_of(40, 2048, torch.bfloat16, 9)
    q0, s0 = call(gdn, x, r, w)
    side = torch.cuda.Stream()
    q1, s1 = call(gdn, x, r, w, stream=side)
    assert torch.equal(q0.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s0, s1)
    shape = gdn.gdn_norm_shape(40, 2048, gdn.GDN_BF16, 1, 1e-6, 0.0)
    q2, s2 = torch.zeros_like(q0.view(torch.uint8)), torch.zeros_like(s0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_rmsnorm_fp8(shape, x, r, w, None, None, q2, s2, torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, q0.view(torch.uint8)) and torch.equal(s2, s0)
