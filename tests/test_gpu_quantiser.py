"""gdn_rmsnorm_fp8 as a plain quantiser (normalize = 0) holds its definition
to the last bit: scale = max |y| / 448 and fp8 = y / scale rounded to nearest
even, both in fp32, in each of its forms (few rows, many rows, any columns).
The definition is evaluated on the CPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def quantise(gdn, x):
    rows, cols = x.shape
    q = torch.empty(rows, cols, device="cuda", dtype=torch.uint8)
    s = torch.empty(rows, -(-cols // 128), device="cuda")
    gdn.gdn_rmsnorm_fp8(gdn.gdn_norm_shape(rows, cols, gdn.dtype_code(x.dtype), 0, 0.0, 0.0),
                        x, None, None, None, None, q, s)
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    return q.cpu(), s.cpu()


def definition(x):
    y = x.float().cpu()
    rows, cols = y.shape
    blocks = torch.nn.functional.pad(y, (0, -cols % 128)).view(rows, -1, 128)
    s = (blocks.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
    return (y / s.repeat_interleave(128, 1)[:, :cols]).to(E4M3).view(torch.uint8), s


FORMS = [(300, 256), (300, 4096), (20001, 272), (2500, 2048), (700, 8192), (300, 387), (5, 32776)]


@pytest.mark.parametrize("rows,cols", FORMS)
def test_ties_go_to_even(gdn, rows, cols):
    # whole multiples of c up to 448 c: the scale is c, and the many odd
    # multiples half way between two e4m3 numbers are ties
    g = torch.Generator("cuda")
    g.manual_seed(rows + cols)
    blocks = -(-cols // 128)
    c = 1 + torch.randint(0, 1 << 12, (rows, blocks), generator=g, device="cuda") / 4096.0
    n = torch.randint(-448, 449, (rows, cols), generator=g, device="cuda")
    n[:, ::128] = 448
    x = n * c.repeat_interleave(128, 1)[:, :cols]
    q, s = quantise(gdn, x)
    assert torch.equal(s, c.cpu())
    assert torch.equal(q, n.float().cpu().to(E4M3).view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", FORMS)
def test_every_value(gdn, rows, cols, dtype):
    g = torch.Generator("cuda")
    g.manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    # sizes from the scale's floor to the largest numbers
    x *= 2.0 ** torch.randint(-110, 120, (rows, 1), generator=g, device="cuda")
    q, s = quantise(gdn, x.to(dtype))
    want, scale = definition(x.to(dtype))
    assert torch.equal(s, scale) and torch.equal(q, want)


@pytest.mark.parametrize("cols", [256, 260])
def test_an_infinity_takes_its_block_alone(gdn, cols):
    # inf / inf is no number; the block's other values are 0 beside it
    x = torch.randn(4, cols, device="cuda")
    x[1, 7] = float("inf")
    q, s = quantise(gdn, x)
    v = q.view(E4M3).float()
    assert bool(v[1, 7].isnan()) and int(v.isnan().sum()) == 1
    assert float(s[1, 0]) == float("inf")
    assert bool((v[1, :7] == 0).all()) and bool((v[1, 8:128] == 0).all())
    keep = torch.ones(4, dtype=torch.bool)
    keep[1] = False
    want, scale = definition(x)
    assert torch.equal(q[keep], want[keep]) and torch.equal(s[keep], scale[keep])
    assert torch.equal(q[1, 128:], want[1, 128:])
