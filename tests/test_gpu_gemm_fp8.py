"""gdn_gemm_fp8 against the sum in 64 bits.

Tolerance of an element, with A = sum_b sa sb sum_k |a b|: a product of two
e4m3 numbers is exact in fp32; the tensor cores add 128 of them and the blocks
are added in fp32, so at most 128 + K/128 roundings of 2^-24 of A and the
scales' product: below 1e-5 A for K up to 4096. An output in bf16 is rounded
once more: 2^-8 of the value."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def inputs_of(M, N, K, seed=0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = (torch.randn(M, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
    b = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
    sa = torch.exp(torch.randn(M, kb, generator=g, device="cuda"))
    sb = torch.exp(torch.randn(nb, kb, generator=g, device="cuda"))
    return a, sa, b, sb


def formula(a, sa, b, sb):
    """(out, A) in 64 bits."""
    K, N = a.shape[1], b.shape[0]
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    y = b.double() * sb.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]
    return x @ y.T, x.abs() @ y.abs().T


def call(gdn, a, sa, b, sb, dtype, stream=None):
    M, K = a.shape
    N = b.shape[0]
    # guard rows around the output: nothing may be written beyond it
    guard = torch.full((M * N + 64,), 7.0, device="cuda", dtype=dtype)
    out = guard[32:32 + M * N].view(M, N)
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    gdn.gdn_gemm_fp8(gdn.gdn_gemm_shape(M, N, K, gdn.dtype_code(dtype)), a, sa, b, sb, out, stream)
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    assert bool((guard[:32] == 7).all()) and bool((guard[32 + M * N:] == 7).all())
    return out


def check(out, want, size):
    tol = 1e-5 * size + (2.0 ** -8 * want.abs() if out.dtype == torch.bfloat16 else 0)
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (3, 7, 144), (15, 129, 128), (16, 256, 512), (17, 1000, 2048),
    (32, 2560, 2048), (33, 130, 1040), (64, 384, 4096), (65, 513, 400), (100, 4099, 256),
    (128, 128, 4096), (129, 260, 384), (256, 1024, 1024), (257, 255, 128), (300, 2050, 528),
    (384, 512, 2048), (511, 777, 640), (1000, 3000, 1024), (2049, 1031, 272), (4096, 2048, 512)])
def test_against_the_sum(gdn, M, N, K, dtype):
    x = inputs_of(M, N, K, M + N + K)
    check(call(gdn, *x, dtype), *formula(*x))


@pytest.mark.parametrize("M", [5, 300])
def test_whole_numbers_come_out_exactly(gdn, M):
    # small whole numbers, scales of 1: every sum fits fp32 exactly, so a
    # wrong row, column or block shows as such
    g = torch.Generator("cuda")
    g.manual_seed(1)
    N, K = 390, 1168
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    one = torch.ones(M, -(-K // 128), device="cuda")
    two = torch.ones(-(-N // 128), -(-K // 128), device="cuda")
    out = call(gdn, a.to(E4M3), one, b.to(E4M3), two, torch.float32)
    assert torch.equal(out.double(), a.double() @ b.double().T)


@pytest.mark.parametrize("M", [4, 200, 600])
def test_zero_scales_and_nans_stay_in_their_rows(gdn, M):
    a, sa, b, sb = inputs_of(M, 400, 512, 2)
    a.view(torch.uint8)[1, 300] = 0x7f     # NaN
    sa[2] = 0
    out = call(gdn, a, sa, b, sb, torch.float32)
    assert bool(out[1].isnan().all()) and bool((out[2] == 0).all())
    keep = [i for i in range(M) if i != 1]
    want, size = formula(a, sa, b, sb)
    check(out[keep], want[keep], size[keep])


@pytest.mark.parametrize("M", [8, 64, 128, 700])
def test_the_same_bits_every_time_streams_and_graphs(gdn, M):
    x = inputs_of(M, 1536, 2048, 3)
    first = call(gdn, *x, torch.float32)
    side = torch.cuda.Stream()
    for _ in range(5):
        assert torch.equal(call(gdn, *x, torch.float32, side), first)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            gdn.gdn_gemm_fp8(gdn.gdn_gemm_shape(M, 1536, 2048, gdn.GDN_F32), *x, out,
                             torch.cuda.current_stream())
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    assert torch.equal(out, first)
