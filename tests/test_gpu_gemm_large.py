"""gdn_gemm_fp8 where it has more than one 128 x 128 tile for each of 152 SMs,
so that pairs of blocks take 256 x 256 tiles: several tiles a pair, and k long
enough for the groups of eight stages' scales to come round more than once.
Tolerances as in test_gpu_gemm_fp8.py."""
import pytest
import torch

from test_gpu_gemm_fp8 import E4M3, TYPES, call, check, formula, inputs_of

pytestmark = pytest.mark.gpu

SMS = 152


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def is_large(M, N):
    return M > 64 and -(-M // 128) * -(-N // 128) > SMS


def tiles_of_a_pair(M, N):
    return -(-(-(-M // 256) * -(-N // 256)) // (SMS // 2))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,tiles", [
    (1100, 3000, 3344, 1), (1100, 3001, 3344, 1), (2049, 2055, 1040, 2), (2304, 6144, 1152, 3),
    (2300, 6151, 1136, 3), (65, 20000, 400, 2), (20000, 130, 2064, 2), (4100, 8200, 144, 8)])
def test_against_the_sum(gdn, M, N, K, tiles, dtype):
    assert is_large(M, N) and tiles_of_a_pair(M, N) == tiles
    x = inputs_of(M, N, K, M + N + K)
    check(call(gdn, *x, dtype), *formula(*x))


@pytest.mark.parametrize("N", [6000, 6003])
def test_whole_numbers_come_out_exactly(gdn, N):
    g = torch.Generator("cuda")
    g.manual_seed(1)
    M, K = 700, 3216
    assert is_large(M, N)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    # powers of two that differ by row and block: a wrong scale shows as such
    sa = 2.0 ** torch.randint(-2, 3, (M, -(-K // 128)), generator=g, device="cuda")
    sb = 2.0 ** torch.randint(-2, 3, (-(-N // 128), -(-K // 128)), generator=g, device="cuda")
    x = (a.to(E4M3), sa, b.to(E4M3), sb)
    assert torch.equal(call(gdn, *x, torch.float32).double(), formula(*x)[0])


@pytest.mark.parametrize("N", [4096, 4099])
def test_zero_scales_and_nans_stay_in_their_rows(gdn, N):
    M = 1000
    assert is_large(M, N)
    a, sa, b, sb = inputs_of(M, N, 2064, 2)
    a.view(torch.uint8)[1, 2050] = 0x7f     # NaN
    sa[2] = 0
    out = call(gdn, a, sa, b, sb, torch.float32)
    assert bool(out[1].isnan().all()) and bool((out[2] == 0).all())
    keep = [i for i in range(M) if i != 1]
    want, size = formula(a, sa, b, sb)
    check(out[keep], want[keep], size[keep])


@pytest.mark.parametrize("N", [6144, 6145])
def test_the_same_bits_every_time_streams_and_graphs(gdn, N):
    M, K = 1500, 2304
    assert is_large(M, N)
    x = inputs_of(M, N, K, 3)
    first = call(gdn, *x, torch.float32)
    side = torch.cuda.Stream()
    for _ in range(5):
        assert torch.equal(call(gdn, *x, torch.float32, side), first)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            gdn.gdn_gemm_fp8(gdn.gdn_gemm_shape(M, N, K, gdn.GDN_F32), *x, out,
                             torch.cuda.current_stream())
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    assert torch.equal(out, first)
