"""gdn_sample against its definition in 64 bits, row by row on the CPU.

Tokens have to be equal: weights are off by at most some 2^-29 of themselves and
their sums are exact, so a token differs from the definition's only where u * mass
lies that near the edge between two tokens (2^-29 of the mass for each of some
1000 tokens with weight: 2e-6 of all rows). prob = w / mass: 2^-24 for its own
rounding, 2^-28 for the weight and the mass, a unit of 2^-44 of the largest, and
what tokens below 2^-44.9 leave out of the mass, 2^18 x 2^-44.9 of it (2^-26.9): less than
2^-22 prob + 2^-38 in all."""
import math

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


def reference(x, temperature, top_k, top_p, min_p, u):
    """(token, prob) of one row, x in 64 bits on the CPU."""
    x = torch.where(x.isnan(), -math.inf, x)
    V, top = x.numel(), x.max()
    if top == -math.inf:
        return -1, 0.0
    order = torch.argsort(x, descending=True, stable=True)
    if not temperature > 0:
        return int(order[0]), 1.0
    w = torch.where(x == top, 1.0, torch.exp((x - top) / temperature) if top < math.inf else 0.0)
    n = min(top_k, V) if top_k > 0 else V
    w_in = w[order]
    if top_p < 1:
        run = w_in[:n].cumsum(0)
        past = (run >= top_p * run[-1]).nonzero()
        m = int(past[0]) + 1 if len(past) else n
    else:
        m = n
    if min_p > 0:
        m = min(m, int((w_in >= min_p).sum()))
    kept = order[:max(m, 1)].sort().values
    run = w[kept].cumsum(0)
    past = (run > (0.0 if not u > 0 else u) * run[-1]).nonzero()
    live = (w[kept] > 0).nonzero()
    at = int(past[0]) if len(past) else int(live[-1])
    return int(kept[at]), float(w[kept[at]] / run[-1])


def run(gdn, x, temperature=None, top_k=None, top_p=None, min_p=None, u=None, stride=0, probs=True,
        stream=None, check=True):
    rows, V = x.shape
    dev = [None if t is None else t.cuda() for t in (temperature, top_k, top_p, min_p)]
    u = torch.rand(rows) if u is None else u
    tokens = torch.full((rows,), -7, device="cuda", dtype=torch.int32)
    out = torch.full((rows,), float("nan"), device="cuda") if probs else None
    ud = u.cuda()
    torch.cuda.synchronize()
    gdn.gdn_sample(gdn.gdn_sample_shape(rows, V, gdn.dtype_code(x.dtype), stride), x, *dev, ud,
                   tokens, out, stream)
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    if check:
        xd = x.double().cpu()
        for i in range(rows):
            want, p = reference(
                xd[i], 1.0 if temperature is None else float(temperature[i]),
                0 if top_k is None else int(top_k[i]), 1.0 if top_p is None else float(top_p[i]),
                0.0 if min_p is None else float(min_p[i]), float(u[i]))
            assert int(tokens[i]) == want, (i, int(tokens[i]), want)
            if probs:
                assert abs(float(out[i]) - p) <= 2.0 ** -22 * p + 2.0 ** -38, (i, float(out[i]), p)
    return tokens, out


def logits(rows, V, dtype, seed, std=2.5):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    torch.manual_seed(seed)
    x = torch.randn(rows, V, generator=g, device="cuda") * std
    spikes = torch.rand(rows, V, generator=g, device="cuda") < 5.0 / V
    return (x + 8 * spikes).to(dtype)


SETTINGS = {
    "none": lambda n: {},
    "warm": lambda n: dict(temperature=0.3 + 1.5 * torch.rand(n)),
    "top_k": lambda n: dict(top_k=torch.randint(1, 60, (n,), dtype=torch.int32)),
    "top_p": lambda n: dict(top_p=torch.rand(n)),
    "min_p": lambda n: dict(min_p=0.2 * torch.rand(n)),
    "k and p": lambda n: dict(top_k=torch.randint(1, 2000, (n,), dtype=torch.int32),
                              top_p=0.5 + 0.5 * torch.rand(n)),
    "all": lambda n: dict(temperature=0.5 + torch.rand(n),
                          top_k=torch.randint(-1, 300, (n,), dtype=torch.int32),
                          top_p=0.6 + 0.5 * torch.rand(n), min_p=0.05 * torch.rand(n) - 0.01),
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V", [(5, 1), (4, 2), (9, 31), (3, 1000), (2, 4097), (70, 777),
                                    (3, 50257), (200, 8192), (2, 131072), (1, 262144)])
@pytest.mark.parametrize("setting", SETTINGS)
def test_settings(gdn, dtype, rows, V, setting):
    x = logits(rows, V, dtype, seed=rows + V)
    run(gdn, x, **SETTINGS[setting](rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("levels", [1, 2, 5])
@pytest.mark.parametrize("setting", ["none", "top_k", "top_p", "k and p", "all"])
def test_ties(gdn, dtype, levels, setting):
    g = torch.Generator("cuda").manual_seed(levels)
    torch.manual_seed(levels)
    x = torch.randint(0, levels, (12, 3001), generator=g, device="cuda").to(dtype)
    run(gdn, x, **SETTINGS[setting](12))


def test_half_of_two_equal_tokens(gdn):
    # masses that meet the bound exactly: 0.5 of two equal weights is one token
    x = torch.zeros(4, 2, device="cuda")
    tokens, probs = run(gdn, x, top_p=torch.tensor([0.5, 0.50001, 0.0, 1.0]),
                        u=torch.tensor([0.99, 0.99, 0.99, 0.4999]))
    assert tokens.tolist() == [0, 1, 0, 0] and probs.tolist() == [1.0, 0.5, 1.0, 0.5]


def test_zeros_of_both_signs_are_equal(gdn):
    x = torch.tensor([[-0.0, 0.0, -1.0], [0.0, -0.0, -1.0]], device="cuda")
    k = torch.ones(2, dtype=torch.int32)
    assert run(gdn, x, top_k=k)[0].tolist() == [0, 0]
    assert run(gdn, x.bfloat16(), temperature=torch.zeros(2))[0].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_rows(gdn, dtype):
    x = logits(8, 2000, dtype, seed=3)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, :1999] = math.nan
    x[4, 5] = x[4, 900] = math.inf
    x[5, ::2] = -math.inf
    x[6, 100:] = math.nan
    x[7, 7], x[7, 8] = math.inf, math.nan
    for setting in SETTINGS:
        torch.manual_seed(1)
        tokens, _ = run(gdn, x, **SETTINGS[setting](8))
        assert tokens[:4].tolist() == [-1, -1, 0, 1999]


@pytest.mark.parametrize("dtype", TYPES)
def test_greedy_takes_the_first_of_the_largest(gdn, dtype):
    x = logits(6, 9000, dtype, seed=4).round()
    t = torch.tensor([0.0, -1.0, math.nan, 0.0, 1.0, 1.0])
    k = torch.tensor([0, 0, 5, 7, 1, 0], dtype=torch.int32)
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, 1.5])
    tokens, _ = run(gdn, x, temperature=t, top_k=k, min_p=m)
    assert torch.equal(tokens.cpu(), x.float().argmax(1).int().cpu())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,shift,temperature", [
    (1e-3, 0.0, 1e-3), (1.0, 1e4, 1.0), (1e4, 0.0, 5.0), (1.0, 0.0, 1e6), (1.0, 0.0, math.inf),
    (1e30, 0.0, 1e30), (1.0, -3e4, 0.05)])
def test_scales_of_logits(gdn, dtype, scale, shift, temperature):
    x = (logits(6, 5000, torch.float32, seed=5) * scale + shift).to(dtype)
    t = torch.full((6,), temperature)
    run(gdn, x, temperature=t)
    run(gdn, x, temperature=t, top_p=torch.linspace(0.1, 0.95, 6))
    run(gdn, x, temperature=t, top_k=torch.arange(1, 1200, 200, dtype=torch.int32))


def test_ends_of_the_random_number(gdn):
    x = logits(6, 3000, torch.float32, seed=6)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 5.0, -1.0, math.nan])
    run(gdn, x, u=u)
    run(gdn, x, u=u, top_p=torch.full((6,), 0.8))


def test_limits_that_are_none(gdn):
    x = logits(5, 700, torch.bfloat16, seed=7)
    u = torch.rand(5)
    want = run(gdn, x, u=u)
    same = run(gdn, x, u=u, top_k=torch.tensor([0, -3, 700, 5000, 0], dtype=torch.int32),
               top_p=torch.tensor([1.0, 2.0, math.nan, 1.0, 1.0]),
               min_p=torch.tensor([0.0, -1.0, math.nan, 0.0, -0.0]), check=False)
    assert torch.equal(want[0], same[0]) and torch.equal(want[1], same[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("stride", [1003, 1009, 1024, 4001])
def test_rows_apart_and_odd(gdn, dtype, stride):
    base = logits(9, stride, dtype, seed=stride)
    x = base[:, :1003]
    run(gdn, x, stride=stride, top_p=torch.full((9,), 0.9))
    run(gdn, x, stride=stride, probs=False)


def test_rows_beyond_32_bits_of_elements(gdn):
    base = torch.full((3, 1 << 30), -1.0, device="cuda", dtype=torch.bfloat16)
    x = base[:, :500]
    x.copy_(logits(3, 500, torch.bfloat16, seed=8))
    run(gdn, x, stride=1 << 30)


def test_same_bits_every_time_and_on_another_stream(gdn):
    x = logits(64, 60000, torch.float32, seed=9)
    args = dict(SETTINGS["all"](64), u=torch.rand(64))
    want = run(gdn, x, **args, check=False)
    stream = torch.cuda.Stream()
    for _ in range(5):
        got = run(gdn, x, **args, check=False, stream=stream)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_and_replayed(gdn):
    x = logits(16, 20000, torch.bfloat16, seed=10)
    u = torch.rand(16, device="cuda")
    p = torch.full((16,), 0.9, device="cuda")
    tokens, probs = torch.empty(16, device="cuda", dtype=torch.int32), torch.empty(16, device="cuda")
    shape = gdn.gdn_sample_shape(16, 20000, gdn.GDN_BF16, 0)

    def call(stream):
        gdn.gdn_sample(shape, x, None, None, p, None, u, tokens, probs, stream)

    call(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(torch.cuda.current_stream())
    for seed in range(3):
        x.copy_(logits(16, 20000, torch.bfloat16, seed=20 + seed))
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        got = tokens.clone()
        want, _ = run(gdn, x, top_p=p.cpu(), u=u.cpu())
        assert torch.equal(got, want)


def test_frequencies_follow_the_weights(gdn):
    # 100000 rows of the same 5 logits: counts within 5 deviations of n p
    n = 100000
    x = torch.tensor([0.0, 1.0, -2.0, 0.5, 2.0], device="cuda").expand(n, 5).contiguous()
    tokens, _ = run(gdn, x, u=torch.rand(n), check=False)
    p = torch.softmax(x[0].double().cpu(), 0)
    count = torch.bincount(tokens.cpu().long(), minlength=5).double()
    assert bool(((count - n * p).abs() <= 5 * (n * p * (1 - p)).sqrt()).all())


@pytest.mark.parametrize("spread", [2.0 ** -10, 2.0 ** -4])
def test_many_logits_of_one_bin(gdn, spread):
    # more values between the bounds of one bin than a block lists, and some rows
    # with fewer; the last kept one takes several rounds to find
    g = torch.Generator("cuda").manual_seed(13)
    torch.manual_seed(13)
    x = torch.randn(7, 60000, generator=g, device="cuda") * spread
    k = torch.tensor([3, 900, 1023, 1025, 5000, 59999, 0], dtype=torch.int32)
    run(gdn, x, top_k=k)
    run(gdn, x, top_k=k, top_p=0.2 + 0.7 * torch.rand(7))
    run(gdn, x, top_p=0.2 + 0.7 * torch.rand(7))
