"""gdn_sample where a limit of its own meets a special value: the definition in 64
bits and the tolerances of test_gpu_sample.py."""
import math

import pytest
import torch

from test_gpu_sample import TYPES, gdn, logits, run  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_with_largest_zero(dtype):
    x = logits(8, 1501, dtype, seed=31)
    x -= x.float().amax(1, keepdim=True).to(dtype)   # as softmax code shifts them
    x[1] = 0.0
    x[2] = -0.0
    x[3, ::2], x[3, 1::2] = 0.0, -0.0
    x[4, 5] = x[4, 900] = math.inf
    x[5, 7] = math.inf
    x[6] = -1.0
    x[6, 3::500] = 0.0
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("more", [
    {}, dict(top_k=5), dict(top_p=0.7), dict(top_k=2000, top_p=0.99), dict(temperature=0.7)])
@pytest.mark.parametrize("min_p", [1.0, 1 - 2.0 ** -24, 0.5])
def test_min_p_with_the_largest_at_zero(gdn, dtype, more, min_p):
    x = rows_with_largest_zero(dtype)
    torch.manual_seed(32)
    args = {key: torch.full((8,), v, dtype=torch.int32 if key == "top_k" else torch.float32)
            for key, v in more.items()}
    run(gdn, x, min_p=torch.full((8,), min_p), u=torch.rand(8), **args)


NEIGHBOURS = [(20.0, 3.115e-8), (1e4, 1.6e-5), (1e8, 0.1307), (-20.0, 3.115e-8), (3.0, 3.9e-9),
              (1.5, 1.9e-9)]


@pytest.mark.parametrize("top,temperature", NEIGHBOURS)
@pytest.mark.parametrize("more", [
    {}, dict(top_k=2), dict(top_k=40), dict(top_p=0.9), dict(top_k=3, top_p=0.99), dict(min_p=1e-9)])
def test_temperatures_of_a_rounding(gdn, top, temperature, more):
    # the logit before the largest is some 50 to 90 octaves of weight below it: no
    # weight, though the bound of 45 octaves lies nearer to it than to the largest
    x = torch.full((6, 777), -1e30, device="cuda")
    value = torch.tensor(top)
    for i in range(60):
        x[:, 13 * i] = value
        value = torch.nextafter(value, torch.tensor(-math.inf))
    x[1] = x[1].flip(0)
    x[2, ::2] = top
    x[3, 5:] = -math.inf
    args = {key: torch.full((6,), v, dtype=torch.int32 if key == "top_k" else torch.float32)
            for key, v in more.items()}
    for scale in (0.7, 0.9, 1.0, 1.1, 1.5, 40.0):
        run(gdn, x, temperature=torch.full((6,), temperature * scale), u=torch.linspace(0, 0.99, 6),
            **args)


@pytest.mark.parametrize("more", [{}, dict(top_k=4), dict(top_p=0.6)])
def test_the_lowest_numbers_beside_minus_infinity(gdn, more):
    low = torch.finfo(torch.float32).min
    x = torch.full((4, 301), -math.inf, device="cuda")
    x[0, 7:20] = low
    x[1, 299:] = low
    x[2] = low
    x[3, ::3] = low * (1 - 2.0 ** -10)
    x[3, 1::3] = low
    args = {key: torch.full((4,), v, dtype=torch.int32 if key == "top_k" else torch.float32)
            for key, v in more.items()}
    for t in (1.0, 1e30, 3e33, math.inf):
        # the largest temperature counts as 3e33
        got = run(gdn, x, temperature=torch.full((4,), t), u=torch.tensor([0.1, 0.5, 0.9, 0.3]),
                  check=t <= 3e33, **args)
        assert bool((x[torch.arange(4), got[0].long()] > -math.inf).all())


def test_min_p_with_temperatures_that_count_as_the_least(gdn):
    # 1e-35 counts as 1e-30 for the weights and for min_p's bound alike
    x = torch.tensor([[0.0, -1e-31, -5e-31, -2e-30, -1.0],
                      [-1e-31, -3e-31, 0.0, -8e-31, -1e-30]], device="cuda").repeat(6, 1)
    m = torch.full((12,), 0.5)
    u = torch.linspace(0.0, 0.99, 12)
    want = run(gdn, x, temperature=torch.full((12,), 1e-30), min_p=m, u=u)
    got = run(gdn, x, temperature=torch.full((12,), 1e-35), min_p=m, u=u, check=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
