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
