"""gdn_qknorm_rope_append where a unit has several tokens, whose angles one lane of a
warp makes and others read: the definition's tolerances (test_gpu_qknorm_rope.py), and
the same bits every time."""
import pytest
import torch

from test_gpu_qknorm_rope import TYPES, gdn, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,H_kv,D,rot,sec,neighbours", [
    (1, 1, 64, 32, (16,), False), (2, 1, 64, 64, (20, 12), True), (1, 1, 64, 50, (25,), False),
    (1, 1, 128, 64, (32,), False)])
def test_angles_of_many_units(gdn, dtype, H, H_kv, D, rot, sec, neighbours):
    n = 30011
    want = None
    for _ in range(4):
        torch.manual_seed(18)   # what the cache holds before
        got = run(gdn, n, H, H_kv, D, rot, sec, False, neighbours, 16, dtype, max_pos=1 << 20,
                  seed=17)
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
