"""Sizes and layouts at the ends of what the attention layer's calls accept."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def test_norm_of_the_most_rows(gdn):
    # 2^31 - 1 rows of 8 columns (34 GB); h = x + x in place
    rows = (1 << 31) - 1
    x = torch.ones(rows, 8, device="cuda", dtype=torch.bfloat16)
    shape = gdn.gdn_norm_shape(rows, 8, gdn.GDN_BF16, 0, 0.0, 0.0)
    gdn.gdn_rmsnorm_fp8(shape, x, x, None, None, x, None, None)
    torch.cuda.synchronize()
    gdn.gdn_check_device_error()
    low, high = float(x.min()), float(x.max())
    del x
    torch.cuda.empty_cache()
    assert low == high == 2
