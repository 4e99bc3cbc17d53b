"""Sizes and layouts at the ends of what the attention layer's calls accept."""
import pytest
import torch

from test_gpu_paged_attention import Case

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


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_strides_that_no_second_element_uses(gdn, D, page):
    # of a level with one element (one kv head, one page) any stride is legal
    c = Case(gdn, [page - 3], 8, 13, 1, D, page, torch.bfloat16, seed=page + D)
    n = c.k.shape[0]
    for head_stride in (8, D, 1 << 20):
        c.cache = gdn.gdn_kv_cache(n, page, 1, D, gdn.GDN_BF16, page * D, D, head_stride)
        c.check(c.run())
    own = int(c.table[0, 0])
    c.k, c.v = c.k[own:own + 1].clone(), c.v[own:own + 1].clone()
    c.table[0, 0] = 0
    for page_stride in (8, page * D, 1 << 40):
        c.cache = gdn.gdn_kv_cache(1, page, 1, D, gdn.GDN_BF16, page_stride, D, 8)
        c.check(c.run())
