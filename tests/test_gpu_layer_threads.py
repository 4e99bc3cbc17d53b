"""The attention layer's calls from several host threads at once, each on its
own stream. What a call tells the driver about a kernel (the dynamic shared
memory that it may use) holds for the whole process, so a call of one thread
must leave the other's launches possible, whatever its sizes."""
import threading

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


def in_threads(gdn, calls, n):
    """Each of `calls` n times in a thread and on a stream of its own; the
    errors that they raised."""
    errors = []
    start = threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(n):
                call(stream)
        except gdn.GDNError as e:
            errors.append(str(e))
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    gdn.gdn_check_device_error()
    return errors


def norm_call(gdn, rows, cols, residual):
    """A call whose rows arrive through a ring, and its output."""
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    r = torch.randn(rows, cols, device="cuda").bfloat16() if residual else None
    out = torch.empty_like(x)
    shape = gdn.gdn_norm_shape(rows, cols, gdn.GDN_BF16, 1, 1e-6, 0.0)
    return out, lambda stream: gdn.gdn_rmsnorm_fp8(shape, x, r, None, None, out, None, None,
                                                   stream)


def rope_call(gdn, n, H, H_kv):
    D = 256
    q, k = torch.randn(n, H, D, device="cuda"), torch.randn(n, H_kv, D, device="cuda")
    kc, vc = (torch.zeros(n, 1, H_kv, D, device="cuda").bfloat16() for _ in range(2))
    out = torch.empty(n, H, D, device="cuda").bfloat16()
    args = (q.bfloat16(), k.bfloat16(), k.bfloat16(),
            torch.arange(n, device="cuda", dtype=torch.int32),
            torch.rand(D // 2, device="cuda"), torch.arange(n, device="cuda"), out, kc, vc)
    shape = gdn.gdn_rope_shape(n, H, D, 0, 1, (gdn.c_int * 4)(D // 2), 0, 0, 0, 0)
    cache = gdn.gdn_kv_cache(n, 1, H_kv, D, gdn.GDN_BF16, 0, 0, 0)
    return out, lambda stream: gdn.gdn_rope_append(shape, cache, *args, stream)


@pytest.mark.parametrize("make", [
    # 96 and 64 KB of a block's shared memory
    lambda gdn: [norm_call(gdn, 700, 8192, True), norm_call(gdn, 700, 8192, False)],
    # 61, 122 and 184 KB
    lambda gdn: [rope_call(gdn, 5, 32, 4), rope_call(gdn, 5, 64, 8), rope_call(gdn, 5, 96, 12)],
], ids=["norm", "rope"])
def test_sizes_that_alternate_between_threads(gdn, make):
    made = make(gdn)
    want = []
    for out, call in made:
        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
    assert in_threads(gdn, [call for _, call in made], 4000) == []
    for (out, _), w in zip(made, want):
        assert torch.equal(out, w)
