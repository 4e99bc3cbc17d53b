"""What the binding and the C entry points of the attention layer accept and
refuse beside the cases of test_layer_host.py (no GPU needed)."""
import pytest
import torch

from test_layer_host import FAKE, STEP, kv, norm, refused, rope


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    return mod


class Address(int):
    """An int of another class, as an enum's member or a wrapped handle is."""


def test_ints_of_another_class_are_addresses_and_streams(gdn):
    assert gdn._stream(Address(7)) == 7 and type(gdn._stream(Address(7))) is int
    shape = gdn.gdn_norm_shape(0, 256, gdn.GDN_BF16, 1, 1e-6, 0.0)
    gdn.gdn_rmsnorm_fp8(shape, *[Address(FAKE)] * 7, Address(0))
    # the refusal shows that the call itself was reached with these addresses
    st, msg = refused(gdn, lambda: rope(gdn, q=Address(FAKE), k_cache=Address(FAKE + 8 * STEP)))
    assert st == gdn.GDN_ERR_INVALID_ARG and "are the same" in msg


def test_rows_of_another_rank_are_refused(gdn):
    for x in (torch.zeros(5, 4 * 128), torch.zeros(5 * 4 * 128), torch.zeros(1, 5, 4, 128)):
        with pytest.raises(ValueError, match="rows must be packed"):
            rope(gdn, q=x)


def strided(gdn, n_pages, page, H_kv, D, strides):
    return kv(gdn, n_pages=n_pages, page_size=page, H_kv=H_kv, D=D, dtype=gdn.GDN_F32,
              page_stride=strides[0], token_stride=strides[1], head_stride=strides[2])


def test_strided_caches_that_match_their_struct(gdn):
    n, p, H, D = 10, 16, 2, 64
    both = torch.zeros(n, 2, p, H, D)
    heads = torch.zeros(n, H, p, D)
    slots = torch.zeros(n * p, 2, H, D)
    packed = torch.zeros(n, p, H, D)
    wide, first = (2 * p * H * D, H * D, D), (H * p * D, D, p * D)
    for x, size, strides in (
            (both[:, 0], (n, p, H), wide), (both[:, 1], (n, p, H), wide),
            (both, (n, p, H), wide), (both[3:, 0], (n - 3, p, H), wide),
            (both[:, 0, :, 1:], (n, p, 1), wide),
            (heads.transpose(1, 2), (n, p, H), first), (heads, (n, p, H), first),
            (heads[:, :, ::2].transpose(1, 2), (n, p // 2, H), (H * p * D, 2 * D, p * D)),
            (slots[:, 1], (n, p, H), (2 * p * H * D, 2 * H * D, D)),
            (packed, (n, p, H), (p * H * D, H * D, D)),
            (packed.view(-1), (n, p, H), (p * H * D, H * D, D)),
            (torch.zeros(n, p, 2 * H * D)[..., :H * D], (n, p, H), (2 * p * H * D, 2 * H * D, D))):
        assert gdn._cache_addr(x, strided(gdn, *size, D, strides)) == x.data_ptr()


def test_strided_caches_that_do_not_match_are_refused(gdn):
    n, p, H, D = 10, 16, 2, 64
    both = torch.zeros(n, 2, p, H, D)
    heads = torch.zeros(n, H, p, D).transpose(1, 2)
    wide = (2 * p * H * D, H * D, D)
    for x, pages, strides in (
            (both[:, 0], n, (p * H * D, H * D, D)),        # as if k stood alone
            (both[:, 0], n, (2 * p * H * D, D, p * D)),    # as if heads came first
            (heads, n, (H * p * D, H * D, D)),             # as if tokens came first
            (heads, n, (H * p * D, D, 2 * p * D)),
            (both, n + 1, wide),                           # a page more than there are
            (torch.zeros(n, p, H, D), n, wide)):           # beyond the tensor's memory
        with pytest.raises(ValueError, match="the cache's strides"):
            gdn._cache_addr(x, strided(gdn, pages, p, H, D, strides))


def test_rows_of_the_two_caches_stay_apart(gdn):
    import random
    rng = random.Random(5)
    seen = set()
    for _ in range(400):
        n, p, H, D = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 3), 64
        # levels in any order, each over all of the one below, with gaps at times
        counts, strides, span = {"p": n, "t": p, "h": H}, {}, D
        for level in rng.sample("pth", 3):
            strides[level] = span + rng.choice([0, 0, 4, 64, 128, 200])
            span += (counts[level] - 1) * strides[level]
        s = [strides[x] for x in "pth"]
        delta = 4 * rng.randint(1, span // 4 + 2) * rng.choice([1, -1])
        k = FAKE + 7 * STEP
        rows = {i * s[0] + j * s[1] + h * s[2] for i in range(n) for j in range(p) for h in range(H)}
        meet = any(abs(a + delta - b) < D for a in rows for b in rows)
        # q_out lies on the k cache: what is refused next where the caches are apart
        st, msg = refused(gdn, lambda: rope(
            gdn, dict(rot_dim=64, section=(16, 8, 8)),
            dict(n_pages=n, page_size=p, H_kv=H, D=D, dtype=gdn.GDN_F32, page_stride=s[0],
                 token_stride=s[1], head_stride=s[2]),
            k_cache=k, v_cache=k + 4 * delta, q_out=k))
        word = "rows of k_cache and v_cache overlap" if meet else "q_out overlaps k_cache"
        assert st == gdn.GDN_ERR_INVALID_ARG and word in msg, (s, (n, p, H), delta)
        seen.add((meet, abs(delta) < span))
    assert {(True, True), (False, True), (False, False)} <= seen
    # one dense layout inside the other
    for off in (16, 256, 4096, 40960 * 2 - 16):
        st, msg = refused(gdn, lambda: rope(gdn, k_cache=k, v_cache=k + off))
        assert "rows of k_cache and v_cache overlap" in msg


def test_norm_refuses_columns_that_its_indexes_cannot_step_over(gdn):
    for cols in (2 ** 31 - 1, 2 ** 31 - 1023):
        st, msg = refused(gdn, lambda: norm(gdn, dict(rows=1, cols=cols)))
        assert st == gdn.GDN_ERR_UNSUPPORTED and "above 2^31 - 1024" in msg
