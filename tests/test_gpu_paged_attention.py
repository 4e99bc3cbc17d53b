"""gdn_paged_attention against softmax attention in 64 bits.

Tolerance of an output element, with A = sum_j p_j |v_j| / sum_j p_j. A score
is a sum of D products in fp32; its roundings add up like a random walk, 16 of
2^-24 for D = 256, on sums of up to about 20: 2e-5 relative on p, once in the
sum over v and once in the sum of p: 5e-5 A. In bf16 each p is rounded (2^-8)
before its product with v, and the output is (2^-8)."""
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


class Case:
    """A cache with shuffled pages; everything that no key owns is NaN."""

    def __init__(self, gdn, lens, T, H, H_kv, D, page, dtype, layout="dense", seed=0, extra=2,
                 kv_map=1, scale=0.0):
        g = torch.Generator("cuda")
        g.manual_seed(seed)
        self.gdn, self.T, self.H, self.H_kv, self.D, self.page = gdn, T, H, H_kv, D, page
        self.lens_host, self.kv_map = list(lens), kv_map
        self.scale = scale or D ** -0.5
        n = len(lens)
        need = [-(-x // page) for x in lens]
        self.max_pages = max(need) + extra
        pages = sum(need) + 3
        nan = float("nan")
        code = gdn.dtype_code(dtype)
        if layout == "dense":
            k = torch.full((pages, page, H_kv, D), nan, device="cuda", dtype=dtype)
            v = k.clone()
            self.cache = gdn.gdn_kv_cache(pages, page, H_kv, D, code, 0, 0, 0)
        elif layout == "heads_first":
            k = torch.full((pages, H_kv, page, D), nan, device="cuda", dtype=dtype)
            v = k.clone().transpose(1, 2)
            k = k.transpose(1, 2)
            self.cache = gdn.gdn_kv_cache(pages, page, H_kv, D, code, H_kv * page * D, D, page * D)
        else:
            kv = torch.full((pages, 2, page, H_kv, D), nan, device="cuda", dtype=dtype)
            k, v = kv[:, 0], kv[:, 1]
            self.cache = gdn.gdn_kv_cache(pages, page, H_kv, D, code, 2 * page * H_kv * D,
                                          H_kv * D, D)
        order = torch.randperm(pages, generator=g, device="cuda")
        table = torch.full((n, self.max_pages), -1, device="cuda", dtype=torch.int32)
        at = 0
        self.keys = []
        for s, x in enumerate(lens):
            ids = order[at:at + need[s]]
            at += need[s]
            table[s, :need[s]] = ids.to(torch.int32)
            j = torch.arange(x, device="cuda")
            ks = torch.randn(x, H_kv, D, generator=g, device="cuda").to(dtype)
            vs = torch.randn(x, H_kv, D, generator=g, device="cuda").to(dtype)
            k[ids[j // page], j % page] = ks
            v[ids[j // page], j % page] = vs
            self.keys.append((ks, vs))
        self.k, self.v, self.table = k, v, table
        self.lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
        self.q = (2 * torch.randn(n * T, H, D, generator=g, device="cuda")).to(dtype)
        self.shape = gdn.gdn_attn_shape(n, T, H, self.max_pages, scale, kv_map)
        self.bytes = gdn.gdn_paged_attention_workspace_size(self.shape, self.cache)
        assert 0 < self.bytes <= 64 << 20

    def run(self, stream=None, check=True):
        out = torch.full_like(self.q, float("nan"))
        ws = torch.full((self.bytes,), 0xff, device="cuda", dtype=torch.uint8)
        torch.cuda.synchronize()
        self.gdn.gdn_paged_attention(self.shape, self.cache, self.q, self.k, self.v, self.table,
                                     self.lens, out, ws, self.bytes, stream)
        torch.cuda.synchronize()
        if check:
            self.gdn.gdn_check_device_error()
        return out

    def want(self, s, t):
        """(out, A) of row t of sequence s in 64 bits, [H, D]."""
        n = self.lens_host[s] - self.T + t + 1
        H, G = self.H, self.H // self.H_kv
        if n <= 0:
            z = torch.zeros(H, self.D, dtype=torch.float64, device="cuda")
            return z, z
        h = torch.arange(H, device="cuda")
        kvh = h // G if self.kv_map else h % self.H_kv
        k = self.keys[s][0][:n].double()[:, kvh]
        v = self.keys[s][1][:n].double()[:, kvh]
        q = self.q[s * self.T + t].double()
        p = torch.softmax(torch.einsum("hd,khd->hk", q, k) * self.scale, -1)
        return torch.einsum("hk,khd->hd", p, v), torch.einsum("hk,khd->hd", p, v.abs())

    def check(self, out):
        for s in range(len(self.lens_host)):
            for t in range(self.T):
                w, a = self.want(s, t)
                tol = 5e-5 * a
                if out.dtype == torch.bfloat16:
                    tol = tol + 2.0 ** -8 * (a + w.abs())
                got = out[s * self.T + t].double()
                assert bool(((got - w).abs() <= tol).all()), (s, t, self.lens_host[s])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,H_kv,T", [(1, 1, 1), (16, 2, 1), (6, 2, 3), (16, 2, 4), (16, 2, 8),
                                      (32, 2, 5), (40, 1, 2)])
def test_heads_and_tokens(gdn, dtype, D, H, H_kv, T):
    lens = [1, 15, 16, 63, 64, 65, 200, 0, 129]
    c = Case(gdn, lens, T, H, H_kv, D, 16, dtype, seed=H + T + D)
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 256])
@pytest.mark.parametrize("layout", ["dense", "heads_first", "k_and_v_in_one"])
def test_pages_and_layouts(gdn, dtype, page, layout):
    c = Case(gdn, [3, 700, 256, 0, 100, 1], 2, 8, 2, 128, page, dtype, layout=layout, seed=page)
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,T", [(8, 1), (16, 8)])
@pytest.mark.parametrize("lens", [
    [40000], [1, 30000, 2], [5000, 1, 1, 9000, 3], [300] * 40, [0] * 7 + [5000] + [0] * 7])
def test_lengths_cut_between_blocks(gdn, dtype, H, T, lens):
    c = Case(gdn, lens, T, H, 2, 128, 32, dtype, seed=len(lens))
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 24, 32, 64, 128, 192])
@pytest.mark.parametrize("layout", ["dense", "heads_first", "k_and_v_in_one"])
def test_many_rows_pages_and_layouts(gdn, D, page, layout):
    # 24, 56 and 104 rows for each kv head
    for H, H_kv, T in ((12, 2, 4), (14, 2, 8), (13, 1, 8)):
        c = Case(gdn, [3, 700, 64, 256, 0, 100, 1, 1025], T, H, H_kv, D, page, torch.bfloat16,
                 layout=layout, seed=page + T)
        c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [4, 8, 16])
def test_many_rows_and_many_tiles_in_a_block(gdn, D, T):
    # some twenty tiles of 64 keys for each block, most items ending inside one
    lens = [1000 + 7 * i for i in range(100)]
    c = Case(gdn, lens, T, 16, 2, D, 16, torch.bfloat16, seed=D + T)
    c.check(c.run())


def test_many_rows_growing_scores(gdn):
    # keys that grow along the sequence: every tile raises the maximum, far
    # beyond what the sums' reference leaves untouched
    c = Case(gdn, [1500, 640, 130], 4, 16, 2, 128, 16, torch.bfloat16, seed=11, scale=0.05)
    for s, (k, v) in enumerate(c.keys):
        n = k.shape[0]
        k *= torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None].bfloat16()
        j = torch.arange(n, device="cuda")
        c.k[c.table[s, j // 16].long(), j % 16] = k
    out = c.run()
    for s in range(3):
        for t in range(4):
            w, a = c.want(s, t)
            # scores of up to six times the other tests' size, and their rounding
            tol = 6 * 5e-5 * a + 2.0 ** -8 * (a + w.abs())
            assert bool(((out[s * 4 + t].double() - w).abs() <= tol).all())


def test_many_short_sequences(gdn):
    g = torch.Generator()
    g.manual_seed(3)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    c = Case(gdn, lens, 1, 4, 2, 64, 8, torch.bfloat16, seed=9)
    c.check(c.run())


def test_no_sequence_has_a_key(gdn):
    c = Case(gdn, [0, 0, 0], 2, 8, 2, 128, 16, torch.bfloat16)
    assert bool((c.run() == 0).all())
    c = Case(gdn, [0], 1, 2, 2, 64, 16, torch.float32, extra=0)   # a page table without columns
    assert bool((c.run() == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_scale_head_map_and_large_scores(gdn, dtype):
    c = Case(gdn, [77, 300], 3, 12, 4, 128, 16, dtype, kv_map=0, scale=0.02, seed=1)
    c.check(c.run())
    # scores of a hundred and more: one key holds nearly all the weight
    c = Case(gdn, [500, 70], 1, 8, 2, 64, 16, dtype, seed=2)
    c.q *= 64
    out = c.run()
    for s in range(2):
        w, a = c.want(s, 0)
        # a score's rounding grows with it: 64 times that of the other tests
        tol = 64 * 5e-5 * a + (2.0 ** -8 * (a + w.abs()) if dtype == torch.bfloat16 else 0)
        assert bool(((out[s].double() - w).abs() <= tol).all())


def test_the_same_bits_every_time_and_on_another_stream(gdn):
    c = Case(gdn, [3000, 17, 9000, 1, 0, 4000], 4, 16, 2, 128, 16, torch.bfloat16, seed=5)
    a = c.run()
    side = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(c.run(side), a)


def test_in_a_graph_with_lengths_that_change(gdn):
    c = Case(gdn, [1000, 2000, 300], 1, 8, 2, 64, 16, torch.bfloat16, seed=6)
    a = c.run()
    out, ws = torch.empty_like(c.q), torch.empty(c.bytes, device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_attention(c.shape, c.cache, c.q, c.k, c.v, c.table, c.lens, out, ws, c.bytes,
                                torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    c.lens_host = [10, 1999, 1]
    c.lens.copy_(torch.tensor(c.lens_host, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_bad_pages_and_lengths_are_reported(gdn):
    for bad in (-1, 1 << 30):
        c = Case(gdn, [100, 200, 50], 1, 8, 2, 128, 16, torch.bfloat16, seed=7)
        c.table[1, 3] = bad
        out = c.run(check=False)
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_check_device_error()
        assert e.value.status == gdn.GDN_ERR_DEVICE_ARG and "page table" in str(e.value)
        for s in (0, 2):     # the others are whole
            w, a = c.want(s, 0)
            assert bool(((out[s].double() - w).abs() <= 2.0 ** -7 * a + 5e-5 * a).all())
    c = Case(gdn, [100, 200, 50], 1, 8, 2, 128, 16, torch.bfloat16, seed=8, extra=0)
    c.lens[1] = 209          # one more than its 13 pages hold
    c.run(check=False)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_check_device_error()
    c.lens[1] = -5           # as 0
    assert bool((c.run()[1] == 0).all())


def test_a_cache_beyond_32_bits_of_elements(gdn):
    pages, page, D = 40, 16, 64
    stride = 1 << 26
    store = torch.zeros(pages * stride, device="cuda", dtype=torch.bfloat16)
    view = (pages, page, 1, D)
    k = store.as_strided(view, (stride, D, D, 1))
    v = store.as_strided(view, (stride, D, D, 1), 1 << 20)
    ids = [39, 3, 38]
    c = Case(gdn, [40], 1, 8, 1, D, page, torch.bfloat16, extra=0, seed=4)
    c.cache = gdn.gdn_kv_cache(pages, page, 1, D, gdn.GDN_BF16, stride, D, D)
    for i, p in enumerate(ids):
        n = min(16, 40 - 16 * i)
        k[p, :n] = c.keys[0][0][16 * i:16 * i + n]
        v[p, :n] = c.keys[0][1][16 * i:16 * i + n]
    c.k, c.v = k, v
    c.table.copy_(torch.tensor([ids], dtype=torch.int32))
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,H_kv,T", [(8, 1, 1), (16, 2, 2), (16, 2, 8)])
@pytest.mark.parametrize("lens", [[20000], [15000, 0, 1, 6001, 130]])
def test_items_of_many_blocks(gdn, dtype, D, H, H_kv, T, lens):
    c = Case(gdn, lens, T, H, H_kv, D, 16, dtype, seed=H + T + D)
    c.check(c.run())
