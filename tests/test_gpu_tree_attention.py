"""gdn_tree_attention against masked softmax attention in 64 bits, with the
tolerance of gdn_paged_attention (tests/test_gpu_paged_attention.py): the same
products and sums, other masks."""
import numpy as np
import pytest
import torch

from test_gpu_paged_attention import TYPES, Case, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def random_words(kind, n, T, seed):
    """[n, T] words: trees, or anything."""
    rng = np.random.default_rng(seed)
    w = np.zeros((n, T), np.uint64)
    if kind == "any":
        w = rng.integers(0, 2 ** 63, (n, T)).astype(np.uint64) * np.uint64(2) + rng.integers(
            0, 2, (n, T)).astype(np.uint64)
        w[rng.random((n, T)) < 0.1] = 0
        return w
    for t in range(T):
        w[:, t] = np.uint64(1) << np.uint64(t)
        if t and kind != "star":
            back = 1 if kind == "line" else 1 + rng.integers(0, min(t, 5), n)
            parent = t - back
            up = w[np.arange(n), parent]
            if kind == "bush":
                up = np.where(rng.random(n) < 0.1, np.uint64(0), up)
            w[:, t] |= up
    return w


class TreeCase(Case):
    def __init__(self, gdn, lens, T, *args, words="bush", nodes=None, seed=0, **kw):
        super().__init__(gdn, lens, T, *args, seed=seed, **kw)
        w = random_words(words, len(lens), T, seed) if isinstance(words, str) else words
        self.words = w
        self.tree = torch.from_numpy(w.view(np.int64)).cuda()
        self.nodes_host = [T] * len(lens) if nodes is None else list(nodes)
        self.nodes = None if nodes is None else torch.tensor(nodes, device="cuda", dtype=torch.int32)
        self.bytes = gdn.gdn_tree_attention_workspace_size(self.shape, self.cache)
        assert 0 < self.bytes <= 64 << 20

    def run(self, stream=None, check=True):
        out = torch.full_like(self.q, float("nan"))
        ws = torch.full((self.bytes,), 0xff, device="cuda", dtype=torch.uint8)
        torch.cuda.synchronize()
        self.gdn.gdn_tree_attention(self.shape, self.cache, self.q, self.k, self.v, self.table,
                                    self.lens, self.nodes, self.tree, out, ws, self.bytes, stream)
        torch.cuda.synchronize()
        if check:
            self.gdn.gdn_check_device_error()
        return out

    def check(self, out):
        T, H = self.T, self.H
        G = H // self.H_kv
        h = torch.arange(H, device="cuda")
        kvh = h // G if self.kv_map else h % self.H_kv
        for s, n in enumerate(self.lens_host):
            m = self.nodes_host[s]
            seen = torch.zeros(T, n, dtype=torch.bool)
            for t in range(m):
                seen[t, :max(n - m, 0)] = True
                for j in range(m):
                    if n - m + j >= 0:
                        seen[t, n - m + j] = bool(int(self.words[s, t]) >> j & 1)
            seen = seen.cuda()
            k, v = (x.double()[:, kvh] for x in self.keys[s])
            q = self.q[s * T:(s + 1) * T].double()
            x = torch.einsum("thd,khd->thk", q, k) * self.scale
            x = x.masked_fill(~seen[:, None], -torch.inf)
            some = seen.any(1)
            p = torch.zeros_like(x)
            p[some] = torch.softmax(x[some], -1)
            want = torch.einsum("thk,khd->thd", p, v)
            a = torch.einsum("thk,khd->thd", p, v.abs())
            tol = 5e-5 * a
            if out.dtype == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (a + want.abs())
            got = out[s * T:(s + 1) * T].double()
            assert bool(((got - want).abs() <= tol).all()), (s, n, m)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,H_kv,T", [(1, 1, 1), (16, 2, 2), (6, 2, 7), (16, 2, 16), (8, 8, 33),
                                      (16, 2, 64), (5, 1, 64)])
@pytest.mark.parametrize("words", ["bush", "any"])
def test_heads_and_nodes(gdn, dtype, D, H, H_kv, T, words):
    lens = [T, T + 1, 64, T + 63, 130, 200, 127, T + 65, 1025]
    lens = [max(x, T) for x in lens]
    c = TreeCase(gdn, lens, T, H, H_kv, D, 16, dtype, words=words, seed=H + T + D)
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 256])
@pytest.mark.parametrize("layout", ["dense", "heads_first", "k_and_v_in_one"])
@pytest.mark.parametrize("T", [5, 24])
def test_pages_and_layouts(gdn, dtype, page, layout, T):
    c = TreeCase(gdn, [T, 700, 256, T + 2, 100, 65], T, 8, 2, 128, page, dtype, layout=layout,
                 seed=page)
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,H_kv", [(8, 4, 2), (20, 16, 2), (64, 8, 1)])
def test_fewer_nodes_and_short_sequences(gdn, dtype, D, T, H, H_kv):
    # padding, no nodes at all, an empty sequence, fewer tokens than nodes
    nodes = [T, T // 2, 0, 1, 3, T, 2, 0]
    lens = [300, 129, 64, 1, 2, max(T - 3, 1), 2, 0]
    c = TreeCase(gdn, lens, T, H, H_kv, D, 16, dtype, words="any", nodes=nodes, seed=T)
    for s, m in enumerate(nodes):
        c.q[s * T + m:(s + 1) * T] = float("nan")      # not used
        c.words[s, m:] = np.uint64(12345)
    c.tree.copy_(torch.from_numpy(c.words.view(np.int64)))
    out = c.run()
    c.q.nan_to_num_(0.0)
    c.check(out)
    assert not bool(out.isnan().any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,T", [(8, 3), (16, 20), (16, 64)])
@pytest.mark.parametrize("lens", [
    [40000], [64, 30000, 65], [5000, 64, 70, 9000, 100], [300] * 40, [64] * 7 + [5000] + [64] * 7])
def test_lengths_cut_between_blocks(gdn, dtype, H, T, lens):
    nodes = [T if i % 3 else max(T - 1, 1) for i in range(len(lens))]
    c = TreeCase(gdn, lens, T, H, 2, 128, 32, dtype, seed=len(lens), nodes=nodes)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,T", [(2, 50), (4, 64), (3, 64)])   # 100, 256 and 192 rows
@pytest.mark.parametrize("lens", [[3000] * 60, [20000, 64, 9000, 127, 128, 129, 15000]])
def test_many_rows_over_many_tiles(gdn, D, H, T, lens):
    # several items in a block, of many tiles, of one and of two
    nodes = [T - i % 4 for i in range(len(lens))]
    c = TreeCase(gdn, lens, T, H, 1, D, 16, torch.bfloat16, seed=len(lens), nodes=nodes)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 24, 32, 64, 128, 192])
@pytest.mark.parametrize("layout", ["dense", "heads_first", "k_and_v_in_one"])
def test_many_rows_pages_and_layouts(gdn, D, page, layout):
    # 24, 60, 104, 260 and 320 rows for each kv head
    for H, H_kv, T in ((12, 2, 4), (10, 2, 12), (8, 1, 13), (5, 1, 52), (20, 4, 64)):
        c = TreeCase(gdn, [T + 3, 700, 64, 256, 100, T, 1025], T, H, H_kv, D, page, torch.bfloat16,
                     layout=layout, seed=page + T)
        c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_line_is_gdn_paged_attention(gdn, dtype, T, D):
    lens = [T, 300, 129, 2000]
    c = TreeCase(gdn, lens, T, 16, 2, D, 16, dtype, words="line", seed=T)
    a, b = c.run(), Case.run(c)
    # the same numbers in the same order
    assert torch.equal(a, b)


def test_tiled_heads_and_scale(gdn):
    c = TreeCase(gdn, [100, 64, 333], 12, 12, 3, 128, 16, torch.bfloat16, kv_map=0, scale=0.03)
    c.check(c.run())


def test_words_of_nothing_see_the_prefix_alone(gdn):
    T = 6
    words = np.zeros((3, T), np.uint64)
    c = TreeCase(gdn, [T, T + 1, 90], T, 4, 2, 64, 16, torch.float32, words=words)
    out = c.run()
    c.check(out)
    assert not bool(out[:T].any())     # no prefix, no nodes: 0


def test_numbers_of_nodes_out_of_range(gdn):
    c = TreeCase(gdn, [100, 64, 70], 8, 4, 2, 128, 16, torch.bfloat16, nodes=[8, 9, -1])
    with pytest.raises(gdn.GDNError) as e:
        c.run()
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG and "tree" in str(e.value)


def test_page_table_entries_out_of_range(gdn):
    c = TreeCase(gdn, [100, 64, 70], 8, 4, 2, 128, 16, torch.bfloat16)
    want = c.run()
    c.table[1, 2] = 10 ** 6
    with pytest.raises(gdn.GDNError) as e:
        c.run()
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG
    c.table[1, 2] = -5
    out = c.run(check=False)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_check_device_error()
    assert torch.equal(out[:8], want[:8]) and torch.equal(out[16:], want[16:])


@pytest.mark.parametrize("T,H", [(5, 4), (32, 16)])
def test_same_bits_every_time_and_on_another_stream(gdn, T, H):
    c = TreeCase(gdn, [5000, 64, 900, 12000], T, H, 2, 128, 16, torch.bfloat16)
    want = c.run()
    stream = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(c.run(stream), want)


def test_captured_and_replayed(gdn):
    c = TreeCase(gdn, [500, 64, 900], 16, 16, 2, 128, 16, torch.bfloat16)
    out = c.run()
    ws = torch.empty(c.bytes, device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_tree_attention(c.shape, c.cache, c.q, c.k, c.v, c.table, c.lens, c.nodes, c.tree, out,
                               ws, c.bytes, torch.cuda.current_stream())
    for seed in range(3):
        c.words = random_words("any", 3, 16, seed)
        c.tree.copy_(torch.from_numpy(c.words.view(np.int64)))
        c.q.normal_()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H", [(64, 40), (33, 96), (64, 640)])
def test_more_blocks_of_rows_than_fit(gdn, D, T, H):
    # one kv head: up to 40960 rows, more blocks of them than the GPU runs at once
    c = TreeCase(gdn, [T + 70, 200, T], T, H, 1, D, 16, torch.bfloat16, seed=H,
                 nodes=[T, T - 1, 1])
    c.check(c.run())


@pytest.mark.parametrize("D,H", [(64, 4), (128, 4), (256, 3)])
@pytest.mark.parametrize("scale", [-0.07, 1e-4])
def test_scales_of_many_rows(gdn, D, H, scale):
    c = TreeCase(gdn, [64, 700, 321, 130], 64, H, 1, D, 16, torch.bfloat16, words="any",
                 nodes=[64, 50, 64, 1], scale=scale, seed=D)
    c.check(c.run())
