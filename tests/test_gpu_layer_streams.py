"""The attention layer's calls under programmatic dependent launch: chains of
dependent calls on one stream, calls in flight on two streams at once, and what
include/gdn.h promises of every call: no allocation and no synchronisation."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


class Layer:
    """The four calls as one layer of n tokens: T of each of n / T sequences,
    which have `before` keys each. Every call reads what the one before wrote."""

    def __init__(self, gdn, n, T, hidden=1024, H=8, H_kv=2, D=128, before=300, seed=0):
        g = torch.Generator("cuda")
        g.manual_seed(seed)
        self.gdn, self.n, self.hidden, self.H, self.D = gdn, n, hidden, H, D
        self.hd, self.wide, page = H * D, (H + 2 * H_kv) * D, 16

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        def buf(*shape, dtype=torch.bfloat16):
            return torch.zeros(*shape, device="cuda", dtype=dtype)

        self.x0, self.h0 = randn(n, hidden).bfloat16(), randn(n, hidden).bfloat16()
        self.x, self.h = self.x0.clone(), self.h0.clone()
        self.norm_w = randn(hidden).bfloat16()
        self.w1, self.w2 = randn(self.wide, hidden).to(E4M3), randn(hidden, self.hd).to(E4M3)
        self.s1 = torch.full((self.wide // 128, hidden // 128), hidden ** -0.5, device="cuda")
        self.s2 = torch.full((hidden // 128, self.hd // 128), self.hd ** -0.5, device="cuda")
        self.x8, self.xs = buf(n, hidden, dtype=E4M3), buf(n, hidden // 128, dtype=torch.float32)
        self.qkv, self.q, self.o = buf(n, self.wide), buf(n, H, D), buf(n, H, D)
        self.o8, self.os = buf(n, self.hd, dtype=E4M3), buf(n, self.hd // 128, dtype=torch.float32)
        seqs, per = n // T, -(-(before + T) // page)
        self.k0 = randn(seqs * per, page, H_kv, D).bfloat16()
        self.k, self.v = self.k0.clone(), self.k0.flip(0)
        self.v0 = self.v.clone()
        self.table = torch.arange(seqs * per, device="cuda", dtype=torch.int32).view(seqs, per)
        self.lens = torch.full((seqs,), before + T, device="cuda", dtype=torch.int32)
        t = torch.arange(n, device="cuda")
        self.pos = (before + t % T).to(torch.int32)
        self.slots = t // T * per * page + before + t % T
        self.inv = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        self.cache = gdn.gdn_kv_cache(seqs * per, page, H_kv, D, gdn.GDN_BF16, 0, 0, 0)
        self.attn = gdn.gdn_attn_shape(seqs, T, H, per, 0.0, gdn.GDN_QK_GROUPED)
        self.rope = gdn.gdn_rope_shape(n, H, D, 0, 1, (gdn.c_int * 4)(D // 2), 0, self.wide,
                                       self.wide, self.wide)
        nbytes = gdn.gdn_paged_attention_workspace_size(self.attn, self.cache)
        self.ws = buf(nbytes, dtype=torch.uint8)
        H2 = (H + H_kv) * D
        self.heads = (self.qkv[:, :self.hd].unflatten(1, (H, D)),
                      self.qkv[:, self.hd:H2].unflatten(1, (H_kv, D)),
                      self.qkv[:, H2:].unflatten(1, (H_kv, D)))
        n1 = gdn.gdn_norm_shape(n, hidden, gdn.GDN_BF16, 1, 1e-6, 0.0)
        n2 = gdn.gdn_norm_shape(n, self.hd, gdn.GDN_BF16, 0, 0.0, 0.0)
        g1 = gdn.gdn_gemm_shape(n, self.wide, hidden, gdn.GDN_BF16)
        g2 = gdn.gdn_gemm_shape(n, hidden, self.hd, gdn.GDN_BF16)
        o2 = self.o.view(n, self.hd)
        self.calls = [
            lambda st: gdn.gdn_rmsnorm_fp8(n1, self.x, self.h, self.norm_w, self.h, None, self.x8,
                                           self.xs, st),
            lambda st: gdn.gdn_gemm_fp8(g1, self.x8, self.xs, self.w1, self.s1, self.qkv, st),
            lambda st: gdn.gdn_rope_append(self.rope, self.cache, *self.heads, self.pos, self.inv,
                                           self.slots, self.q, self.k, self.v, st),
            lambda st: gdn.gdn_paged_attention(self.attn, self.cache, self.q, self.k, self.v,
                                               self.table, self.lens, self.o, self.ws, nbytes, st),
            lambda st: gdn.gdn_rmsnorm_fp8(n2, o2, None, None, None, None, self.o8, self.os, st),
            lambda st: gdn.gdn_gemm_fp8(g2, self.o8, self.os, self.w2, self.s2, self.x, st)]

    def reset(self):
        for a, b in ((self.x, self.x0), (self.h, self.h0), (self.k, self.k0), (self.v, self.v0)):
            a.copy_(b)
        for a in (self.x8.view(torch.uint8), self.xs, self.qkv, self.q, self.o,
                  self.o8.view(torch.uint8), self.os):
            a.zero_()
        torch.cuda.synchronize()

    def run(self, stream, rounds, sync=False):
        for _ in range(rounds):
            for call in self.calls:
                call(stream)
                if sync:
                    torch.cuda.synchronize()

    def state(self):
        torch.cuda.synchronize()
        self.gdn.gdn_check_device_error()
        assert not bool(self.x.isnan().any())
        return [t.clone() for t in (self.x, self.h, self.qkv, self.q, self.o, self.k, self.v)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# decode (few rows), verify (square tiles), a prompt (pairs of blocks, rings)
SHAPES = [(5, 1), (64, 1), (136, 8), (520, 8), (6000, 8)]


@pytest.mark.parametrize("n,T", SHAPES)
def test_chains_without_synchronisation(gdn, n, T):
    layer = Layer(gdn, n, T)
    layer.run(torch.cuda.current_stream(), 3, sync=True)
    want = layer.state()
    stream = torch.cuda.Stream()
    for _ in range(3):
        layer.reset()
        layer.run(stream, 3)
        assert same(layer.state(), want)


@pytest.mark.parametrize("first,second", [
    # the product's forms for up to 16, 32 and 64 rows beside its square tiles,
    # and those beside pairs of blocks
    ((16, 1), (256, 8)), ((32, 1), (256, 8)), ((64, 1), (256, 8)), ((16, 1), (64, 1)),
    ((16, 1), (6000, 8)), ((256, 8), (6000, 8)), ((256, 8), (256, 8))])
def test_two_streams_at_once(gdn, first, second):
    layers = [Layer(gdn, *first, seed=1), Layer(gdn, *second, seed=2)]
    want = []
    for x in layers:
        x.run(torch.cuda.current_stream(), 20, sync=True)
        want.append(x.state())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in layers:
        x.reset()
    for _ in range(20):
        for x, st in zip(layers, streams):
            x.run(st, 1)
    for x, w in zip(layers, want):
        assert same(x.state(), w)


@pytest.mark.parametrize("n,T", SHAPES)
def test_no_allocation_and_no_synchronisation(gdn, n, T):
    layer = Layer(gdn, n, T)
    stream = torch.cuda.Stream()
    layer.run(stream, 2)               # the first launches load the kernels
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    done = torch.cuda.Event()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)   # some 0.2 s of the GPU
    layer.run(stream, 2)
    done.record(stream)
    assert not done.query()            # every call came back while the stream was busy
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    layer.state()
