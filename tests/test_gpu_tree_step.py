"""The calls for trees of drafted tokens one after the other, as a model with
both kinds of layer verifies a draft: the nodes' keys and values into the
cache, their attention, the delta rule along the branches, a token for every
node, and the state after the accepted one. Every stage is held to its own 64-bit
definition, from what the stage before left, with the tolerance that its own
tests derive."""
import threading
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from test_gpu_qknorm_rope import check as check_rotated, normed
from test_gpu_rope_append import axis_of_freq
from test_gpu_sample import reference as chosen
from test_gpu_tree_attention import TreeCase
from test_gpu_tree_delta import TOL, Case as DeltaCase, gdn, parents_of, rel, words_of  # noqa: F401

pytestmark = pytest.mark.gpu


class Step:
    """One step of n sequences with trees of up to T nodes, which have 40, 177, ..
    keys before them. reset() takes back what a step changes."""

    def __init__(self, gdn, n, T, H=8, H_kv=2, D=128, vocab=5003, mode="gda", seed=0, ragged=True):
        g = torch.Generator("cuda").manual_seed(seed)
        self.gdn, self.n, self.T, self.H, self.H_kv, self.D, self.V = gdn, n, T, H, H_kv, D, vocab
        self.mode, page = mode, 16

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        rows, wide = n * T, (H + 2 * H_kv) * D
        self.parents = parents_of("bush", n, T, seed)
        self.tree = words_of(self.parents)
        self.nodes_host = [max(1, T - 3 * s % T if ragged else T) for s in range(n)]
        self.nodes = torch.tensor(self.nodes_host, device="cuda", dtype=torch.int32)
        before = [40 + 137 * s for s in range(n)]
        self.lens_host = [b + m for b, m in zip(before, self.nodes_host)]
        self.lens = torch.tensor(self.lens_host, device="cuda", dtype=torch.int32)
        per = -(-max(self.lens_host) // page)
        self.table = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per)
        depth = np.zeros((n, T), np.int64)
        for t in range(1, T):
            up = self.parents[:, t]
            depth[:, t] = np.where(up < 0, 0, depth[np.arange(n), up] + 1)
        self.pos = (torch.tensor(before)[:, None] + torch.from_numpy(depth)).to(torch.int32).cuda().view(1, -1)
        slots = torch.full((n, T), -1, dtype=torch.int64)
        table = self.table.cpu()
        for s in range(n):
            at = before[s] + torch.arange(self.nodes_host[s])
            slots[s, :len(at)] = table[s, at // page].long() * page + at % page
        self.slots = slots.view(-1).cuda()
        self.cache = gdn.gdn_kv_cache(n * per, page, H_kv, D, gdn.GDN_BF16, 0, 0, 0)
        self.k0, self.v0 = (randn(n * per, page, H_kv, D).bfloat16() for _ in range(2))
        self.kc, self.vc = self.k0.clone(), self.v0.clone()
        self.qkv = (2 * randn(rows, wide)).bfloat16()
        self.heads = [x.unflatten(1, (-1, D)) for x in
                      self.qkv.split([H * D, H_kv * D, H_kv * D], dim=1)]
        self.norm = gdn.gdn_qk_norm(1e-6, 1.0)
        self.qw, self.kw = (0.2 * randn(D).bfloat16() for _ in range(2))
        self.inv = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        self.rope = gdn.gdn_rope_shape(rows, H, D, 0, 1, (gdn.c_int * 4)(D // 2), 0, wide, wide, wide)
        self.attn = gdn.gdn_attn_shape(n, T, H, per, 0.0, gdn.GDN_QK_GROUPED)
        self.ws_bytes = gdn.gdn_tree_attention_workspace_size(self.attn, self.cache)
        unit = torch.nn.functional.normalize
        self.dq, self.dk = (unit(randn(rows, H, D), dim=-1).bfloat16() for _ in range(2))
        soft = torch.nn.functional.softplus
        self.g = -soft(randn(rows, H)) if mode == "gda" else -0.1 * soft(randn(rows, H, D))
        self.beta = torch.sigmoid(randn(rows, H))
        self.state0 = 0.1 * randn(n, H, D, D)
        self.state = self.state0.clone()
        self.ptrs = gdn.state_ptr_array(gdn.per_seq_state_ptrs(self.state, n), "cuda")
        self.shape = gdn.gdn_shape(n, T, H, D, D, gdn.GDN_BF16, 0.0, 0, 0)
        self.head = randn(H * D, vocab) * 0.5
        self.temperature = 0.4 + torch.rand(rows, generator=g, device="cuda")
        self.top_p = 0.5 + 0.5 * torch.rand(rows, generator=g, device="cuda")
        self.top_k = torch.randint(0, 90, (rows,), generator=g, device="cuda", dtype=torch.int32)
        self.u = torch.rand(rows, generator=g, device="cuda")
        self.sample = gdn.gdn_sample_shape(rows, vocab, gdn.GDN_F32, 0)
        f = dict(device="cuda")
        self.q, self.o = (torch.empty(rows, H, D, dtype=torch.bfloat16, **f) for _ in range(2))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, **f)
        self.out, self.updates = (torch.empty(rows, H, D, **f) for _ in range(2))
        self.logits = torch.empty(rows, vocab, **f)
        self.tokens, self.leaf = torch.empty(rows, dtype=torch.int32, **f), torch.empty(n, dtype=torch.int32, **f)
        self.probs = torch.empty(rows, **f)
        self.reset()

    def reset(self):
        for a, b in ((self.kc, self.k0), (self.vc, self.v0), (self.state, self.state0)):
            a.copy_(b)
        for x in (self.q, self.o, self.out, self.updates, self.logits, self.probs):
            x.fill_(float("nan"))
        self.ws.fill_(0xff)
        self.tokens.fill_(-7)
        self.leaf.fill_(-7)
        torch.cuda.synchronize()

    def run(self, stream, commit=True):
        g = self.gdn
        with torch.cuda.stream(stream):
            g.gdn_qknorm_rope_append(self.rope, self.cache, self.norm, *self.heads, self.qw, self.kw,
                                     self.pos, self.inv, self.slots, self.q, self.kc, self.vc, stream)
            g.gdn_tree_attention(self.attn, self.cache, self.q, self.kc, self.vc, self.table, self.lens,
                                 self.nodes, self.tree, self.o, self.ws, self.ws_bytes, stream)
            g.gdn_tree_forward(self.shape, self.dq, self.dk, self.o, self.g, self.beta, self.ptrs,
                               self.nodes, self.tree, self.out, self.updates, self.mode, stream)
            torch.mm(self.out.view(self.n * self.T, -1), self.head, out=self.logits)
            g.gdn_sample(self.sample, self.logits, self.temperature, self.top_k, self.top_p, None,
                         self.u, self.tokens, self.probs, stream)
            # the node that is accepted: any that the tokens name
            torch.remainder(self.tokens.view(self.n, self.T)[:, 0], self.nodes, out=self.leaf)
            if commit:   # in place
                g.gdn_tree_commit(self.shape, self.dk, self.g, self.updates, self.ptrs, self.tree,
                                  self.leaf, self.state, self.mode, stream)

    def results(self):
        torch.cuda.synchronize()
        self.gdn.gdn_check_device_error()
        return [x.clone() for x in (self.q, self.kc, self.vc, self.o, self.out, self.updates,
                                    self.tokens, self.probs, self.leaf, self.state)]

    def check(self):
        T, D, half = self.T, self.D, self.D // 2
        axis = axis_of_freq((half,), half, False)
        q, k, v = self.heads
        use = self.slots >= 0
        at = self.slots[use]
        check_rotated(self.q, normed(q, self.qw, 1.0, 1e-6), self.pos, self.inv, axis, D, False)
        check_rotated(self.kc[at // 16, at % 16], normed(k, self.kw, 1.0, 1e-6)[use],
                      self.pos[:, use], self.inv, axis, D, False)
        assert torch.equal(self.vc[at // 16, at % 16], v[use])
        keys = []
        for s, n in enumerate(self.lens_host):
            at = torch.arange(n, device="cuda")
            pages = self.table[s, at // 16].long()
            keys.append((self.kc[pages, at % 16], self.vc[pages, at % 16]))
        TreeCase.check(SimpleNamespace(
            T=T, H=self.H, H_kv=self.H_kv, kv_map=1, lens_host=self.lens_host,
            nodes_host=self.nodes_host, words=self.tree.cpu().numpy().view(np.uint64), keys=keys,
            q=self.q, scale=D ** -0.5), self.o)
        out, d, states = DeltaCase.reference(SimpleNamespace(
            n=self.n, T=T, H=self.H, Hq=self.H, qk_map=0, q=self.dq, k=self.dk, v=self.o,
            beta=self.beta, g=self.g, parents=self.parents, nodes=self.nodes, state=self.state0,
            Dk=D, Dv=D))
        assert rel(self.out, out.view_as(self.out)) <= TOL
        assert rel(self.updates, d.view_as(self.updates)) <= TOL
        logits = self.logits.double().cpu()
        for i in range(0, self.n * T, 7):
            token, p = chosen(logits[i], float(self.temperature[i]), int(self.top_k[i]),
                              float(self.top_p[i]), 0.0, float(self.u[i]))
            assert int(self.tokens[i]) == token
            assert abs(float(self.probs[i]) - p) <= 2.0 ** -22 * p + 2.0 ** -38
        want = torch.stack([states[s, int(self.leaf[s])] for s in range(self.n)])
        assert rel(self.state, want) <= TOL


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("mode", ["gda", "kda"])
@pytest.mark.parametrize("n,T,H,H_kv", [(1, 1, 8, 2), (3, 7, 6, 3), (5, 16, 8, 2), (4, 32, 8, 1),
                                        (3, 64, 12, 3)])
def test_a_step(gdn, n, T, H, H_kv, mode):
    x = Step(gdn, n, T, H, H_kv, mode=mode, seed=T)
    x.run(torch.cuda.current_stream())
    x.results()
    x.check()


@pytest.mark.parametrize("T", [8, 64])
def test_captured_and_replayed(gdn, T):
    x, stream = Step(gdn, 4, T, seed=1), torch.cuda.Stream()
    x.run(stream)
    want = x.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        x.run(stream)
    for _ in range(3):
        x.reset()
        graph.replay()
        assert same(x.results(), want)
    # other trees, numbers of nodes, lengths and inputs in the same places
    y = Step(gdn, 4, T, seed=2, ragged=False)
    for a, b in ((x.tree, y.tree), (x.qkv, y.qkv), (x.g, y.g), (x.u, y.u)):
        a.copy_(b)
    x.parents = y.parents
    x.reset()
    graph.replay()
    x.results()
    x.check()


@pytest.mark.parametrize("first,second", [((4, 8), (6, 16)), ((4, 32), (3, 64)), ((3, 64), (3, 64))])
def test_two_streams_at_once(gdn, first, second):
    steps = [Step(gdn, *first, seed=3), Step(gdn, *second, mode="kda", seed=4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for x in steps:
        x.run(torch.cuda.current_stream())
        want.append(x.results())
    for _ in range(5):
        for x in steps:
            x.reset()
        for _ in range(4):   # commits change no call before them but through the state
            for x, stream in zip(steps, streams):
                x.run(stream, commit=False)
        for x, stream in zip(steps, streams):
            x.run(stream)
        for x, w in zip(steps, want):
            assert same(x.results(), w)


def test_two_threads_at_once(gdn):
    steps = [Step(gdn, 4, 16, seed=5), Step(gdn, 3, 64, mode="kda", vocab=70001, seed=6)]
    want = []
    for x in steps:
        x.run(torch.cuda.current_stream())
        want.append(x.results())
        x.reset()
    errors, start = [], threading.Barrier(2)

    def work(x):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(20):
                x.run(stream, commit=False)
            x.run(stream)
            stream.synchronize()
        except Exception as e:   # noqa: BLE001  told by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(x,)) for x in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for x, w in zip(steps, want):
        assert same(x.results(), w)


@pytest.mark.parametrize("T", [8, 64])
def test_no_allocation_and_no_synchronisation(gdn, T):
    x, stream = Step(gdn, 4, T, seed=7), torch.cuda.Stream()
    x.run(stream)                      # the first launches load the kernels
    want = x.results()
    x.reset()
    free = torch.cuda.mem_get_info()[0]
    done = torch.cuda.Event()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)   # some 0.2 s of the GPU
    x.run(stream)
    done.record(stream)
    assert not done.query()            # every call came back while the stream was busy
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    assert same(x.results(), want)
