"""gdn_tree_forward and gdn_tree_commit against the recurrence along every
branch in 64 bits, and against gdn_forward where the tree is a line.

Tolerance: relative L2 error 1e-5 over a whole tensor, the one that fp32 inputs
of the recurrence have everywhere here, for bf16 inputs too: their values are
exact, and the products and sums are as exact as fp32 ones (a sum of 128
products: 128 x 2^-24 of their size at most, some 1e-6 as a root of squares)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
TOL = 1e-5


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_net_02_gb300 import build
    build.build()
    from gated_delta_net_02_gb300 import gdn as mod
    assert torch.cuda.is_available()
    return mod


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm().clamp_min(1e-300))


def parents_of(kind, n, T, seed=0):
    rng = np.random.default_rng(seed)
    p = np.full((n, T), -1)
    for t in range(1, T):
        if kind == "line":
            p[:, t] = t - 1
        elif kind == "bush":
            p[:, t] = np.where(rng.random(n) < 0.15, -1, t - 1 - rng.integers(0, min(t, 5), n))
        elif kind == "binary":
            p[:, t] = (t - 1) // 2
    return p   # "star": every node follows the root


def words_of(parents):
    n, T = parents.shape
    w = np.zeros((n, T), np.uint64)
    for t in range(T):
        w[:, t] = np.uint64(1) << np.uint64(t)
        for s in range(n):
            if parents[s, t] >= 0:
                w[s, t] |= w[s, parents[s, t]]
    return torch.from_numpy(w.view(np.int64)).cuda()


class Case:
    def __init__(self, gdn, n, T, H, Dk, Dv, dtype, mode, kind="bush", H_qk=0, qk_map=0, nodes=None,
                 seed=0, zero_state=False, gate=None):
        g = torch.Generator("cuda").manual_seed(seed)
        self.gdn, self.n, self.T, self.H, self.Dk, self.Dv = gdn, n, T, H, Dk, Dv
        self.mode, self.Hq, self.qk_map = mode, H_qk or H, qk_map

        def randn(*s):
            return torch.randn(*s, generator=g, device="cuda")

        unit = torch.nn.functional.normalize
        self.q = unit(randn(n * T, self.Hq, Dk), dim=-1).to(dtype)
        self.k = unit(randn(n * T, self.Hq, Dk), dim=-1).to(dtype)
        self.v = randn(n * T, H, Dv).to(dtype)
        self.beta = torch.sigmoid(randn(n * T, H))
        soft = torch.nn.functional.softplus
        self.g = -soft(randn(n * T, H)) if mode == "gda" else -0.1 * soft(randn(n * T, H, Dk))
        if gate is not None:
            gate(self.g)
        self.state = randn(n, H, Dk, Dv) * 0.1
        self.ptrs = gdn.state_ptr_array(
            [0] * n if zero_state else gdn.per_seq_state_ptrs(self.state, n), "cuda")
        if zero_state:
            self.state.zero_()
        self.parents = parents_of(kind, n, T, seed)
        self.tree = words_of(self.parents)
        self.nodes = None if nodes is None else torch.tensor(nodes, device="cuda", dtype=torch.int32)
        self.shape = gdn.gdn_shape(n, T, H, Dk, Dv, gdn.dtype_code(dtype), 0.0, H_qk, qk_map)
        self.out = torch.full((n * T, H, Dv), float("nan"), device="cuda")
        self.updates = torch.full((n * T, H, Dv), float("nan"), device="cuda")
        torch.cuda.synchronize()

    def forward(self, stream=None, check=True):
        self.gdn.gdn_tree_forward(self.shape, self.q, self.k, self.v, self.g, self.beta, self.ptrs,
                                  self.nodes, self.tree, self.out, self.updates, self.mode, stream)
        torch.cuda.synchronize()
        if check:
            self.gdn.gdn_check_device_error()
        return self

    def commit(self, leaf, state_out=None, stream=None, check=True):
        leaf = torch.tensor(leaf, device="cuda", dtype=torch.int32)
        if state_out is None:
            state_out = torch.full_like(self.state, float("nan"))
        self.gdn.gdn_tree_commit(self.shape, self.k, self.g, self.updates, self.ptrs, self.tree,
                                 leaf, state_out, self.mode, stream)
        torch.cuda.synchronize()
        if check:
            self.gdn.gdn_check_device_error()
        return state_out

    def reference(self):
        """out, d [n, T, H, Dv] and every node's state, in 64 bits; padding 0."""
        n, T, H = self.n, self.T, self.H
        h = torch.arange(H, device="cuda")
        hq = h % self.Hq if self.qk_map == 0 else h // (H // self.Hq)
        q, k = (x.double().view(n, T, self.Hq, -1)[:, :, hq] for x in (self.q, self.k))
        v, beta = self.v.double().view(n, T, H, -1), self.beta.double().view(n, T, H, 1)
        a = self.g.double().exp().view(n, T, H, -1, 1)
        out, d = torch.zeros_like(v), torch.zeros_like(v)
        states = torch.zeros(n, T, H, self.Dk, self.Dv, dtype=torch.float64, device="cuda")
        for s in range(n):
            for t in range(T if self.nodes is None else int(self.nodes[s])):
                p = int(self.parents[s, t])
                S = self.state[s].double() if p < 0 else states[s, p]
                S = torch.where(a[s, t] == 0, 0.0, a[s, t] * S)
                d[s, t] = beta[s, t] * (v[s, t] - torch.einsum("hij,hi->hj", S, k[s, t]))
                S = S + k[s, t][:, :, None] * d[s, t][:, None]
                states[s, t] = S
                out[s, t] = self.Dk ** -0.5 * torch.einsum("hij,hi->hj", S, q[s, t])
        return out, d, states

    def check(self):
        out, d, states = self.reference()
        flat = (self.n * self.T, self.H, self.Dv)
        assert not bool(self.out.isnan().any()) and not bool(self.updates.isnan().any())
        assert rel(self.out, out.view(flat)) <= TOL
        assert rel(self.updates, d.view(flat)) <= TOL
        pad = (d == 0).all(-1).all(-1).view(-1)
        assert not bool(self.out[pad].any()) and not bool(self.updates[pad].any())
        return states


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["gda", "kda"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("T,kind", [(1, "line"), (2, "star"), (5, "bush"), (8, "line"), (16, "bush"),
                                    (17, "binary"), (33, "bush"), (64, "bush"), (64, "line")])
def test_trees(gdn, dtype, mode, Dk, Dv, T, kind):
    c = Case(gdn, 3, T, 2, Dk, Dv, dtype, mode, kind, seed=T + Dk).forward()
    states = c.check()
    leaf = [T - 1, T // 2, 0]
    want = torch.stack([states[s, leaf[s]] for s in range(3)])
    assert rel(c.commit(leaf), want) <= TOL


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["gda", "kda"])
@pytest.mark.parametrize("H,H_qk,qk_map", [(6, 3, 0), (6, 3, 1), (8, 1, 0), (5, 5, 1)])
def test_shared_heads_and_padding(gdn, dtype, mode, H, H_qk, qk_map):
    T, nodes = 12, [12, 5, 0, 1, 11]
    c = Case(gdn, 5, T, H, 128, 128, dtype, mode, H_qk=H_qk, qk_map=qk_map, nodes=nodes, seed=H)
    # what padding holds is not used
    for s, m in enumerate(nodes):
        for x in (c.q, c.k, c.v, c.g, c.beta):
            x[s * T + m:(s + 1) * T] = float("nan")
        c.tree[s, m:] = -12345
    c.forward()
    # the definition with the padding's inputs out of the way
    for x in (c.q, c.k, c.v, c.g, c.beta):
        x.nan_to_num_(0.0)
    states = c.check()
    leaf = [11, 4, -1, 0, 3]
    got = c.commit(leaf)
    want = torch.stack([c.state[s].double() if j < 0 else states[s, j] for s, j in enumerate(leaf)])
    assert rel(got, want) <= TOL and torch.equal(got[2], c.state[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["gda", "kda"])
@pytest.mark.parametrize("T", [1, 8, 20])
def test_a_line_is_gdn_forward(gdn, dtype, mode, T):
    n, H, D = 4, 3, 128
    c = Case(gdn, n, T, H, D, D, dtype, mode, "line", seed=T).forward()
    slots = torch.empty(n, T, H, D, D, device="cuda")
    out = torch.empty(n * T, H, D, device="cuda")
    gdn.gdn_forward(c.shape, c.q, c.k, c.v, c.g, c.beta, c.ptrs, slots, out, T, mode)
    gdn.gdn_check_device_error()
    assert rel(c.out, out) <= TOL
    for t in {0, T // 2, T - 1}:
        assert rel(c.commit([t] * n), slots[:, t]) <= TOL


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["gda", "kda"])
def test_gates_that_reset_grow_and_vanish(gdn, dtype, mode):
    def gate(g):
        flat = g.view(g.shape[0], g.shape[1], -1)
        flat[3::7, 0] = -math.inf          # whole rows of a head
        flat[5::7, 1, ::2] = -math.inf
        flat[2::5, 1] = 1.5                # growth
        flat[4::9] = -200.0                # far below fp32's range when multiplied
    c = Case(gdn, 3, 40, 2, 128, 128, dtype, mode, "bush", seed=1, gate=gate).forward()
    states = c.check()
    got = c.commit([39, 17, 4])
    assert rel(got, torch.stack([states[0, 39], states[1, 17], states[2, 4]])) <= TOL


@pytest.mark.parametrize("dtype", TYPES)
def test_zero_states(gdn, dtype):
    c = Case(gdn, 2, 9, 2, 64, 128, dtype, "gda", zero_state=True).forward()
    states = c.check()
    got = c.commit([8, -1])
    assert rel(got[0], states[0, 8]) <= TOL and not bool(got[1].any())


def test_commit_in_place(gdn):
    c = Case(gdn, 4, 10, 3, 128, 128, torch.bfloat16, "kda").forward()
    leaf = [9, -1, 0, 5]
    want, before = c.commit(leaf), c.state.clone()
    c.commit(leaf, state_out=c.state)
    assert torch.equal(c.state, want) and torch.equal(c.state[1], before[1])


def test_overlapping_states_are_refused(gdn):
    c = Case(gdn, 3, 4, 2, 64, 64, torch.bfloat16, "gda").forward()
    big = torch.zeros(5, 2, 64, 64, device="cuda")
    each = 4 * 2 * 64 * 64
    # sequence 1 reads the place of sequence 2; the others are elsewhere
    c.ptrs = gdn.state_ptr_array([c.state.data_ptr(), big.data_ptr() + 2 * each, 0], "cuda")
    got = torch.full((3, 2, 64, 64), 7.0, device="cuda")
    big[:3] = 7.0
    with pytest.raises(gdn.GDNError) as e:
        c.commit([3, 3, 3], state_out=big[:3])
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG
    assert torch.equal(big[1], got[1]) and not torch.equal(big[0], got[0])
    assert not torch.equal(big[2], got[2])


@pytest.mark.parametrize("word", [
    lambda w: w.__setitem__((1, 3), 0),                        # no own bit
    lambda w: w.__setitem__((1, 3), int(w[1, 3]) | 1 << 5),    # a later node
    lambda w: w.__setitem__((1, 4), 1 << 4 | 1 << 3),          # not the parent's ancestors
    lambda w: w.__setitem__((1, 5), -1)])
def test_words_that_are_no_tree(gdn, word):
    c = Case(gdn, 3, 8, 2, 128, 128, torch.bfloat16, "gda", "line")
    word(c.tree)
    c.forward(check=False)
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_check_device_error()
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG and "tree" in str(e.value)
    rows = c.out.view(3, 8, 2, 128)
    assert bool(rows[1].isnan().all()) and not bool(rows[::2].isnan().any())


@pytest.mark.parametrize("nodes", [[8, 9, 8], [8, -1, 8]])
def test_numbers_of_nodes_out_of_range(gdn, nodes):
    c = Case(gdn, 3, 8, 2, 128, 128, torch.float32, "gda", nodes=nodes)
    with pytest.raises(gdn.GDNError) as e:
        c.forward()
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG
    rows = c.out.view(3, 8, 2, 128)
    assert bool(rows[1].isnan().all()) and not bool(rows[::2].isnan().any())


@pytest.mark.parametrize("leaf", [8, -2, 1 << 30])
def test_leaves_out_of_range(gdn, leaf):
    c = Case(gdn, 3, 8, 2, 128, 128, torch.float32, "gda").forward()
    out = torch.full_like(c.state, float("nan"))
    with pytest.raises(gdn.GDNError) as e:
        c.commit([1, leaf, -1], state_out=out)
    assert e.value.status == gdn.GDN_ERR_DEVICE_ARG
    assert bool(out[1].isnan().all()) and not bool(out[::2].isnan().any())


def test_same_bits_every_time_and_on_another_stream(gdn):
    c = Case(gdn, 40, 16, 8, 128, 128, torch.bfloat16, "gda").forward()
    out, d, state = c.out.clone(), c.updates.clone(), c.commit([5] * 40)
    stream = torch.cuda.Stream()
    for _ in range(3):
        c.out.fill_(float("nan"))
        c.updates.fill_(float("nan"))
        c.forward(stream)
        assert torch.equal(c.out, out) and torch.equal(c.updates, d)
        assert torch.equal(c.commit([5] * 40, stream=stream), state)


def test_a_batch_changes_no_sequence(gdn):
    # a sequence alone and among others: the same bits
    c = Case(gdn, 9, 16, 4, 128, 128, torch.bfloat16, "kda").forward()
    one = Case(gdn, 9, 16, 4, 128, 128, torch.bfloat16, "kda")
    one.shape.n_seqs = 1
    one.forward()
    assert torch.equal(c.out[:16], one.out[:16]) and bool(one.out[16:].isnan().all())


def test_captured_and_replayed(gdn):
    c = Case(gdn, 4, 12, 4, 128, 128, torch.bfloat16, "gda").forward()
    leaf = torch.tensor([3, 11, -1, 6], device="cuda", dtype=torch.int32)
    state_out = torch.empty_like(c.state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream()
        gdn.gdn_tree_forward(c.shape, c.q, c.k, c.v, c.g, c.beta, c.ptrs, None, c.tree, c.out,
                             c.updates, c.mode, st)
        gdn.gdn_tree_commit(c.shape, c.k, c.g, c.updates, c.ptrs, c.tree, leaf, state_out, c.mode,
                            st)
    for seed in range(3):
        other = Case(gdn, 4, 12, 4, 128, 128, torch.bfloat16, "gda", seed=10 + seed)
        for x in ("q", "k", "v", "g", "beta", "state", "tree"):
            getattr(c, x).copy_(getattr(other, x))
        c.parents = other.parents
        graph.replay()
        torch.cuda.synchronize()
        gdn.gdn_check_device_error()
        states = c.check()
        want = torch.stack([states[0, 3], states[1, 11], c.state[2].double(), states[3, 6]])
        assert rel(state_out, want) <= TOL


def test_states_beyond_32_bits_of_elements(gdn):
    n, H, D = 2100, 64, 128     # 2.2e9 elements
    k = torch.nn.functional.normalize(torch.randn(n, H, D, device="cuda"), dim=-1).bfloat16()
    v, g = torch.randn(n, H, D, device="cuda").bfloat16(), torch.zeros(n, H, device="cuda")
    beta = torch.ones(n, H, device="cuda")
    state = torch.zeros(n, H, D, D, device="cuda")
    ptrs = gdn.state_ptr_array(gdn.per_seq_state_ptrs(state, n), "cuda")
    tree = torch.ones(n, 1, device="cuda", dtype=torch.int64)
    out, d = torch.empty(n, H, D, device="cuda"), torch.empty(n, H, D, device="cuda")
    shape = gdn.gdn_shape(n, 1, H, D, D, gdn.GDN_BF16, 1.0)
    for _ in range(2):   # the second reads what the first committed
        gdn.gdn_tree_forward(shape, k, k, v, g, beta, ptrs, None, tree, out, d, "gda")
        gdn.gdn_tree_commit(shape, k, g, d, ptrs, tree, torch.zeros(n, device="cuda", dtype=torch.int32),
                            state, "gda")
    gdn.gdn_check_device_error()
    # beta = 1 on a bf16-rounded unit key: S^T k is v |k|^2, and |k|^2 is 1 to 2^-8
    for s in (0, 1023, n - 1):
        got = torch.einsum("hij,hi->hj", state[s], k[s].float())
        assert rel(got, v[s]) <= 2.0 ** -7
