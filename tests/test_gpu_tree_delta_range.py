"""gdn_tree_forward on states whose elements differ widely in size, element by
element against the recurrence in 64 bits.

Tolerance of an element: (1 + depth) x 1e-5 of its size, the size being the same
recurrence over absolute values (S' = a S' + |k| d', d' = beta (|v| + S'^T |k|),
o' = scale S'^T |q|), which bounds the sum of the sizes of all products behind the
element. A level of the tree adds to it at most 128 roundings of a sum of 128
products and less than 40 of decays, parts, ancestors' products, beta and scale,
2^-24 each: 168 x 2^-24 = 1.0e-5. Sums that hold a number only to a fraction of the
largest one beside it miss this by orders of magnitude for the small ones."""
import pytest
import torch

from test_gpu_tree_delta import TYPES, Case, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def columns(c):
    # columns from 1 down to 1e-6, and v with them; neighbours differ
    size = 10.0 ** (-6.0 * torch.arange(c.Dv, device="cuda") / (c.Dv - 1))
    size = size[torch.arange(c.Dv, device="cuda") * 37 % c.Dv]
    c.state *= size
    c.v *= size


def first_rows_zero(size):
    def f(c):
        c.state *= size
        c.state[:, :, :16] = 0
        c.state[:, :, c.Dk // 2:c.Dk // 2 + 16] = 0
        c.v *= size
    return f


def rows(c):
    # each other row a millionth, and keys and queries that see those rows alone
    c.state[:, :, ::2] *= 1e-6
    c.v *= 1e-6
    c.k[:, :, 1::2] = 0
    c.q[:, :, 1::2] = 0


def keys(c):
    # keys and queries that are large where the state is small
    size = 10.0 ** (-5.0 * torch.rand(c.Dk, device="cuda"))
    c.state *= size[:, None]
    c.k /= size / size.min()
    c.q /= size / size.min()


def ends(c):
    # a first element beside which the others of its block are 1e-7
    c.state *= 1e-6
    c.v *= 1e-6
    c.state[:, :, 0, ::32] = 1.0
    c.k[:, :, 0] = 0
    c.q[:, :, 0] = 0


FORMS = {"columns": columns, "1e-2": first_rows_zero(1e-2), "1e-4": first_rows_zero(1e-4),
         "1e-7": first_rows_zero(1e-7), "1e-20": first_rows_zero(1e-20), "rows": rows, "keys": keys,
         "ends": ends}


def sizes(c):
    """Size of every element of out and updates, and the nodes' depths."""
    n, T, H = c.n, c.T, c.H
    q, k = (x.double().abs().view(n, T, c.Hq, -1) for x in (c.q, c.k))
    v, beta = c.v.double().abs().view(n, T, H, -1), c.beta.double().view(n, T, H, 1)
    a = c.g.double().exp().view(n, T, H, -1, 1)
    out, d = torch.zeros_like(v), torch.zeros_like(v)
    states = torch.zeros(n, T, H, c.Dk, c.Dv, dtype=torch.float64, device="cuda")
    depth = torch.zeros(n, T, 1, 1, dtype=torch.float64, device="cuda")
    for s in range(n):
        for t in range(T):
            p = int(c.parents[s, t])
            depth[s, t] = 0 if p < 0 else depth[s, p] + 1
            S = a[s, t] * (c.state[s].double().abs() if p < 0 else states[s, p])
            d[s, t] = beta[s, t] * (v[s, t] + torch.einsum("hij,hi->hj", S, k[s, t]))
            S = S + k[s, t][:, :, None] * d[s, t][:, None]
            states[s, t] = S
            out[s, t] = c.Dk ** -0.5 * torch.einsum("hij,hi->hj", S, q[s, t])
    return out, d, depth


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["gda", "kda"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [5, 14, 40])
@pytest.mark.parametrize("form", FORMS)
def test_sizes_of_states(gdn, dtype, mode, Dk, Dv, T, form):
    c = Case(gdn, 2, T, 2, Dk, Dv, dtype, mode, "bush", seed=T + Dv)
    FORMS[form](c)
    c.forward()
    out, d, _ = c.reference()
    out_size, d_size, depth = sizes(c)
    tol = 1e-5 * (1 + depth)
    assert bool(((c.updates.double().view_as(d) - d).abs() <= tol * d_size).all())
    assert bool(((c.out.double().view_as(out) - out).abs() <= tol * out_size).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_tiny_and_huge_states(gdn, dtype, size):
    c = Case(gdn, 2, 10, 2, 128, 128, dtype, "kda", "bush", seed=3)
    c.state *= size
    c.v *= size
    c.forward()
    out, d, _ = c.reference()
    out_size, d_size, depth = sizes(c)
    tol = 1e-5 * (1 + depth)
    assert bool(((c.updates.double().view_as(d) - d).abs() <= tol * d_size).all())
    assert bool(((c.out.double().view_as(out) - out).abs() <= tol * out_size).all())
