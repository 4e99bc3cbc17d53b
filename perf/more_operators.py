"""The measured cases of the operators that verify a tree of drafted tokens in
a hybrid model (layers of the gated delta rule, layers of attention).

Five operators of the framework, each with a plain form in elementary torch
operations:

  qknorm  gdn_qknorm_rope_append: RMS norm of every q and k head, rotary
          positions, and k and v written into the pages of a key-value cache
  attend  gdn_tree_attention: attention of a tree of drafted tokens over the
          sequence's pages: the whole prefix, and a node's own ancestors
  delta   gdn_tree_forward: the gated delta rule along every branch of the
          tree, from one state for each sequence
  commit  gdn_tree_commit: the state after the branch that was accepted
  sample  gdn_sample: one token for each row of logits (temperature, top-k,
          top-p, min-p) from given random numbers

A tree is one 64-bit word for each node: bit j of word t says that node j is an
ancestor of node t or t itself; an ancestor has a smaller number.

``own`` false: the plain form; true: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----------------------------------------------------------------

def listed():
    return [
        # the drafted tokens of a few sequences: latency is all there is
        dict(name="qknorm decode", op="qknorm", tokens=64, H=16, H_kv=2, D=128, rot=128, axes=1,
             interleaved=False, pairs=False, page=16, max_pos=8192, dtype="bf16", offset=0.0),
        # a prefill batch's tokens with image positions, part of the head rotated
        dict(name="qknorm prefill", op="qknorm", tokens=34739, H=16, H_kv=2, D=256, rot=64, axes=3,
             interleaved=True, pairs=False, page=64, max_pos=131072, dtype="bf16", offset=1.0),
        # one sequence of a chat, 16 drafted tokens
        dict(name="attend one", op="attend", seqs=1, T=16, H=16, H_kv=2, D=128, page=16,
             min_len=1025, max_len=1025, dtype="bf16", ragged=False),
        # 32 ragged sequences with trees of up to 32 nodes
        dict(name="attend batch", op="attend", seqs=32, T=32, H=16, H_kv=2, D=128, page=16,
             min_len=512, max_len=8192, dtype="bf16", ragged=True),
        # the widest trees over long contexts, wide heads
        dict(name="attend long", op="attend", seqs=8, T=64, H=16, H_kv=2, D=256, page=64,
             min_len=30000, max_len=65000, dtype="bf16", ragged=False),
        # trees of 8 nodes in the recurrence: the shape that a line of 8 drafts has
        dict(name="delta verify", op="delta", seqs=32, T=8, H=16, H_qk=16, Dk=128, Dv=128,
             kda=False, dtype="bf16", ragged=False),
        # large batch, 32 nodes, gates for each row
        dict(name="delta wide", op="delta", seqs=64, T=32, H=32, H_qk=32, Dk=128, Dv=128,
             kda=True, dtype="bf16", ragged=True),
        # fp32, few sequences, shared q and k heads, odd sizes
        dict(name="delta odd f32", op="delta", seqs=3, T=13, H=6, H_qk=3, Dk=64, Dv=128, kda=False,
             dtype="f32", ragged=True),
        # the accepted branch into the states of a small batch
        dict(name="commit verify", op="commit", seqs=32, T=8, H=16, H_qk=16, Dk=128, Dv=128,
             kda=False, dtype="bf16"),
        # and of a large one
        dict(name="commit wide", op="commit", seqs=128, T=32, H=32, H_qk=32, Dk=128, Dv=128,
             kda=True, dtype="bf16"),
        # one decode step of 64 sequences, each with its own settings
        dict(name="sample decode", op="sample", rows=64, vocab=131072, dtype="bf16", top_k=50,
             top_p=True, min_p=False),
        # every node of 32 trees of 16, an odd vocabulary, no limit on their number
        dict(name="sample trees", op="sample", rows=512, vocab=150001, dtype="f32", top_k=0,
             top_p=True, min_p=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["qknorm", "attend", "delta", "commit", "sample"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    e = 4 if dtype == "f32" else 2
    if op == "sample":
        vocab = _log(rng, 32, 262144)
        rows = _log(rng, 1, min(1024, 512 * 150001 // vocab))
        return dict(op=op, rows=rows, vocab=vocab, dtype=dtype,
                    top_k=rng.choice([0, 0, 1, 20, 50, 1000]), top_p=rng.random() < 0.6,
                    min_p=rng.random() < 0.4)
    if op in ("delta", "commit"):
        Dk, Dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        H_qk = rng.choice([1, 2, 3, 4, 8, 16])
        H = H_qk * rng.choice([1, 1, 2, 3, 4])
        T = rng.choice([1, 2, 5, 8, 13, 16, 24, 32, 48, 64])
        most = (64 if op == "delta" else 128) * 32 * 32
        seqs = _log(rng, 1, max(1, min(256, most // (H * max(T, 32)))))
        c = dict(op=op, seqs=seqs, T=T, H=H, H_qk=H_qk, Dk=Dk, Dv=Dv, kda=rng.random() < 0.4,
                 dtype=dtype)
        if op == "delta":
            c["ragged"] = rng.random() < 0.5
        return c
    D = rng.choice([64, 128, 256])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    H = H_kv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([1, 7, 16, 32, 64, 100, 256])
    if op == "qknorm":
        axes = rng.choice([1, 2, 3])
        rot = D if rng.random() < 0.5 else 2 * axes * rng.randint(1, D // (2 * axes))
        tokens = _log(rng, 1, min(34739, 34739 * 20 * 256 * 2 // ((H + 2 * H_kv) * D * e)))
        return dict(op=op, tokens=tokens, H=H, H_kv=H_kv, D=D, rot=rot, axes=axes,
                    interleaved=rng.random() < 0.5, pairs=rng.random() < 0.3, page=page,
                    max_pos=_log(rng, 4096, 131072), dtype=dtype,
                    offset=rng.choice([0.0, 1.0]))
    T = rng.choice([1, 2, 5, 8, 13, 16, 24, 32, 48, 64])
    seqs = _log(rng, 1, 128)
    most = 8 * 47000 * 2 * 256 // (seqs * H_kv * D * (e // 2))       # keys by their bytes
    most = min(most, 8 * 47000 * 16 * 64 * 256 // (seqs * H * T * D * (16 if e == 4 else 1)))
    max_len = max(T, _log(rng, 1, max(2, min(131072, most))))
    return dict(op=op, seqs=seqs, T=T, H=H, H_kv=H_kv, D=D, page=page,
                min_len=max(T, _log(rng, 1, max_len)), max_len=max_len, dtype=dtype,
                ragged=rng.random() < 0.5)


def _lengths(c):
    """The sequences' lengths, spread evenly between the shortest and the longest."""
    n = c["seqs"]
    if n == 1:
        return [c["max_len"]]
    return [c["min_len"] + (c["max_len"] - c["min_len"]) * i // (n - 1) for i in range(n)]


def _sections(c):
    """Frequencies of each axis: an even split, the first axis takes the rest."""
    half, axes = c["rot"] // 2, c["axes"]
    each = half // axes
    return [half - each * (axes - 1)] + [each] * (axes - 1)


def _axis_of_freq(c):
    """Axis of each frequency: one run per axis, or the axes in turn."""
    sec, half = _sections(c), c["rot"] // 2
    if not c["interleaved"]:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    return [i % len(sec) if i // len(sec) < sec[i % len(sec)] else 0 for i in range(half)]


# ---- inputs ---------------------------------------------------------------

def _trees(n, T, seed):
    """[n][T] words of ancestors: a node continues one of the six before it,
    or, one time in ten, starts a branch at the root."""
    rng = np.random.default_rng(seed)
    words = np.zeros((n, T), np.uint64)
    at = np.arange(n)
    for t in range(T):
        words[:, t] = np.uint64(1) << np.uint64(t)
        if t:
            parent = t - 1 - rng.integers(0, min(t, 6), n)
            parent[rng.random(n) < 0.1] = -1
            words[:, t] |= np.where(parent >= 0, words[at, np.maximum(parent, 0)], np.uint64(0))
    return words


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": c}
    dt = TYPES[c["dtype"]]
    if c["op"] in ("attend", "delta", "commit"):
        n, T = c["seqs"], c["T"]
        s["tree"] = torch.from_numpy(_trees(n, T, seed).view(np.int64)).cuda()
        s["n_nodes"] = None
        if c.get("ragged"):
            s["n_nodes"] = torch.randint(T // 2, T + 1, (n,), generator=gen, device="cuda",
                                         dtype=torch.int32)
    if c["op"] == "qknorm":
        n, D = c["tokens"], c["D"]
        # q, k and v are column ranges of the projection's output
        s["qkv"] = randn(n, (c["H"] + 2 * c["H_kv"]) * D, dtype=dt, std=3.0)
        s["q_weight"] = (1 - c["offset"] + 0.1 * randn(D)).to(dt)
        s["k_weight"] = (1 - c["offset"] + 0.1 * randn(D)).to(dt)
        s["eps"] = 1e-6
        s["positions"] = torch.randint(0, c["max_pos"], (c["axes"], n), generator=gen,
                                       device="cuda", dtype=torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        pages = -(-n // c["page"]) + 3
        s["slots"] = torch.randperm(pages * c["page"], generator=gen, device="cuda")[:n].contiguous()
        s["k_cache"] = randn(pages, c["page"], c["H_kv"], D, dtype=dt)
        s["v_cache"] = randn(pages, c["page"], c["H_kv"], D, dtype=dt)
        s["q_out"] = empty(n, c["H"], D, dtype=dt)
    elif c["op"] == "attend":
        D, page = c["D"], c["page"]
        lens = torch.tensor(_lengths(c), device="cuda")[
            torch.randperm(n, generator=gen, device="cuda")]
        most = -(-c["max_len"] // page)
        used = int(((lens + page - 1) // page).sum())
        pages = used + 5
        s["k_cache"] = randn(pages, page, c["H_kv"], D, dtype=dt)
        s["v_cache"] = randn(pages, page, c["H_kv"], D, dtype=dt)
        held = torch.arange(most, device="cuda")[None] * page < lens[:, None]
        table = torch.zeros(n, most, device="cuda", dtype=torch.int32)
        table[held] = torch.randperm(pages, generator=gen, device="cuda")[:used].to(torch.int32)
        s["table"], s["lens"] = table, lens.to(torch.int32)
        s["q"] = randn(n * T, c["H"], D, dtype=dt, std=2.0)
        s["scale"] = D ** -0.5
        s["out"] = empty(n * T, c["H"], D, dtype=dt)
    elif c["op"] in ("delta", "commit"):
        H, Dk, Dv = c["H"], c["Dk"], c["Dv"]
        unit = torch.nn.functional.normalize
        s["k"] = unit(randn(n * T, c["H_qk"], Dk), dim=-1).to(dt)
        if c["kda"]:
            s["g"] = -0.1 * torch.nn.functional.softplus(randn(n * T, H, Dk))
        else:
            s["g"] = -torch.nn.functional.softplus(randn(n * T, H))
        s["state"] = randn(n, H, Dk, Dv, std=0.05)
        s["state_in"] = s["state"].data_ptr() + 4 * H * Dk * Dv * torch.arange(n, device="cuda")
        if c["op"] == "delta":
            s["q"] = unit(randn(n * T, c["H_qk"], Dk), dim=-1).to(dt)
            s["v"] = randn(n * T, H, Dv, dtype=dt)
            s["beta"] = torch.sigmoid(randn(n * T, H))
            s["scale"] = Dk ** -0.5
            s["out"], s["updates"] = empty(n * T, H, Dv), empty(n * T, H, Dv)
        else:
            s["updates"] = randn(n * T, H, Dv, std=0.6)
            s["leaf"] = torch.randint(-1, T, (n,), generator=gen, device="cuda", dtype=torch.int32)
            s["state_out"] = empty(n, H, Dk, Dv)
    else:
        n, V = c["rows"], c["vocab"]
        # many unlikely tokens, some likely ones
        x = randn(n, V, std=2.0)
        s["logits"] = (x + 8.0 * (rand(n, V) < 20.0 / V)).to(dt)
        s["temperature"] = 0.5 + rand(n)
        if n > 8:
            s["temperature"][torch.randint(0, n, (n // 8,), generator=gen, device="cuda")] = 0.0
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if c["top_k"]:
            s["top_k"] = torch.randint(1, c["top_k"] + 1, (n,), generator=gen, device="cuda",
                                       dtype=torch.int32)
        if c["top_p"]:
            s["top_p"] = 0.7 + 0.3 * rand(n)
        if c["min_p"]:
            s["min_p"] = 0.1 * rand(n)
        s["uniform"] = rand(n)
        s["tokens"] = empty(n, dtype=torch.int32)
        s["probs"] = empty(n)
    return s


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "qknorm":
        wide = c["H"] + 2 * c["H_kv"]
        heads = c["H"] + c["H_kv"]
        return {"bytes": c["tokens"] * (2 * wide * c["D"] * e + 4 * c["axes"] + 8),
                "flops": c["tokens"] * heads * (4 * c["D"] + 3 * c["rot"])}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * e + 24), "flops": 4 * c["rows"] * c["vocab"]}
    n, T, H = c["seqs"], c["T"], c["H"]
    if c["op"] == "attend":
        tokens = sum(_lengths(c))
        return {"bytes": 2 * e * c["H_kv"] * c["D"] * tokens + 2 * e * n * T * H * c["D"],
                "flops": 4 * T * H * c["D"] * tokens}
    Dk, Dv, gate = c["Dk"], c["Dv"], c["Dk"] if c["kda"] else 1
    if c["op"] == "delta":
        token = 2 * e * c["H_qk"] * Dk + H * (e * Dv + 4 * gate + 4 + 8 * Dv)
        return {"bytes": n * (4 * H * Dk * Dv + T * token), "flops": 4 * n * T * H * Dk * Dv}
    depth = min(T, 1 + T // 4)
    token = e * c["H_qk"] * Dk + H * (4 * gate + 4 * Dv)
    return {"bytes": n * (8 * H * Dk * Dv + depth * token),
            "flops": 2 * n * H * Dk * Dv * (depth + 1)}


# ---- one pass ---------------------------------------------------------------

def run(state):
    if own:
        return OWN[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


def _split(a):
    """a as the sum of two fp32 numbers of 12 bits each (Veltkamp)."""
    t = a * 4097.0
    hi = t - (t - a)
    return hi, a - hi


def _product(a, b):
    """a b as the sum of two fp32 numbers (Dekker)."""
    p = a * b
    (ah, al), (bh, bl) = _split(a), _split(b)
    return p, ((ah * bh - p) + ah * bl + al * bh) + al * bl


def _angles(s):
    """Rotation angles [tokens, rot/2] within a turn: position x inverse
    frequency, kept to 32 bits beyond the whole turns, which fp32 alone loses
    at long positions."""
    c = s["case"]
    if "axis" not in s:   # sizes alone: a program builds this once for its model
        s["axis"] = torch.tensor(_axis_of_freq(c)).cuda()
    pos = s["positions"].float()[s["axis"]].T           # exact below 2^24
    inv_hi = torch.full((), 1 / (2 * math.pi), dtype=torch.float32, device=pos.device)
    inv_lo = 1 / (2 * math.pi) - 0.15915493667125702    # what fp32 leaves of 1/(2 pi)
    f_hi, f_lo = _product(s["inv_freq"], inv_hi)
    f_lo = f_lo + s["inv_freq"] * inv_lo
    t, rest = _product(pos, f_hi.expand_as(pos))
    turns = (t - torch.round(t)) + (rest + pos * f_lo)
    return turns * (2 * math.pi)


def _rotate(x, cos, sin, rot, pairs):
    """x [tokens, heads, D] with its first `rot` elements rotated."""
    r = x[..., :rot]
    if pairs:
        a, b = r[..., 0::2], r[..., 1::2]
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
    cos, sin = cos[:, None], sin[:, None]
    c, d = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((c, d), -1).flatten(-2) if pairs else torch.cat((c, d), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _heads(s):
    c = s["case"]
    H, G, D = c["H"], c["H_kv"], c["D"]
    qkv = s["qkv"]
    return (qkv[:, :H * D].unflatten(1, (H, D)), qkv[:, H * D:(H + G) * D].unflatten(1, (G, D)),
            qkv[:, (H + G) * D:].unflatten(1, (G, D)))


def _plain_qknorm(s):
    c = s["case"]
    angle = _angles(s)
    cos, sin = torch.cos(angle), torch.sin(angle)
    q, k, v = _heads(s)
    dt = s["qkv"].dtype

    def head(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        return _rotate(x * (c["offset"] + weight.float()), cos, sin, c["rot"], c["pairs"]).to(dt)

    s["k_cache"].view(-1, c["H_kv"], c["D"])[s["slots"]] = head(k, s["k_weight"])
    s["v_cache"].view(-1, c["H_kv"], c["D"])[s["slots"]] = v
    return {"q": head(q, s["q_weight"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _bits(words, T):
    """[..., T] truth values of 64-bit words."""
    return (words[..., None] >> torch.arange(T, device=words.device) & 1).bool()


def _plain_attend(s):
    c = s["case"]
    n, T, H, G, D = c["seqs"], c["T"], c["H"], c["H_kv"], c["D"]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).float()         # [seqs, keys, H_kv, D]
    v = s["v_cache"][table].flatten(1, 2).float()
    q = s["q"].float().view(n, T, G, H // G, D)
    scores = torch.einsum("ntghd,nkgd->ngthk", q, k) * s["scale"]
    nodes = torch.full_like(s["lens"], T) if s["n_nodes"] is None else s["n_nodes"]
    first = s["lens"] - nodes                             # position of node 0
    node = torch.arange(k.shape[1], device=k.device) - first[:, None]     # [seqs, keys]
    # a node sees the whole prefix and the nodes of its word
    word = _bits(s["tree"], T).gather(2, node.clamp(0, T - 1)[:, None].expand(n, T, -1).long())
    seen = (node < 0)[:, None] | word & (node < nodes[:, None])[:, None]
    seen &= (torch.arange(T, device=k.device) < nodes[:, None])[..., None]  # [seqs, T, keys]
    scores = scores.masked_fill(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.einsum("ngthk,nkgd->ntghd", p, v)
    return {"out": out.reshape(n * T, H, D).to(s["out"].dtype)}


def _per_head(x, c):
    """Rows of H_qk heads as [seqs, T, H, D] in fp32: value head h reads head h mod H_qk."""
    return x.float().view(c["seqs"], c["T"], c["H_qk"], -1).repeat(1, 1, c["H"] // c["H_qk"], 1)


def _plain_delta(s):
    c = s["case"]
    n, T, H, Dk, Dv = c["seqs"], c["T"], c["H"], c["Dk"], c["Dv"]
    at, number = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    above = _bits(s["tree"], T) & (number < number[:, None])
    parent = (above * (number + 1)).amax(-1)              # 1 + the parent's number, 0: the root
    q, k = _per_head(s["q"], c), _per_head(s["k"], c)
    v = s["v"].float().view(n, T, H, Dv)
    beta = s["beta"].view(n, T, H, 1)
    decay = torch.exp(s["g"]).view(n, T, H, -1, 1)
    states = torch.empty(n, T + 1, H, Dk, Dv, device="cuda")
    states[:, 0] = s["state"]
    out, updates = torch.zeros(n, T, H, Dv, device="cuda"), torch.zeros(n, T, H, Dv, device="cuda")
    for t in range(T):                                    # a node needs its parent's state
        state = states[at, parent[:, t]] * decay[:, t]
        d = beta[:, t] * (v[:, t] - (state * k[:, t, :, :, None]).sum(-2))
        state += k[:, t, :, :, None] * d[:, :, None]
        states[:, t + 1] = state
        out[:, t] = s["scale"] * (state * q[:, t, :, :, None]).sum(-2)
        updates[:, t] = d
    if s["n_nodes"] is not None:
        absent = number >= s["n_nodes"][:, None]
        out[absent], updates[absent] = 0.0, 0.0
    return {"out": out.view(n * T, H, Dv), "updates": updates.view(n * T, H, Dv)}


def _plain_commit(s):
    c = s["case"]
    n, T, H, Dk, Dv = c["seqs"], c["T"], c["H"], c["Dk"], c["Dv"]
    leaf = s["leaf"].long()
    word = s["tree"].gather(1, leaf.clamp(0)[:, None])[:, 0]
    path = _bits(torch.where(leaf < 0, 0, word), T)       # [seqs, T]
    decay = torch.exp(s["g"]).view(n, T, H, -1)
    decay = torch.where(path[:, :, None, None], decay, 1.0)
    # what is left of node j's update at the leaf: the decays of the path behind it
    left = decay.flip(1).cumprod(1).flip(1)
    behind = torch.cat((left[:, 1:], torch.ones_like(left[:, :1])), 1)
    k = _per_head(s["k"], c) * behind * path[:, :, None, None]
    d = s["updates"].view(n, T, H, Dv)
    return {"state": s["state"] * left[:, 0, :, :, None] + torch.einsum("nthi,nthj->nhij", k, d)}


def _plain_sample(s):
    # in 64 bits: which token a number falls on depends on sums next to it
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    n, V = x.shape
    rank = torch.arange(V, device=x.device)
    temperature = s["temperature"].double()[:, None]
    greedy = temperature <= 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, temperature))
    kept = torch.where(greedy, rank < 1, True).expand(n, V)
    if s["min_p"] is not None:
        kept = kept & (w >= s["min_p"].double()[:, None])
    if s["top_k"] is not None:
        first = rank < s["top_k"][:, None]
        kept, w = kept & first, w * first
    if s["top_p"] is not None:
        before = w.cumsum(1) - w
        kept = kept & (before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True))
    kept = kept | (rank < 1)
    # by index again, and the first whose running mass passes the number's place
    mass = torch.zeros_like(w).scatter_(1, order, w * kept)
    run_ = mass.cumsum(1)
    total = run_[:, -1:]
    token = (run_ > s["uniform"].double()[:, None] * total).to(torch.uint8).argmax(1, keepdim=True)
    return {"tokens": token[:, 0].to(torch.int32),
            "probs": (mass.gather(1, token) / total)[:, 0].float()}


PLAIN = {"qknorm": _plain_qknorm, "attend": _plain_attend, "delta": _plain_delta,
         "commit": _plain_commit, "sample": _plain_sample}


# ---- the framework's calls ---------------------------------------------------

def _own_qknorm(s):
    from gated_delta_net_02_gb300 import gdn
    c = s["case"]
    if "plan" not in s:   # sizes alone: a program builds these once for its model
        dt = gdn.dtype_code(s["qkv"].dtype)
        wide = (c["H"] + 2 * c["H_kv"]) * c["D"]
        cache = gdn.gdn_kv_cache(s["k_cache"].shape[0], c["page"], c["H_kv"], c["D"], dt, 0, 0, 0)
        shape = gdn.gdn_rope_shape(
            c["tokens"], c["H"], c["rot"],
            gdn.GDN_ROPE_NEIGHBOURS if c["pairs"] else gdn.GDN_ROPE_HALVES, c["axes"],
            (gdn.c_int * 4)(*_sections(c)),
            gdn.GDN_ROPE_AXES_INTERLEAVED if c["interleaved"] else gdn.GDN_ROPE_AXES_SECTIONED,
            wide, wide, wide)
        s["plan"] = (shape, cache, gdn.gdn_qk_norm(s["eps"], c["offset"])) + _heads(s)
    shape, cache, norm, q, k, v = s["plan"]
    gdn.gdn_qknorm_rope_append(shape, cache, norm, q, k, v, s["q_weight"], s["k_weight"],
                               s["positions"], s["inv_freq"], s["slots"], s["q_out"],
                               s["k_cache"], s["v_cache"], torch.cuda.current_stream())
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    from gated_delta_net_02_gb300 import gdn
    c = s["case"]
    if "plan" not in s:   # sizes alone: a program builds these once for its model
        cache = gdn.gdn_kv_cache(s["k_cache"].shape[0], c["page"], c["H_kv"], c["D"],
                                 gdn.dtype_code(s["q"].dtype), 0, 0, 0)
        shape = gdn.gdn_attn_shape(c["seqs"], c["T"], c["H"], s["table"].shape[1], s["scale"],
                                   gdn.GDN_QK_GROUPED)
        nbytes = gdn.gdn_tree_attention_workspace_size(shape, cache)
        s["plan"] = shape, cache, torch.empty(nbytes, dtype=torch.uint8, device="cuda"), nbytes
    shape, cache, workspace, nbytes = s["plan"]
    gdn.gdn_tree_attention(shape, cache, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                           s["n_nodes"], s["tree"], s["out"], workspace, nbytes,
                           torch.cuda.current_stream())
    return {"out": s["out"]}


def _gdn_shape(gdn, c, scale):
    return gdn.gdn_shape(c["seqs"], c["T"], c["H"], c["Dk"], c["Dv"],
                         gdn.dtype_code(TYPES[c["dtype"]]), scale, c["H_qk"], gdn.GDN_QK_TILED)


def _own_delta(s):
    from gated_delta_net_02_gb300 import gdn
    c = s["case"]
    if "plan" not in s:
        s["plan"] = _gdn_shape(gdn, c, s["scale"])
    gdn.gdn_tree_forward(s["plan"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state_in"],
                         s["n_nodes"], s["tree"], s["out"], s["updates"],
                         "kda" if c["kda"] else "gda", torch.cuda.current_stream())
    return {"out": s["out"], "updates": s["updates"]}


def _own_commit(s):
    from gated_delta_net_02_gb300 import gdn
    c = s["case"]
    if "plan" not in s:
        s["plan"] = _gdn_shape(gdn, c, 0.0)
    gdn.gdn_tree_commit(s["plan"], s["k"], s["g"], s["updates"], s["state_in"], s["tree"],
                        s["leaf"], s["state_out"], "kda" if c["kda"] else "gda",
                        torch.cuda.current_stream())
    return {"state": s["state_out"]}


def _own_sample(s):
    from gated_delta_net_02_gb300 import gdn
    c = s["case"]
    if "plan" not in s:
        s["plan"] = gdn.gdn_sample_shape(c["rows"], c["vocab"], gdn.dtype_code(s["logits"].dtype), 0)
    gdn.gdn_sample(s["plan"], s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                   s["uniform"], s["tokens"], s["probs"], torch.cuda.current_stream())
    return {"tokens": s["tokens"], "probs": s["probs"]}


OWN = {"qknorm": _own_qknorm, "attend": _own_attend, "delta": _own_delta, "commit": _own_commit,
       "sample": _own_sample}


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def _exact_qknorm(s):
    c = s["case"]
    angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i].double()
                         for i, a in enumerate(_axis_of_freq(c))], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]     # [tokens, 1, rot/2]

    def rotated(x, weight):
        x = x.double()
        rms = torch.sqrt((x ** 2).sum(-1) / c["D"] + s["eps"])
        x = x / rms[..., None] * (weight.double() + c["offset"])
        half = c["rot"] // 2
        at = torch.arange(half, device=x.device)
        first, second = (2 * at, 2 * at + 1) if c["pairs"] else (at, at + half)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = _heads(s)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    k_cache[page, at] = rotated(k, s["k_weight"])
    v_cache[page, at] = v.double()
    return {"q": rotated(q, s["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attend(s):
    c = s["case"]
    n, T, H, G, D = c["seqs"], c["T"], c["H"], c["H_kv"], c["D"]
    if 4 * T * H * D * sum(_lengths(c)) > 4e12:
        return None
    out = torch.zeros(n, T, H, D, dtype=torch.float64, device="cuda")
    nodes = [T] * n if s["n_nodes"] is None else s["n_nodes"].tolist()
    for i, (length, m) in enumerate(zip(s["lens"].tolist(), nodes)):
        if m == 0:
            continue
        pages = s["table"][i, :-(-length // c["page"])].long()
        k = s["k_cache"][pages].reshape(-1, G, D)[:length].double()
        v = s["v_cache"][pages].reshape(-1, G, D)[:length].double()
        hidden = torch.zeros(m, length, dtype=torch.bool, device="cuda")
        hidden[:, length - m:] = ~_bits(s["tree"][i, :m], m)
        for g in range(G):
            q = s["q"][i * T:i * T + m, g * (H // G):(g + 1) * (H // G)].double()
            x = (s["scale"] * q @ k[:, g].T).masked_fill(hidden[:, None], -math.inf)
            out[i, :m, g * (H // G):(g + 1) * (H // G)] = torch.softmax(x, -1) @ v[:, g]
    return {"out": out.view(n * T, H, D)}


def _exact_delta(s):
    """Without any state but the first: the updates solve a triangular system."""
    c = s["case"]
    n, T, H, Dk, Dv = c["seqs"], c["T"], c["H"], c["Dk"], c["Dv"]
    head = torch.arange(H, device="cuda") % c["H_qk"]
    out = torch.zeros(n, T, H, Dv, dtype=torch.float64, device="cuda")
    updates = torch.zeros_like(out)
    eye = torch.eye(T, dtype=torch.float64, device="cuda")
    for i in range(n):
        rows = slice(i * T, (i + 1) * T)
        q, k = (s[x][rows][:, head].double().transpose(0, 1) for x in ("q", "k"))    # [H, T, Dk]
        v = s["v"][rows].double().transpose(0, 1)
        beta = s["beta"][rows].double().T[..., None]
        line = _bits(s["tree"][i], T)
        g = s["g"][rows].double().reshape(T, H, -1)
        gamma = torch.einsum("tj,jhi->hti", line.double(), g)                        # along the path
        between = torch.exp((gamma[:, :, None] - gamma[:, None]).masked_fill(
            ~line[None, :, :, None], -math.inf))                                     # [H, T, T, Dk|1]
        kk = (k[:, :, None] * k[:, None] * between).sum(-1)
        qk = (q[:, :, None] * k[:, None] * between).sum(-1)
        state = s["state"][i].double()
        from_state = torch.exp(gamma)
        rhs = beta * (v - (k * from_state) @ state)
        d = torch.linalg.solve_triangular(eye + beta * kk * (1 - eye), rhs, upper=False)
        o = s["scale"] * ((q * from_state) @ state + qk @ d)
        out[i], updates[i] = o.transpose(0, 1), d.transpose(0, 1)
    if s["n_nodes"] is not None:
        for i, m in enumerate(s["n_nodes"].tolist()):
            out[i, m:] = updates[i, m:] = 0
    return {"out": out.view(n * T, H, Dv), "updates": updates.view(n * T, H, Dv)}


def _exact_commit(s):
    c = s["case"]
    n, T, H, Dk, Dv = c["seqs"], c["T"], c["H"], c["Dk"], c["Dv"]
    head = torch.arange(H, device="cuda") % c["H_qk"]
    state = s["state"].double()
    g = s["g"].double().view(n, T, H, -1, 1)
    k = s["k"].view(n, T, -1, Dk)[:, :, head].double()
    d = s["updates"].view(n, T, H, Dv).double()
    leaf, words = s["leaf"].tolist(), s["tree"].tolist()
    for i in range(n):
        for t in range(T):
            if leaf[i] >= 0 and words[i][leaf[i]] >> t & 1:
                state[i] = torch.exp(g[i, t]) * state[i] + k[i, t, :, :, None] * d[i, t, :, None]
    return {"state": state}


def _exact_sample(s):
    n, V = s["logits"].shape
    tokens, probs = [], []
    for i in range(n):
        x = s["logits"][i].double()
        temperature = float(s["temperature"][i])
        top = x.max()
        if temperature <= 0:
            tokens.append(int((x == top).nonzero()[0]))
            probs.append(1.0)
            continue
        index = torch.argsort(x, descending=True, stable=True)
        if s["top_k"] is not None:
            index = index[:int(s["top_k"][i])]
        w = torch.exp((x[index] - top) / temperature)
        count = len(index)
        if s["top_p"] is not None:
            reach = w.cumsum(0) >= float(s["top_p"][i]) * w.sum()
            if bool(reach.any()):
                count = int(reach.nonzero()[0]) + 1
        if s["min_p"] is not None:
            count = min(count, max(1, int((w >= float(s["min_p"][i])).sum())))
        kept = index[:count].sort().values
        w = torch.exp((x[kept] - top) / temperature)
        run_ = w.cumsum(0)
        past = (run_ > float(s["uniform"][i]) * run_[-1]).nonzero()
        at = int(past[0]) if len(past) else count - 1
        tokens.append(int(kept[at]))
        probs.append(float(w[at] / run_[-1]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32),
            "probs": torch.tensor(probs, dtype=torch.float64)}


EXACT = {"qknorm": _exact_qknorm, "attend": _exact_attend, "delta": _exact_delta,
         "commit": _exact_commit, "sample": _exact_sample}
