"""One full-attention layer of a hybrid model, decoded with libgdn's calls.

Models that run the gated delta-net recurrence in most layers attend to the
whole context every few layers. This program runs such a layer for a batch of
sequences: the prompts' keys and values go into a paged cache, then every step
takes T new tokens of each sequence (T = 1 decodes; T = draft + 1 verifies)
through

    h, x8   = gdn_rmsnorm_fp8(x + h)             residual stream, 8-bit input
    qkv     = gdn_gemm_fp8(x8, W_qkv)
    q, K, V = gdn_rope_append(qkv)               rotate q, k; append k, v
    o       = gdn_paged_attention(q, K, V)
    o8      = gdn_rmsnorm_fp8(o, normalize=0)    8-bit input of the projection
    x       = gdn_gemm_fp8(o8, W_out)

    python examples/attention_layer.py [--seqs 8] [--tokens 1] [--steps 4] [--check]

--check compares every step with the same layer in 64 bits (weights as the
8-bit values they are, activations not rounded).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

E4M3 = torch.float8_e4m3fn


def quantise_weight(w):
    """e4m3 values and one scale for each 128 x 128 block of w [N, K] (both
    multiples of 128): done once, when the weights are loaded."""
    N, K = w.shape
    blocks = w.float().view(N // 128, 128, K // 128, 128)
    scale = blocks.abs().amax((1, 3)).clamp_min(2.0 ** -100) / 448
    q = (blocks / scale[:, None, :, None]).view(N, K).to(E4M3)
    return q, scale.contiguous()


class AttentionLayer:
    """Weights, cache and buffers of one layer for a fixed batch of sequences."""

    def __init__(self, seqs, tokens, max_len, H=16, H_kv=2, D=128, hidden=2048, page=16,
                 eps=1e-6, seed=0, prompt_tokens=0):
        from gated_delta_net_02_gb300 import gdn
        self.gdn = gdn
        self.N, self.T, self.H, self.H_kv, self.D, self.hidden = seqs, tokens, H, H_kv, D, hidden
        self.eps, self.page = eps, page
        self.wide = (H + 2 * H_kv) * D
        gen = torch.Generator("cuda")
        gen.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.norm_w = (1 + 0.1 * randn(hidden)).bfloat16()
        self.w_qkv, self.s_qkv = quantise_weight(randn(self.wide, hidden) / hidden ** 0.5)
        self.w_out, self.s_out = quantise_weight(randn(hidden, H * D) / (H * D) ** 0.5)
        half = D // 2
        self.inv_freq = (1e4 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        # three position axes (time, height, width); text has the same in all
        self.sections = (half - 2 * (half // 4), half // 4, half // 4)

        # the cache: every sequence owns max_len / page pages, in any order
        per = -(-max_len // page)
        self.table = torch.randperm(seqs * per, generator=gen, device="cuda").to(
            torch.int32).view(seqs, per).contiguous()
        self.k_cache = torch.zeros(seqs * per, page, H_kv, D, device="cuda", dtype=torch.bfloat16)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.lens = torch.zeros(seqs, device="cuda", dtype=torch.int32)
        self.cache = gdn.gdn_kv_cache(seqs * per, page, H_kv, D, gdn.GDN_BF16, 0, 0, 0)
        self.attn = gdn.gdn_attn_shape(seqs, tokens, H, per, 0.0, gdn.GDN_QK_GROUPED)
        self.ws_bytes = gdn.gdn_paged_attention_workspace_size(self.attn, self.cache)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, device="cuda", dtype=dtype)

        n = max(seqs * tokens, prompt_tokens)
        self.x8, self.xs = buf(n, hidden, dtype=E4M3), buf(n, hidden // 128, dtype=torch.float32)
        self.qkv, self.q = buf(n, self.wide), buf(n, H, D)
        self.o = buf(n, H, D)
        self.o8, self.os = buf(n, H * D, dtype=E4M3), buf(n, H * D // 128, dtype=torch.float32)

    def project(self, x, h, positions, slots):
        """Norm, q/k/v projection, rotation and append of n tokens. h, the
        residual stream, is updated in place."""
        g, n = self.gdn, x.shape[0]
        st = torch.cuda.current_stream()
        g.gdn_rmsnorm_fp8(g.gdn_norm_shape(n, self.hidden, g.GDN_BF16, 1, self.eps, 0.0), x, h,
                          self.norm_w, h, None, self.x8[:n], self.xs[:n], st)
        g.gdn_gemm_fp8(g.gdn_gemm_shape(n, self.wide, self.hidden, g.GDN_BF16), self.x8[:n],
                       self.xs[:n], self.w_qkv, self.s_qkv, self.qkv[:n], st)
        H, G, D = self.H, self.H_kv, self.D
        qkv = self.qkv[:n]
        q = qkv[:, :H * D].unflatten(1, (H, D))
        k = qkv[:, H * D:(H + G) * D].unflatten(1, (G, D))
        v = qkv[:, (H + G) * D:].unflatten(1, (G, D))
        shape = g.gdn_rope_shape(n, H, D, g.GDN_ROPE_HALVES, 3, (g.c_int * 4)(*self.sections),
                                 g.GDN_ROPE_AXES_INTERLEAVED, self.wide, self.wide, self.wide)
        g.gdn_rope_append(shape, self.cache, q, k, v, positions, self.inv_freq, slots, self.q[:n],
                          self.k_cache, self.v_cache, st)

    def place(self, seq, pos):
        """Cache slots and positions [3, n] of tokens `pos` of sequences `seq`."""
        page = self.table[seq, pos // self.page].long()
        slots = page * self.page + pos % self.page
        return pos.to(torch.int32).expand(3, -1).contiguous(), slots.contiguous()

    def append_prompt(self, seq, x, h):
        """The keys and values of a prompt's tokens x [n, hidden] of one sequence."""
        pos = torch.arange(x.shape[0], device="cuda")
        self.project(x, h, *self.place(torch.full_like(pos, seq), pos))
        self.lens[seq] = x.shape[0]

    def step(self, x, h):
        """T new tokens of each sequence: x [N*T, hidden] and the residual
        stream h (updated in place). Returns the layer's output [N*T, hidden]."""
        g, N, T = self.gdn, self.N, self.T
        st = torch.cuda.current_stream()
        pos = (self.lens[:, None] + torch.arange(T, device="cuda")).reshape(-1).long()
        seq = torch.arange(N, device="cuda").repeat_interleave(T)
        self.project(x, h, *self.place(seq, pos))
        self.lens += T
        n, hd = N * T, self.H * self.D
        g.gdn_paged_attention(self.attn, self.cache, self.q[:n], self.k_cache, self.v_cache,
                              self.table, self.lens, self.o[:n], self.ws, self.ws_bytes, st)
        g.gdn_rmsnorm_fp8(g.gdn_norm_shape(n, hd, g.GDN_BF16, 0, 0.0, 0.0), self.o[:n].view(n, hd),
                          None, None, None, None, self.o8[:n], self.os[:n], st)
        out = torch.empty(n, self.hidden, device="cuda", dtype=torch.bfloat16)
        g.gdn_gemm_fp8(g.gdn_gemm_shape(n, self.hidden, hd, g.GDN_BF16), self.o8[:n], self.os[:n],
                       self.w_out, self.s_out, out, st)
        return out


class Reference:
    """The same layer in 64 bits, keys and values kept densely."""

    def __init__(self, layer):
        L = self.L = layer

        def weight(q, s):
            return q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)

        self.w_qkv, self.w_out = weight(L.w_qkv, L.s_qkv), weight(L.w_out, L.s_out)
        self.k = [[] for _ in range(L.N)]
        self.v = [[] for _ in range(L.N)]

    def token(self, seq, x, h):
        """(q, new h) of one token, its key and value appended."""
        L = self.L
        h = h.double() + x.double()
        y = h / torch.sqrt((h * h).mean() + L.eps) * L.norm_w.double()
        qkv = (self.w_qkv @ y).view(-1, L.D)
        ang = len(self.k[seq]) * L.inv_freq.double()
        half = L.D // 2

        def turn(t):
            a, b = t[:, :half], t[:, half:]
            return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), 1)

        self.k[seq].append(turn(qkv[L.H:L.H + L.H_kv]))
        self.v[seq].append(qkv[L.H + L.H_kv:])
        return turn(qkv[:L.H])

    def out(self, seq, q):
        L = self.L
        G = L.H // L.H_kv
        k = torch.stack(self.k[seq], 1).repeat_interleave(G, 0)
        v = torch.stack(self.v[seq], 1).repeat_interleave(G, 0)
        p = torch.softmax(torch.einsum("hd,hkd->hk", q, k) * L.D ** -0.5, -1)
        return self.w_out @ torch.einsum("hk,hkd->hd", p, v).reshape(-1)


def run(seqs=8, tokens=1, steps=4, prompt=40, check=False, seed=0):
    """Runs the layer; returns the largest relative error of a step (or None)."""
    prompts = [prompt + 7 * s for s in range(seqs)]
    layer = AttentionLayer(seqs, tokens, max(prompts) + steps * tokens, seed=seed,
                           prompt_tokens=max(prompts))
    ref = Reference(layer) if check else None
    gen = torch.Generator("cuda")
    gen.manual_seed(seed + 1)

    def stream(n):
        return torch.randn(n, layer.hidden, generator=gen, device="cuda").bfloat16()

    for s, n in enumerate(prompts):
        x, h = stream(n), stream(n)
        if check:
            for i in range(n):
                ref.token(s, x[i], h[i])
        layer.append_prompt(s, x, h)
    worst = 0.0
    for _ in range(steps):
        x, h = stream(seqs * tokens), stream(seqs * tokens)
        want = []
        if check:
            for i in range(seqs * tokens):
                s = i // tokens
                want.append(ref.out(s, ref.token(s, x[i], h[i])))
        got = layer.step(x, h)
        layer.gdn.gdn_check_device_error()
        if check:
            w = torch.stack(want)
            worst = max(worst, float((got.double() - w).norm() / w.norm()))
    return worst if check else None


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=40)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    err = run(a.seqs, a.tokens, a.steps, a.prompt, a.check)
    torch.cuda.synchronize()
    print(f"{a.steps} steps of {a.seqs} x {a.tokens} tokens" +
          (f", rel-L2 error {err:.3f} against 64 bits" if a.check else ""))


if __name__ == "__main__":
    main()
