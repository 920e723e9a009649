"""A small hybrid stack served with this package: two gated delta-rule layers and one softmax-attention layer.

Two sequences of different length are prefilled in chunks, one of them branches, all three decode a few tokens, one ends,
and the cache is compacted while the others go on.  Every operator of the package takes part: the delta rule (chunked for
the prefill, recurrent for single tokens), the residual root-mean-square norm, rotary positions written straight into the
paged cache, attention over that cache, and the upkeep of its pages.

    python examples/hybrid.py

prints how far the logits of every decoded token are from those of a dense fp32 computation of the same model that keeps no
cache and recomputes each sequence from its first token.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_15_gb300 as g  # noqa: E402

H, HKV, D, VOCAB, PAGE = 4, 2, 128, 256, 16
WIDTH = H * D
LAYERS = ("delta", "delta", "attention")


def weights(device, seed=0):
    """Random weights, bf16 for the projections and fp32 for norms and gates."""
    gen = torch.Generator().manual_seed(seed)

    def mat(rows, cols):
        return (torch.randn(rows, cols, generator=gen) / math.sqrt(rows)).to(device, torch.bfloat16)

    w = dict(embed=torch.randn(VOCAB, WIDTH, generator=gen).to(device, torch.bfloat16), head=mat(WIDTH, VOCAB),
             norm=torch.ones(WIDTH, device=device), layers=[])
    for kind in LAYERS:
        heads = 3 * H if kind == "delta" else H + 2 * HKV
        w["layers"].append(dict(kind=kind, norm=(1 + 0.1 * torch.randn(WIDTH, generator=gen)).to(device),
                                qkv=mat(WIDTH, heads * D), out=mat(WIDTH, WIDTH), gates=mat(WIDTH, 2 * H)))
    return w


def gates(x, layer):
    """(log-gate, beta) of every token and head."""
    a, b = (x @ layer["gates"]).float().split(H, -1)
    return -torch.nn.functional.softplus(a - 2.0), torch.sigmoid(b)


class Server:
    """Slots for `slots` sequences: one page table for the attention layer's cache, one state per delta-rule layer."""

    def __init__(self, w, slots=8, pages=64, width=16, device="cuda"):
        self.w, self.slots, self.device = w, slots, device
        self.page_table = torch.full((slots, width), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(slots, dtype=torch.int32, device=device)
        self.refcount = torch.zeros(pages, dtype=torch.int32, device=device)
        self.k_cache = torch.zeros(pages, PAGE, HKV, D, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.states = [torch.zeros(slots, H, D, D, device=device) for kind in LAYERS if kind == "delta"]
        self.angles = g.rotary_table(width * PAGE, D, device=device)

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.device)

    def step(self, slots, tokens):
        """The next `tokens` (a list of as many for each of `slots`) through the stack; logits of every last token."""
        n, t = len(slots), len(tokens[0])
        ids, idx = torch.tensor(tokens, device=self.device), torch.tensor(slots, device=self.device)
        assert g.extend_pages(self.page_table, self.seq_lens, self.refcount, self.ints(slots), self.ints([t] * n), PAGE).all()
        table, lens = self.page_table[idx], self.seq_lens[idx]
        residual, x = None, self.w["embed"][ids].view(n * t, WIDTH)
        state = iter(self.states)
        for layer in self.w["layers"]:
            normed = g.rms_norm(x, layer["norm"], residual)
            residual, y = normed.h, normed.y
            qkv = y @ layer["qkv"]
            if layer["kind"] == "delta":
                q, k, v = (u.contiguous() for u in qkv.view(n, t, 3, H, D).unbind(2))
                gate, beta = (u.view(n, t, H).contiguous() for u in gates(y, layer))
                s = next(state)
                if t == 1:
                    o, new = g.recurrent_gated_delta_rule(q, k, v, gate, beta, s[idx], use_qk_l2norm_in_kernel=True)
                else:
                    o, new = g.chunk_gated_delta_rule_fwd(q, k, v, gate, beta, s[idx], use_qk_l2norm_in_kernel=True)
                s[idx] = new
            else:
                q, k, v = qkv.view(n * t, H + 2 * HKV, D).split([H, HKV, HKV], 1)
                q = g.rotary_append(q, k, v, self.angles, self.k_cache, self.v_cache, table, lens)
                o = g.paged_attention(q, self.k_cache, self.v_cache, table, lens, max_q=t)
            x = o.reshape(n * t, WIDTH) @ layer["out"]
        y = g.rms_norm(x, self.w["norm"], residual).y
        return (y.view(n, t, WIDTH)[:, -1] @ self.w["head"]).float()

    def fork(self, parents, children):
        new = g.fork_pages(self.page_table, self.seq_lens, self.refcount, self.ints(parents), self.ints(children),
                           [self.k_cache, self.v_cache], PAGE, self.states)
        assert (new != -2).all()

    def end(self, slots):
        g.free_pages(self.page_table, self.seq_lens, self.refcount, self.ints(slots))
        for s in self.states:
            s[torch.tensor(slots, device=self.device)] = 0

    def compact(self):
        return int(g.compact_pages(self.page_table, self.refcount, [self.k_cache, self.v_cache])[2])


def dense(w, tokens):
    """Logits after the last of `tokens`, in fp32 without a cache: the delta rule token by token, full attention."""
    f = torch.float32
    x = w["embed"][torch.tensor(tokens, device=w["norm"].device)].to(f)
    t = x.shape[0]

    def norm(x, weight):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight

    for layer in w["layers"]:
        y = norm(x, layer["norm"])
        qkv = y @ layer["qkv"].to(f)
        if layer["kind"] == "delta":
            q, k, v = qkv.view(t, 3, H, D).unbind(1)
            q, k = (u * torch.rsqrt(u.square().sum(-1, keepdim=True) + 1e-6) for u in (q, k))
            a, b = (y @ layer["gates"].to(f)).split(H, -1)
            alpha, beta = (-torch.nn.functional.softplus(a - 2.0)).exp(), torch.sigmoid(b)
            s, out = torch.zeros(H, D, D, device=x.device), []
            for i in range(t):
                s = alpha[i, :, None, None] * s
                u = beta[i, :, None] * (v[i] - torch.einsum("hvk,hk->hv", s, k[i]))
                s = s + u[..., None] * k[i][:, None]
                out.append(torch.einsum("hvk,hk->hv", s, q[i]) / math.sqrt(D))
            o = torch.stack(out)
        else:
            q, k, v = qkv.view(t, H + 2 * HKV, D).split([H, HKV, HKV], 1)
            freq, _ = g.rotary_frequencies(D)
            angle = (torch.arange(t, dtype=torch.float64)[:, None] * freq).to(x.device)
            c, s = angle.cos().to(f)[:, None], angle.sin().to(f)[:, None]

            def turn(u):
                lo, hi = u.chunk(2, -1)
                return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)

            q, k, v = turn(q), turn(k).repeat_interleave(H // HKV, 1), v.repeat_interleave(H // HKV, 1)
            z = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
            z = z.masked_fill(torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1), -math.inf)
            o = torch.einsum("hij,jhd->ihd", z.softmax(-1), v)
        x = x + o.reshape(t, WIDTH) @ layer["out"].to(f)
    return norm(x[-1:], w["norm"]) @ w["head"].to(f)


def main(device="cuda", quiet=False):
    w = weights(device)
    server = Server(w, device=device)
    gen = torch.Generator().manual_seed(1)

    def draw(n):
        return torch.randint(0, VOCAB, (n,), generator=gen).tolist()

    history, worst = {}, 0.0

    def step(slots, tokens):
        nonlocal worst
        logits = server.step(slots, tokens)
        for slot, more, got in zip(slots, tokens, logits):
            history[slot] = history.get(slot, []) + more
            want = dense(w, history[slot])[0]
            err = float((got - want).norm() / want.norm())
            worst = max(worst, err)
            if not quiet:
                print(f"slot {slot}, {len(history[slot]):3d} tokens: logits off by {err:.4f} of their norm")

    step([0], [draw(70)])                       # a prompt in two chunks, the second over the cached first
    step([0], [draw(21)])
    step([5], [draw(33)])
    step([0, 5], [draw(1), draw(1)])            # both decode
    server.fork([0], [3])                       # the first branches: full pages shared, the last one and the states copied
    history[3] = list(history[0])
    for _ in range(3):
        step([0, 3, 5], [draw(1) for _ in range(3)])
    server.end([0])                             # its pages go back, those shared with the branch stay
    moved = server.compact()
    if not quiet:
        print(f"compacted: {moved} pages moved")
    for _ in range(2):
        step([3, 5], [draw(1) for _ in range(2)])
    if not quiet:
        print(f"worst {worst:.4f}")
    return worst


if __name__ == "__main__":
    main()
