"""A small stack with a gated linear recurrence and two softmax-attention layers: many branches of one prompt, and training.

A prompt is prefilled in two chunks, branches into 32 sequences, and all of them decode a few tokens.  The layers are a gated
linear recurrence with one state per channel, attention over a window with the first tokens kept visible, and attention
over everything.  The heads of both attention layers are normed and turned on their way into the paged cache; the branches
read the prompt's keys of the last layer once for all of them.  The same stack then takes a training step's gradients.

    python examples/branches.py

prints how far logits and gradients are from those of a dense fp32 computation of the same model.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_15_gb300 as g  # noqa: E402

H, HKV, D, VOCAB, PAGE = 4, 2, 128, 256, 16
WIDTH, WINDOW, SINKS = H * D, 40, 5
LAYERS = ("scan", "window", "full")
BRANCHES, PAGES_EACH = 32, 260


def weights(device, seed=0):
    """Random weights, bf16 for the projections and fp32 for norms."""
    gen = torch.Generator().manual_seed(seed)

    def mat(rows, cols):
        return (torch.randn(rows, cols, generator=gen) / math.sqrt(rows)).to(device, torch.bfloat16)

    def ones(n):
        return (1 + 0.1 * torch.randn(n, generator=gen)).to(device)

    w = dict(embed=torch.randn(VOCAB, WIDTH, generator=gen).to(device, torch.bfloat16), head=mat(WIDTH, VOCAB), norm=ones(WIDTH))
    for i, kind in enumerate(LAYERS):
        w[f"norm{i}"] = ones(WIDTH)
        w[f"in{i}"] = mat(WIDTH, 3 * WIDTH if kind == "scan" else (H + 2 * HKV) * D)
        w[f"out{i}"] = mat(WIDTH, WIDTH)
        if kind != "scan":
            w[f"q{i}"], w[f"k{i}"] = ones(D), ones(D)
    return w


def log_gate(a):
    return -torch.nn.functional.softplus(a.float() - 2.0)


def mask(t, kind, device):
    """Keys [.., j] that query i does not see."""
    i, j = torch.arange(t, device=device)[:, None], torch.arange(t, device=device)[None]
    hidden = j > i
    return hidden | ((j <= i - WINDOW) & (j >= SINKS)) if kind == "window" else hidden


def attend(q, k, v, kind):
    """Attention of whole sequences [n, t, heads, D], in fp32."""
    q, k, v = q.float(), k.float().repeat_interleave(H // HKV, 2), v.float().repeat_interleave(H // HKV, 2)
    z = torch.einsum("nihd,njhd->nhij", q, k) / math.sqrt(D)
    p = z.masked_fill(mask(q.shape[1], kind, q.device), -math.inf).softmax(-1)
    return torch.einsum("nhij,njhd->nihd", p, v)


class Server:
    """Slots for `slots` sequences: one page table for the attention layers' caches, one state for the recurrence."""

    def __init__(self, w, slots=1 + BRANCHES, pages=256, device="cuda"):
        self.w, self.device = w, device
        self.page_table = torch.full((slots, PAGES_EACH), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(slots, dtype=torch.int32, device=device)
        self.refcount = torch.zeros(pages, dtype=torch.int32, device=device)
        self.caches = [torch.zeros(pages, PAGE, HKV, D, dtype=torch.bfloat16, device=device) for _ in range(4)]
        self.state = torch.zeros(slots, WIDTH, device=device)
        self.angles = g.rotary_table(PAGES_EACH * PAGE, D, device=device)

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.device)

    def grow(self, slots, tokens):
        ok = g.extend_pages(self.page_table, self.seq_lens, self.refcount, self.ints(slots), self.ints([tokens] * len(slots)), PAGE)
        assert ok.all()

    def forward(self, rows, ids, prefix=None):
        """The tokens ids [n, t] of the slots `rows`, for which there is room already; logits of every last token.  prefix
        int32 [1]: tokens that all of them have in common.  Everything is on the device, so that a graph can hold it."""
        w, (n, t) = self.w, ids.shape
        table, lens = self.page_table[rows], self.seq_lens[rows]
        caches = iter(self.caches)
        residual, x = None, w["embed"][ids].view(n * t, WIDTH)
        for i, kind in enumerate(LAYERS):
            normed = g.rms_norm(x, w[f"norm{i}"], residual)
            residual, y = normed.h, normed.y @ w[f"in{i}"]
            if kind == "scan":
                u, a, z = (p.contiguous() for p in y.view(n, t, 3, WIDTH).unbind(2))
                if t == 1:
                    s = self.state[rows]
                    o, s = g.gated_scan_step(u[:, 0], log_gate(a[:, 0]), s)
                else:
                    o, s = g.gated_scan(u, log_gate(a), self.state[rows])
                self.state[rows] = s
                o = o.view(n, t, WIDTH) * torch.sigmoid(z)
            else:
                q, k, v = y.view(n * t, H + 2 * HKV, D).split([H, HKV, HKV], 1)
                kc, vc = next(caches), next(caches)
                q = g.norm_rotary_append(q, k, v, w[f"q{i}"], w[f"k{i}"], self.angles, kc, vc, table, lens)
                if kind == "window":
                    o = g.paged_attention(q, kc, vc, table, lens, max_q=t, window=WINDOW, sinks=SINKS)
                elif prefix is None:
                    o = g.paged_attention(q, kc, vc, table, lens, max_q=t)
                else:
                    o = g.prefix_attention(q, kc, vc, table, lens, prefix, max_q=t, max_group=n * t)
            x = o.reshape(n * t, WIDTH) @ w[f"out{i}"]
        y = g.rms_norm(x, w["norm"], residual).y
        return (y.view(n, t, WIDTH)[:, -1] @ w["head"]).float()

    def step(self, slots, tokens, prefix=None):
        self.grow(slots, len(tokens[0]))
        rows, ids = torch.tensor(slots, device=self.device), torch.tensor(tokens, device=self.device)
        return self.forward(rows, ids, None if prefix is None else self.ints([prefix]))

    def fork(self, parent, children):
        new = g.fork_pages(self.page_table, self.seq_lens, self.refcount, self.ints([parent] * len(children)), self.ints(children),
                           self.caches, PAGE, [self.state])
        assert (new != -2).all()


def train(w, ids):
    """Logits of every token of ids [n, t], with a graph: the operators that have gradients."""
    n, t = ids.shape
    angles = g.rotary_table(t, D, device=ids.device)
    positions = torch.arange(t, dtype=torch.int32, device=ids.device).repeat(n)
    x, h = w["embed"][ids].view(n * t, WIDTH), None
    for i, kind in enumerate(LAYERS):
        if h is None:
            h, y = x, g.residual_rms_norm(x, w[f"norm{i}"])
        else:
            y, h = g.residual_rms_norm(x, w[f"norm{i}"], h)
        y = y @ w[f"in{i}"]
        if kind == "scan":
            u, a, z = (p.contiguous() for p in y.view(n, t, 3, WIDTH).unbind(2))
            o = g.gated_linear_recurrence(u, log_gate(a))[0] * torch.sigmoid(z)
        else:
            q, k, v = y.view(n * t, H + 2 * HKV, D).split([H, HKV, HKV], 1)
            q, k = g.norm_rotary_embedding(q, k, w[f"q{i}"], w[f"k{i}"], angles, positions)
            o = attend(*(p.reshape(n, t, -1, D) for p in (q, k, v)), kind).to(torch.bfloat16)
        x = o.reshape(n * t, WIDTH) @ w[f"out{i}"]
    return (g.residual_rms_norm(x, w["norm"], h)[0] @ w["head"]).view(n, t, VOCAB).float()


def dense(w, ids):
    """The same in fp32 without any of the package's operators: the recurrence token by token."""
    f, (n, t) = torch.float32, ids.shape
    w = {name: p.to(f) for name, p in w.items()}
    x = w["embed"][ids]

    def norm(x, weight):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight

    freq, _ = g.rotary_frequencies(D)
    angle = (torch.arange(t, dtype=torch.float64)[:, None] * freq).to(x.device)
    c, s = angle.cos().to(f)[:, None], angle.sin().to(f)[:, None]

    def turn(u):
        lo, hi = u.chunk(2, -1)
        return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)

    for i, kind in enumerate(LAYERS):
        y = norm(x, w[f"norm{i}"]) @ w[f"in{i}"]
        if kind == "scan":
            u, a, z = y.view(n, t, 3, WIDTH).unbind(2)
            gate, state, out = log_gate(a).exp(), 0, []
            for j in range(t):
                state = gate[:, j] * state + u[:, j]
                out.append(state)
            o = torch.stack(out, 1) * torch.sigmoid(z)
        else:
            q, k, v = y.view(n, t, H + 2 * HKV, D).split([H, HKV, HKV], 2)
            o = attend(turn(norm(q, w[f"q{i}"])), turn(norm(k, w[f"k{i}"])), v, kind)
        x = x + o.reshape(n, t, WIDTH) @ w[f"out{i}"]
    return norm(x, w["norm"]) @ w["head"]


def off(got, want):
    return float((got.float() - want.float()).norm() / want.float().norm())


def serve(device="cuda", quiet=False):
    """How far the logits of a served prompt and its branches are from the dense ones, at worst."""
    w = weights(device)
    server = Server(w, device=device)
    gen = torch.Generator().manual_seed(1)

    def draw(n, t):
        return torch.randint(0, VOCAB, (n, t), generator=gen).tolist()

    def check(slots, logits):
        want = dense(w, torch.tensor([history[s] for s in slots], device=device))[:, -1]
        errs = [off(a, b) for a, b in zip(logits, want)]
        if not quiet:
            print(f"{len(slots)} sequences of {len(history[slots[0]])} tokens: logits off by at most {max(errs):.4f} of their norm")
        return max(errs)

    history, worst = {0: []}, 0.0
    for t in (70, 51):  # the prompt in two chunks, the second over the cached first
        more = draw(1, t)
        history[0] += more[0]
        worst = max(worst, check([0], server.step([0], more)))
    prompt, branches = len(history[0]), list(range(1, 1 + BRANCHES))
    server.fork(0, branches)  # full pages shared, the last one and the states copied
    for b in branches:
        history[b] = list(history[0])
    for _ in range(4):
        more = draw(BRANCHES, 1)
        for b, m in zip(branches, more):
            history[b] += m
        # what the branches share: the prompt's full pages
        worst = max(worst, check(branches, server.step(branches, more, prefix=prompt // PAGE * PAGE)))
    return worst


def gradients(device="cuda", quiet=False):
    """How far a training step's gradients are from the dense ones: {weight: distance}."""
    w = {name: p.requires_grad_() for name, p in weights(device).items()}
    gen = torch.Generator().manual_seed(2)
    ids = torch.randint(0, VOCAB, (3, 77), generator=gen).to(device)
    d_logits = torch.randn(3, 77, VOCAB, generator=gen).to(device)
    got = torch.autograd.grad(train(w, ids), list(w.values()), d_logits)
    want = torch.autograd.grad(dense(w, ids), list(w.values()), d_logits)
    errs = {name: off(a, b) for name, a, b in zip(w, got, want)}
    if not quiet:
        for name, e in errs.items():
            print(f"gradient of {name:6s} off by {e:.4f} of its norm")
    return errs


if __name__ == "__main__":
    serve()
    gradients()
