"""More operators of a hybrid stack, as measurable cases: a gated linear recurrence, the norm of each query and key head with
the position rotation, attention with a sliding window and first tokens that stay visible, and attention of sequences that
share a prefix.

Next to delta-rule layers a stack may carry layers whose state is a vector: ``scan``, h_t = exp(g_t) h_{t-1} + x_t in every
channel, forward, backward and by single tokens.  Its softmax layers often norm each head of q and k before the rotation
(``qknorm``: with gradients, or written into the paged cache), limit long contexts to a window that keeps the first tokens
(``sinks``), and serve many continuations of one prompt, whose cache pages they share (``prefix``).

``listed()`` names the cases, ``draw(rng)`` gives others of the same ranges, ``prepare`` makes what a program has in hand
before the call, ``run`` makes one pass: with ``own`` through this package, without it in elementary torch operations in 32
bits, rounded once at the end.  ``exact`` computes the same from the definitions in 64 bits, and ``work`` counts what a pass
has to read, write and compute.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # training a recurrent layer of 2048 channels on 4 sequences of 4096 tokens: forward and all gradients
        dict(name="scan_train_b4_t4096", op="scan", kind="train", dtype="bf16", gate="same", N=4, T=4096, D=2048, packed=False,
             spread=0),
        # prefill of 16 packed prompts of uneven length, fp32, an odd number of channels, states carried in and out
        dict(name="scan_prefill_packed_fp32", op="scan", kind="prefill", dtype="fp32", gate="same", N=16, T=32749, D=1001,
             packed=True, spread=3),
        # one decode step of 256 sequences, the fp32 state updated in place
        dict(name="scan_step_256x4096", op="scan", kind="step", dtype="bf16", gate="same", N=256, T=1, D=4096, packed=False,
             spread=0),
        # a prefill of 8192 tokens: heads normed, turned and written into the cache
        dict(name="qknorm_append_t8192", op="qknorm", kind="append", dtype="bf16", D=128, rot=128, Hq=32, Hkv=8, page=64, N=1,
             q=8192, kv=8192, spread=0, interleaved=False, offset=0.0),
        # the same in a decode step of 64 sequences
        dict(name="qknorm_append_b64", op="qknorm", kind="append", dtype="bf16", D=128, rot=128, Hq=32, Hkv=8, page=64, N=64,
             q=1, kv=4096, spread=5, interleaved=False, offset=0.0),
        # training: gradients of q, k and both weights, 4 x 4096 tokens, a zero-centred weight, half of each head turned
        dict(name="qknorm_bwd_b4_t4096", op="qknorm", kind="bwd", dtype="bf16", D=128, rot=64, Hq=16, Hkv=4, T=16384,
             interleaved=True, offset=1.0),
        # a server's decode step over long contexts cut to a window of 2048 tokens and the first 4
        dict(name="sinks_decode_b48", op="sinks", dtype="bf16", D=128, Hkv=8, G=4, page=64, N=48, q=1, mixed=False, kv=32768,
             spread=4, window=2048, sinks=4),
        # chunked prefill under the window: 2048 new tokens after 8192 cached ones
        dict(name="sinks_chunk2048_ctx10240", op="sinks", dtype="bf16", D=128, Hkv=8, G=4, page=64, N=1, q=2048, mixed=False,
             kv=10240, spread=0, window=1024, sinks=128),
        # fp32 check of a ragged batch in which some sequences decode and some prefill; sinks that end inside a page
        dict(name="sinks_mixed_fp32_d64", op="sinks", dtype="fp32", D=64, Hkv=4, G=2, page=16, N=8, q=256, mixed=True, kv=3000,
             spread=7, window=300, sinks=21),
        # four samples of one user's prompt of about 1000 tokens: latency counts
        dict(name="prefix_decode_1x4_ctx1000", op="prefix", dtype="bf16", D=128, Hkv=8, G=4, page=16, groups=1, per=4, q=1,
             prefix=992, tail=40, spread=1),
        # 64 requests behind one system prompt of 8192 tokens, each with up to 1024 tokens of its own
        dict(name="prefix_decode_1x64_ctx8192", op="prefix", dtype="bf16", D=128, Hkv=8, G=4, page=64, groups=1, per=64, q=1,
             prefix=8192, tail=1024, spread=2),
        # eight prompts with eight branches each, five drafted tokens checked at once
        dict(name="prefix_draft_8x8_d64", op="prefix", dtype="bf16", D=64, Hkv=4, G=8, page=32, groups=8, per=8, q=5,
             prefix=4090, tail=300, spread=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _top():
    """The largest listed case of each count: a drawn one costs no more."""
    w = [work(c) for c in listed()]
    return max(x["bytes"] for x in w), max(x["flops"] for x in w)


def draw(rng):
    most_bytes, most_flops = _top()
    while True:
        op = rng.choice(["scan", "qknorm", "sinks", "prefix"])
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        D, Hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
        if op == "scan":
            kind = rng.choice(["train", "prefill", "step"])
            c = dict(op=op, kind=kind, dtype=dtype, gate=rng.choice(["same", "fp32"]), N=_log(rng, 1, 64), T=_log(rng, 1, 32768),
                     D=rng.choice([64, 100, 256, 1001, 1024, 2048, 2560, 4096]), packed=rng.random() < 0.5,
                     spread=rng.randrange(1 << 16))
            if kind == "step":
                c.update(N=_log(rng, 1, 512), T=1, packed=False)
            if c["packed"]:
                c["T"] = max(c["T"], c["N"])
            if _tokens(c) * c["D"] > 1 << 25:
                continue
        elif op == "qknorm":
            kind = rng.choice(["append", "append", "fwd", "bwd"])
            c = dict(op=op, kind=kind, dtype=dtype, D=D, rot=rng.choice([D, D // 2, D // 4]), Hq=Hkv * rng.choice([1, 2, 4, 8]),
                     Hkv=Hkv, interleaved=rng.random() < 0.5, offset=rng.choice([0.0, 1.0]))
            if kind == "append":
                c.update(page=page, N=_log(rng, 1, 64), q=_log(rng, 1, 4096), spread=rng.randrange(1 << 16))
                c["kv"] = c["q"] + _log(rng, 1, 16384)
                if c["N"] * c["kv"] * Hkv * D * 4 > 2e9:
                    continue
            else:
                c["T"] = _log(rng, 1, 32768)
        elif op == "sinks":
            kind = rng.choice(["decode", "decode", "draft", "chunk", "mixed"])
            c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, G=rng.choice([1, 2, 3, 4, 6, 8, 16]), page=page, N=_log(rng, 1, 64),
                     q=1, mixed=kind == "mixed", kv=_log(rng, 1, 32768), spread=rng.randrange(1 << 16),
                     window=_log(rng, 16, 4096), sinks=_log(rng, 1, 512))
            if kind == "draft":
                c["q"] = rng.randint(2, 8)
            if kind in ("chunk", "mixed"):
                c["q"] = _log(rng, 16, 2048)
            c["kv"] = max(c["kv"], c["q"])
            # the plain form gathers padded keys and holds all scores at once
            if c["N"] * c["kv"] * Hkv * D * 4 > 6e9 or c["N"] * Hkv * c["G"] * c["q"] * c["kv"] * 4 > 4e9:
                continue
        else:
            c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, G=rng.choice([1, 2, 3, 4, 6, 8, 16]), page=page, groups=_log(rng, 1, 8),
                     per=_log(rng, 1, 64), q=rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 8, 64)]),
                     prefix=_log(rng, 1, 16384), tail=_log(rng, 1, 2048), spread=rng.randrange(1 << 16))
            c["tail"] = max(c["tail"], c["q"])
            N, L = c["groups"] * c["per"], c["prefix"] + c["tail"]
            if N * L * Hkv * D * 4 > 6e9 or N * Hkv * c["G"] * c["q"] * L * 4 > 4e9:
                continue
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


# ------------------------------------------------------------------------------------- lengths of a ragged batch
def _tokens(c):
    return c["T"] if c["packed"] else c["N"] * c["T"]


def _scan_lengths(c):
    """Tokens of every sequence of a recurrence: equal, or packed ones that add up to T (empty ones among them)."""
    if not c["packed"]:
        return [c["T"]] * c["N"]
    r = random.Random(c["spread"])
    cuts = sorted(r.randint(0, c["T"]) for _ in range(c["N"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [c["T"]])]


def _lengths(c):
    """(new tokens, cached tokens with them) of every sequence: the first has the case's sizes."""
    r = random.Random(c["spread"])
    qs, ks = [], []
    for n in range(c["N"]):
        q, kv = c["q"], c["kv"]
        if n:
            kv = r.randint(max(1, kv // 32), kv)
            if c.get("mixed"):
                q = r.choice([1, 1, r.randint(0, q), q])
            kv = max(kv, q)
        qs.append(q)
        ks.append(kv)
    return qs, ks


def _tails(c):
    """Tokens behind the shared prefix, the new ones among them, of every sequence of every group."""
    r = random.Random(c["spread"])
    return [r.randint(c["q"], c["tail"]) for _ in range(c["groups"] * c["per"])]


def _seen(c, q, kv):
    """Keys of a sequence that some query sees, and (query, key) pairs, under a window with first tokens that stay."""
    W, S = c["window"], c["sinks"]
    pos = range(kv - q, kv)
    pairs = sum(p + 1 if p + 1 <= W + S else W + S for p in pos)
    lo = max(0, kv - q + 1 - W)  # the first query's window begins here
    return (kv - lo + min(S, lo)) if q else 0, pairs


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    op, D = c["op"], c["D"]
    if op == "scan":
        n = _tokens(c) * D
        eg = 4 if c["gate"] == "fp32" else e
        states = 8 * c["N"] * D
        if c["kind"] == "train":  # x, g, dy and the states' gradients in; y, dx, dg out
            return dict(bytes=n * (4 * e + 2 * eg) + 2 * states, flops=10 * n)
        return dict(bytes=n * (2 * e + eg) + states, flops=3 * n)
    if op == "qknorm":
        if c["kind"] == "append":
            T = sum(_lengths(c)[0])
            values = T * (c["Hq"] + 2 * c["Hkv"]) * D
            return dict(bytes=2 * values * e + T * c["rot"] * 4 + 8 * D, flops=7 * T * (c["Hq"] + c["Hkv"]) * D)
        values = c["T"] * (c["Hq"] + c["Hkv"]) * D
        table = c["T"] * (c["rot"] * 4 + 4)
        if c["kind"] == "fwd":
            return dict(bytes=2 * values * e + table + 8 * D, flops=7 * values)
        return dict(bytes=3 * values * e + table + 16 * D, flops=14 * values)
    Hq = c["Hkv"] * c["G"]
    if op == "sinks":
        seen = [_seen(c, q, k) for q, k in zip(*_lengths(c))]
        keys, pairs, rows = sum(s[0] for s in seen), sum(s[1] for s in seen), sum(_lengths(c)[0]) * Hq
    else:
        tails = _tails(c)
        rows = len(tails) * c["q"] * Hq
        keys = c["groups"] * c["prefix"] + sum(tails)
        pairs = sum(c["q"] * (c["prefix"] + t) - c["q"] * (c["q"] - 1) // 2 for t in tails)
    return dict(bytes=2 * keys * c["Hkv"] * D * e + rows * (2 * D * e + 4), flops=4 * pairs * Hq * D)


# ------------------------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _paged(c, gen, need, shared=0, per=1):
    """A page table for sequences of `need` pages each, of which the first `shared` are the same within every `per` sequences;
    the pages lie in random order, and some belong to nobody.  Returns the size of the pool and the table, -1 after a
    sequence's last page."""
    total = sum(n - shared for n in need) + len(need) // per * shared + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for n, pages in enumerate(need):
        if n % per == 0:
            head = perm[at:at + shared]
            at += shared
        table[n, :shared] = head
        table[n, shared:pages] = perm[at:at + pages - shared]
        at += pages - shared
    return total, table


def _table(c, positions):
    """cos and sin of every position and pair, [positions, rot / 2, 2] fp32: a program builds it once."""
    i = torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-i / c["rot"])
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, op, D = TYPES[c["dtype"]], c["op"], c["D"]
    s = dict(case=c)
    if op == "scan":
        N, lens = c["N"], _scan_lengths(c)
        lead = (1, c["T"]) if c["packed"] else (N, c["T"])
        gt = dt if c["gate"] == "same" else torch.float32
        s["x"] = _randn(gen, *lead, D, dtype=dt)
        # channels remember from one to some thousand tokens
        rate = 10.0 ** (-3.5 * torch.rand(D, generator=gen, device=DEV))
        s["g"] = (-rate * torch.log1p(torch.exp(_randn(gen, *lead, D)))).to(gt)
        s["h0"] = _randn(gen, N, D)
        s["cu"] = _ints(_cu(lens)) if c["packed"] else None
        if c["kind"] == "step":
            s["x"], s["g"] = s["x"][:, 0].contiguous(), s["g"][:, 0].contiguous()
        if c["kind"] == "train":
            s["dy"] = _randn(gen, *lead, D, dtype=dt)
            s["dhT"] = _randn(gen, N, D)
        return s
    if op == "qknorm":
        s["wq"], s["wk"] = (1.0 - c["offset"] + 0.1 * _randn(gen, D) for _ in range(2))
        if c["kind"] != "append":
            s["q"], s["k"] = _randn(gen, c["T"], c["Hq"] + c["Hkv"], D, dtype=dt).split([c["Hq"], c["Hkv"]], 1)
            s["positions"] = torch.arange(c["T"], device=DEV, dtype=torch.int32) % 4096
            s["table"] = _table(c, 4096)
            if c["kind"] == "bwd":
                s["dq"], s["dk"] = _randn(gen, c["T"], c["Hq"], D, dtype=dt), _randn(gen, c["T"], c["Hkv"], D, dtype=dt)
            return s
    if op == "prefix":
        tails = _tails(c)
        qs, ks = [c["q"]] * len(tails), [c["prefix"] + t for t in tails]
        total, s["page_table"] = _paged(c, gen, [-(-k // c["page"]) for k in ks], -(-c["prefix"] // c["page"]), c["per"])
        s["prefix_lens"] = _ints([c["prefix"]] * c["groups"])
        s["cu_seqs"] = _ints([i * c["per"] for i in range(c["groups"] + 1)])
    else:
        qs, ks = _lengths(c)
        total, s["page_table"] = _paged(c, gen, [-(-k // c["page"]) for k in ks])
    cu = _cu(qs)
    s["kv_lens"], s["cu_q"], s["total"], s["max_q"], s["max_kv"] = _ints(ks), _ints(cu), cu[-1], max(qs), max(ks)
    s["k_cache"] = _randn(gen, total, c["page"], c["Hkv"], D, dtype=dt)
    s["v_cache"] = _randn(gen, total, c["page"], c["Hkv"], D, dtype=dt)
    if op == "qknorm":  # queries, keys and values are slices of one projection's output
        qkv = _randn(gen, cu[-1], c["Hq"] + 2 * c["Hkv"], D, dtype=dt)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        s["table"] = _table(c, max(ks))
    else:
        s["q"] = _randn(gen, cu[-1], c["Hkv"] * c["G"], D, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------------- the plain forms
def _shift(a, s):
    """a [tokens, D] moved s tokens later, zeros first."""
    return torch.cat([torch.zeros_like(a[:s]), a[:-s]])


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t over the first dimension, h_{-1} = 0, in log2 steps: spans of tokens are joined in pairs."""
    s = 1
    while s < a.shape[0]:
        b = b + a * _shift(b, s)
        a = a * _shift(a, s)
        s *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    D = c["D"]
    if c["kind"] == "step":
        h = s["g"].float().exp() * s["h0"] + s["x"].float()
        s["h0"].copy_(h)
        return dict(y=h.to(s["x"].dtype), state=s["h0"])
    # in 64 bits: gates near one are multiplied thousands of times
    x, a = s["x"].double().reshape(-1, D), s["g"].double().reshape(-1, D).exp()
    cu = s["cu"] if s["cu"] is not None else torch.arange(c["N"] + 1, device=DEV) * c["T"]
    beg, end = cu[:-1].long(), cu[1:].long()
    some = (end > beg)[:, None]
    tokens = x.shape[0]
    # rows of empty sequences go to a row of their own behind the others
    first, last = torch.where(end > beg, beg, tokens), torch.where(end > beg, end - 1, tokens)
    zeros, h0 = torch.zeros(tokens + 1, D, dtype=torch.float64, device=DEV), s["h0"].double()
    start = zeros.index_copy(0, first, h0)[:-1]                      # the state before each sequence's first token
    begins = zeros[:, :1].index_fill(0, first, 1.0)[:-1] > 0
    h = _doubling(torch.where(begins, 0.0, a), x + a * start)
    pad = torch.cat([h, h[:1]])
    got = dict(y=h.to(s["x"].dtype).view_as(s["x"]), final=torch.where(some, pad[last], h0).float())
    if c["kind"] == "prefill":
        return got
    dhT = s["dhT"].double()
    dy = s["dy"].double().reshape(-1, D) + zeros.index_copy(0, last, dhT)[:-1]
    after = torch.cat([torch.where(begins, 0.0, a)[1:], torch.zeros_like(a[:1])])  # the gate of the next token
    d = _doubling(after.flip(0), dy.flip(0)).flip(0)
    back = a * d
    before = torch.where(begins, start, _shift(h, 1))
    padded = torch.cat([back, back[:1]])
    return dict(got, dx=d.to(s["x"].dtype).view_as(s["x"]), dg=(back * before).to(s["g"].dtype).view_as(s["g"]),
                dh0=torch.where(some, padded[first], dhT).float())


def _plain_rotate(x, cs, interleaved, inverse=False):
    """x [T, H, D] fp32, cs [T, rot / 2, 2]: the leading features turn by the pairs' angles."""
    rot = 2 * cs.shape[1]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_headnorm(x, w, cs, c):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (w + c["offset"])
    return _plain_rotate(y, cs, c["interleaved"]).to(x.dtype)


def _plain_headnorm_bwd(dy, x, w, cs, c):
    u = _plain_rotate(dy.float(), cs, c["interleaved"], True)
    h = x.float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    h = h * rstd
    g = u * (w + c["offset"])
    dx = rstd * (g - h * (g * h).mean(-1, keepdim=True))
    return dx.to(x.dtype), (u * h).sum((0, 1))


def _places(s):
    """Position, page and slot of every new token of a batch."""
    c = s["case"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(s["total"], device=DEV)
    n = torch.bucketize(t, cu[1:], right=True)
    pos = kv[n] - cu[n + 1] + t
    return pos, s["page_table"][n, pos // c["page"]].long(), pos % c["page"]


def _plain_qknorm(s):
    c = s["case"]
    if c["kind"] == "append":
        pos, page, off = _places(s)
        cs = s["table"][pos]
        s["k_cache"][page, off] = _plain_headnorm(s["k"], s["wk"], cs, c)
        s["v_cache"][page, off] = s["v"]
        return dict(q=_plain_headnorm(s["q"], s["wq"], cs, c), k_cache=s["k_cache"], v_cache=s["v_cache"])
    cs = s["table"][s["positions"].long()]
    if c["kind"] == "fwd":
        return dict(q=_plain_headnorm(s["q"], s["wq"], cs, c), k=_plain_headnorm(s["k"], s["wk"], cs, c))
    dq, dwq = _plain_headnorm_bwd(s["dq"], s["q"], s["wq"], cs, c)
    dk, dwk = _plain_headnorm_bwd(s["dk"], s["k"], s["wk"], cs, c)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _plain_attention(s):
    c = s["case"]
    N, Hkv, G, D = s["kv_lens"].shape[0], c["Hkv"], c["G"], c["D"]
    Q, L = s["max_q"], s["max_kv"]
    pages = s["page_table"].clamp(min=0).long()
    k = s["k_cache"][pages].view(N, -1, Hkv, D)[:, :L].float()
    v = s["v_cache"][pages].view(N, -1, Hkv, D)[:, :L].float()
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    i, j = torch.arange(Q, device=DEV), torch.arange(L, device=DEV)
    qlen = cu[1:] - cu[:-1]
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["total"] - 1)].float()              # [N, Q, Hq, D]
    q = q.view(N, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, Hkv, Q * G, D)
    scores = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(D)                            # [N, Hkv, Q * G, L]
    pos = (kv - qlen)[:, None] + i                                                 # [N, Q]
    sees = j <= pos[..., None]
    if c.get("window"):
        sees = sees & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    scores = scores.view(N, Hkv, Q, G, L).masked_fill(~sees[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp()
    mass = p.sum(-1, keepdim=True)
    o = (p / mass.clamp(min=1e-30)).view(N, Hkv, Q * G, L) @ v.permute(0, 2, 1, 3)
    lse = (top + mass.log()).view(N, Hkv, Q, G).permute(0, 2, 1, 3).reshape(N * Q, Hkv * G)
    o = o.view(N, Hkv, Q, G, D).permute(0, 2, 1, 3, 4).reshape(N * Q, Hkv * G, D)
    t = torch.arange(s["total"], device=DEV)
    n = torch.bucketize(t, cu[1:], right=True)
    row = n * Q + t - cu[n]
    return dict(o=o[row].to(s["q"].dtype), lse=lse[row])


# ----------------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return dict(scan=_plain_scan, qknorm=_plain_qknorm, sinks=_plain_attention, prefix=_plain_attention)[op](s)
    import gated_deltanet_linear_15_gb300 as g
    if op == "scan":
        if c["kind"] == "step":
            y, state = g.gated_scan_step(s["x"], s["g"], s["h0"])
            return dict(y=y, state=state)
        if c["kind"] == "prefill":
            y, final = g.gated_scan(s["x"], s["g"], s["h0"], cu_seqlens=s["cu"])
            return dict(y=y, final=final)
        y, final, states = g.gated_scan(s["x"], s["g"], s["h0"], cu_seqlens=s["cu"], save_states=True)
        dx, dg, dh0 = g.gated_scan_bwd(s["dy"], s["x"], s["g"], states, s["h0"], s["dhT"], cu_seqlens=s["cu"])
        return dict(y=y, final=final, dx=dx, dg=dg, dh0=dh0)
    if op == "qknorm":
        how = dict(eps=EPS, weight_offset=c["offset"], interleaved=c["interleaved"])
        if c["kind"] == "append":
            q = g.norm_rotary_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["table"], s["k_cache"], s["v_cache"],
                                     s["page_table"], s["kv_lens"], cu_q=s["cu_q"], **how)
            return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
        if c["kind"] == "fwd":
            q, k = g.norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"], **how)
            return dict(q=q, k=k)
        dq, dk, dwq, dwk = g.norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"], **how)
        return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    if op == "sinks":
        o, lse = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], cu_q=s["cu_q"],
                                   max_q=s["max_q"], window=c["window"], sinks=c["sinks"], return_lse=True)
    else:
        o, lse = g.prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["prefix_lens"],
                                    cu_seqs=s["cu_seqs"], cu_q=s["cu_q"], max_q=s["max_q"], max_group=c["per"] * c["q"],
                                    return_lse=True)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_scan(c, s):
    """Token by token, all sequences at once, padded to the longest."""
    lens, D, N = _scan_lengths(c), c["D"], c["N"]
    if c["kind"] == "step":
        h = torch.exp(s["g"].double()) * s["h0"].double() + s["x"].double()
        return dict(y=h, state=h)
    L = max(lens)
    if N * L * D > 1 << 27 or L > 40000:
        return None
    n_of = torch.tensor([n for n, k in enumerate(lens) for _ in range(k)], device=DEV)
    t_of = torch.tensor([t for k in lens for t in range(k)], device=DEV)
    length = torch.tensor(lens, device=DEV)[:, None]

    def padded(v):
        p = torch.zeros(L, N, D, dtype=torch.float64, device=DEV)
        p[t_of, n_of] = v.reshape(-1, D).double()
        return p

    x, alpha = padded(s["x"]), padded(s["g"]).exp()
    h = s["h0"].double()
    hs = torch.empty(L + 1, N, D, dtype=torch.float64, device=DEV)
    hs[0] = h
    for t in range(L):
        h = torch.where(t < length, alpha[t] * h + x[t], h)
        hs[t + 1] = h
    got = dict(y=hs[t_of + 1, n_of].view(s["x"].shape), final=h)
    if c["kind"] == "prefill":
        return got
    dy, d = padded(s["dy"]), s["dhT"].double()
    dx, dg = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        live = t < length
        dx[t] = d + dy[t]          # all that reaches h_t
        flow = alpha[t] * dx[t]    # what of it reaches h_{t-1}
        dg[t] = flow * hs[t]
        d = torch.where(live, flow, d)
    return dict(got, dx=dx[t_of, n_of].view(s["x"].shape), dg=dg[t_of, n_of].view(s["x"].shape), dh0=d)


def _turn(c, x, cs, inverse=False):
    """Each pair of leading features as a complex number, times exp(+-i angle), with cos and sin as the program holds them."""
    rot = c["rot"]
    w = torch.complex(cs[..., 0].double(), -cs[..., 1].double() if inverse else cs[..., 1].double())[:, None]
    y = x.clone()
    head = y[..., :rot]
    if c["interleaved"]:
        z = torch.view_as_complex(head.reshape(x.shape[0], -1, rot // 2, 2).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_head(c, x, w, cs):
    x = x.double()
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / c["D"] + EPS).sqrt()
    return _turn(c, x / rms * (w.double() + c["offset"]), cs)


def _exact_head_bwd(c, dy, x, w, cs):
    u, x = _turn(c, dy.double(), cs, True), x.double()
    v = w.double() + c["offset"]
    r = (torch.einsum("thd,thd->th", x, x) / c["D"] + EPS) ** -0.5
    dot = torch.einsum("thd,d,thd->th", u, v, x)
    dx = r[..., None] * u * v - (r ** 3 * dot / c["D"])[..., None] * x
    return dx, torch.einsum("thd,thd,th->d", u, x, r)


def _exact_qknorm(c, s):
    if c["kind"] == "append":
        qs, ks = _lengths(c)
        pos = torch.cat([torch.arange(k - q, k, device=DEV) for q, k in zip(qs, ks)])
        seq = torch.repeat_interleave(torch.arange(c["N"], device=DEV), torch.tensor(qs, device=DEV))
        slot = s["page_table"][seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.view(-1, c["Hkv"], c["D"])[slot] = _exact_head(c, s["k"], s["wk"], s["table"][pos])
        vc.view(-1, c["Hkv"], c["D"])[slot] = s["v"].double()
        return dict(q=_exact_head(c, s["q"], s["wq"], s["table"][pos]), k_cache=kc, v_cache=vc)
    cs = s["table"][s["positions"].long()]
    if c["kind"] == "fwd":
        return dict(q=_exact_head(c, s["q"], s["wq"], cs), k=_exact_head(c, s["k"], s["wk"], cs))
    dq, dwq = _exact_head_bwd(c, s["dq"], s["q"], s["wq"], cs)
    dk, dwk = _exact_head_bwd(c, s["dk"], s["k"], s["wk"], cs)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _exact_attention(c, s, qs, ks):
    Hkv, G, D, P = c["Hkv"], c["G"], c["D"], c["page"]
    out, lse, at = [], [], 0
    for n, (ql, kl) in enumerate(zip(qs, ks)):
        pages = s["page_table"][n, :-(-kl // P)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:kl].double()
        v = s["v_cache"][pages].flatten(0, 1)[:kl].double()
        for t in range(0, ql, 128):
            q = s["q"][at + t:at + min(ql, t + 128)].double()
            pos = (kl - ql + t + torch.arange(q.shape[0], device=DEV))[:, None]
            key = torch.arange(kl, device=DEV)[None]
            off = key > pos
            if c.get("window"):
                off = off | ((pos - key >= c["window"]) & (key >= c["sinks"]))
            heads_o, heads_l = [], []
            for h in range(Hkv * G):
                z = (q[:, h] @ k[:, h // G].T) * D ** -0.5
                z[off] = -math.inf
                l = torch.logsumexp(z, -1)
                heads_o.append(torch.exp(z - l[:, None]) @ v[:, h // G])
                heads_l.append(l)
            out.append(torch.stack(heads_o, 1))
            lse.append(torch.stack(heads_l, 1))
        at += ql
    return dict(o=torch.cat(out), lse=torch.cat(lse))


def exact(c, seed):
    op = c["op"]
    if op in ("sinks", "prefix"):
        if op == "sinks":
            qs, ks = _lengths(c)
        else:
            ks = [c["prefix"] + t for t in _tails(c)]
            qs = [c["q"]] * len(ks)
        if sum(q * k for q, k in zip(qs, ks)) * c["Hkv"] * c["G"] * c["D"] > 1e11 or len(qs) * c["G"] * c["Hkv"] > 4096:
            return None
        return _exact_attention(c, prepare(c, seed), qs, ks)
    s = prepare(c, seed)
    return _exact_scan(c, s) if op == "scan" else _exact_qknorm(c, s)
