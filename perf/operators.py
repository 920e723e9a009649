"""The operators that a hybrid stack puts next to its gated delta-rule layers, as measurable cases.

A stack of gated delta-rule layers usually carries a softmax-attention layer after every few of them.  Such a
layer, and the blocks around both kinds, need: attention of new tokens over a paged cache of keys and values,
rotary positions (with the write of the new keys and values into that cache), the upkeep of the cache's pages
(fork, free, compact, copy; a fork also copies the sequence's delta-rule state), and the residual's
root-mean-square norm, whose output may be 8-bit.

``listed()`` names the cases, ``draw(rng)`` gives others of the same ranges, ``prepare`` makes what a program has
in hand before the call, ``run`` makes one pass: with ``own`` through this package, without it in elementary torch
operations in 32 bits, rounded once at the end.  ``exact`` computes the same from the definitions in 64 bits, and
``work`` counts what a pass has to read, write and compute.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30


# --------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token over a short conversation: launch and latency count
        dict(name="attn_decode_b1_ctx1024", op="attn", dtype="bf16", D=128, Hkv=8, G=4, page=16, N=1, q=1, mixed=False,
             kv=1024, spread=0, window=0),
        # a server's decode step: 64 ragged sequences of 512 .. 16384 tokens
        dict(name="attn_decode_b64_ragged", op="attn", dtype="bf16", D=128, Hkv=8, G=4, page=64, N=64, q=1, mixed=False,
             kv=16384, spread=4, window=0),
        # one agent's long context with few heads, four drafted tokens checked at once, odd length
        dict(name="attn_draft4_b1_ctx65531", op="attn", dtype="bf16", D=128, Hkv=2, G=8, page=128, N=1, q=4, mixed=False,
             kv=65531, spread=0, window=0),
        # chunked prefill: 2048 new tokens after 8192 cached ones, 32 heads
        dict(name="attn_chunk2048_ctx10240", op="attn", dtype="bf16", D=128, Hkv=8, G=4, page=64, N=1, q=2048, mixed=False,
             kv=10240, spread=0, window=0),
        # fp32 check of a ragged batch in which some sequences decode and some prefill, under a sliding window
        dict(name="attn_mixed_fp32_d64", op="attn", dtype="fp32", D=64, Hkv=4, G=2, page=16, N=8, q=256, mixed=True,
             kv=3000, spread=7, window=1024),
        # the keys and values of a prefill of 8192 tokens: rotated and written into the cache
        dict(name="rope_append_t8192", op="append", dtype="bf16", D=128, rot=128, Hq=32, Hkv=8, page=64, N=1, q=8192,
             mixed=False, kv=8192, spread=0, interleaved=False, factor=1.0),
        # training: gradients through rotary positions on half of each head, pairs interleaved, long-context scaling
        dict(name="rope_bwd_b4_t4096_fp32", op="rope", dtype="fp32", D=128, rot=64, Hq=16, Hkv=16, T=16384,
             interleaved=True, factor=4.0, inverse=True),
        # parallel samples: the last step's 64 branches are dropped and 64 sequences branch anew (page bookkeeping, last
        # pages and delta-rule states copied)
        dict(name="pages_fork_64", op="fork", dtype="bf16", D=128, Hkv=8, page=64, layers=2, N=64, kv=4096, spread=5,
             state_heads=8),
        # the cache after many sequences ended: live pages moved to the front
        dict(name="pages_compact_8192", op="compact", dtype="bf16", D=128, Hkv=8, page=16, layers=2, pages=8192, N=64,
             live=0.55),
        # the norm before a decode step's projections: 64 rows of 32 x 128 features, 8-bit output
        dict(name="norm_fp8_64x4096", op="norm", dtype="bf16", T=64, D=4096, residual=True, out="fp8", group=128),
        # the same in a prefill of 8192 tokens
        dict(name="norm_fp8_8192x4096", op="norm", dtype="bf16", T=8192, D=4096, residual=True, out="fp8", group=128),
        # training: gradients of the residual stream and of the weight, 4 x 4096 tokens of 16 x 128 features
        dict(name="norm_bwd_16384x2048", op="norm_bwd", dtype="bf16", T=16384, D=2048, residual=True),
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
        op = rng.choice(["attn", "attn", "attn", "append", "rope", "fork", "compact", "norm", "norm_bwd"])
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        D, Hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
        if op == "attn":
            kind = rng.choice(["decode", "decode", "draft", "chunk", "mixed"])
            c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, G=rng.choice([1, 2, 3, 4, 6, 8, 16]), page=page, N=_log(rng, 1, 96),
                     q=1, mixed=kind == "mixed", kv=_log(rng, 1, 65536), spread=rng.randrange(1 << 16),
                     window=0 if rng.random() < 0.75 else _log(rng, 16, 4096))
            if kind == "draft":
                c["q"] = rng.randint(2, 8)
            if kind in ("chunk", "mixed"):
                c["q"] = _log(rng, 16, 2048)
            c["kv"] = max(c["kv"], c["q"])
            # the plain form gathers padded keys and holds all scores at once
            if c["N"] * c["kv"] * Hkv * D * 4 > 6e9 or c["N"] * Hkv * c["G"] * c["q"] * c["kv"] * 4 > 4e9:
                continue
        elif op == "append":
            c = dict(op=op, dtype=dtype, D=D, rot=rng.choice([D, D // 2, D // 4]), Hq=Hkv * rng.choice([1, 2, 4, 8]),
                     Hkv=Hkv, page=page, N=_log(rng, 1, 64), q=_log(rng, 1, 4096), mixed=rng.random() < 0.5, kv=0,
                     spread=rng.randrange(1 << 16), interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 2.0, 8.0]))
            c["kv"] = c["q"] + _log(rng, 1, 16384)
            if c["N"] * c["kv"] * Hkv * D * 4 > 2e9:
                continue
        elif op == "rope":
            c = dict(op=op, dtype=dtype, D=D, rot=rng.choice([D, D // 2, D // 4]), Hq=rng.choice([1, 4, 8, 16, 32]),
                     Hkv=rng.choice([1, 2, 8]), T=_log(rng, 1, 32768), interleaved=rng.random() < 0.5,
                     factor=rng.choice([1.0, 2.0, 8.0]), inverse=rng.random() < 0.5)
        elif op == "fork":
            c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, page=page, layers=rng.randint(1, 4), N=_log(rng, 1, 128),
                     kv=_log(rng, 1, 8192), spread=rng.randrange(1 << 16), state_heads=rng.choice([1, 4, 8]))
            if c["N"] * (c["kv"] + 2 * page) * Hkv * D * 4 * 2 * c["layers"] > 4e9:
                continue
        elif op == "compact":
            c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, page=page, layers=rng.randint(1, 3), pages=_log(rng, 16, 16384),
                     N=_log(rng, 1, 128), live=round(rng.uniform(0.05, 0.95), 3))
            if c["pages"] * page * Hkv * D * 4 * 2 * c["layers"] > 4e9:
                continue
        else:
            c = dict(op=op, dtype=dtype, T=_log(rng, 1, 32768), D=rng.choice([64, 128, 1000, 1024, 2048, 4096, 5120, 8192]),
                     residual=rng.random() < 0.7)
            if op == "norm":
                c["out"] = rng.choice(["same", "fp8", "fp8"])
                c["group"] = 0 if c["out"] == "same" or c["D"] % 128 or rng.random() < 0.4 else 128
            if c["T"] * c["D"] > 1 << 26:
                continue
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


# ------------------------------------------------------------------------------------- lengths of a ragged batch
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


def _pairs(q, kv, window):
    """(query, key) pairs that attend: query i of q sits at position kv - q + i and sees the keys up to its own
    position, the last `window` of them where there is a window."""
    first, last = kv - q + 1, kv
    total = (first + last) * q // 2
    if window and last > window:
        lo = max(first, window)
        total -= (lo - window + last - window) * (last - lo + 1) // 2
    return total


def _seen(q, kv, window):
    """Keys that some query of the sequence sees."""
    if not q:
        return 0
    return kv - (max(0, kv - q + 1 - window) if window else 0)


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    op, D = c["op"], c["D"]
    if op == "attn":
        qs, ks = _lengths(c)
        keys = sum(_seen(q, k, c["window"]) for q, k in zip(qs, ks))
        pairs = sum(_pairs(q, k, c["window"]) for q, k in zip(qs, ks))
        Hq = c["Hkv"] * c["G"]
        rows = sum(qs) * Hq
        return dict(bytes=2 * keys * c["Hkv"] * D * e + rows * (2 * D * e + 4), flops=4 * pairs * Hq * D)
    if op == "append":
        T = sum(_lengths(c)[0])
        values = T * (c["Hq"] + 2 * c["Hkv"]) * D
        return dict(bytes=2 * values * e + T * c["rot"] * 4, flops=3 * T * (c["Hq"] + c["Hkv"]) * c["rot"])
    if op == "rope":
        values = c["T"] * (c["Hq"] + c["Hkv"]) * D
        return dict(bytes=2 * values * e + c["T"] * (c["rot"] * 4 + 4), flops=3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"])
    if op == "fork":
        ks = _lengths(dict(c, q=0))[1]
        part = sum(k % c["page"] != 0 for k in ks)
        pages = sum(-(-k // c["page"]) for k in ks)
        moved = part * c["page"] * c["Hkv"] * D * e * 2 * c["layers"] + c["N"] * c["state_heads"] * D * D * 4
        return dict(bytes=2 * moved + 6 * 4 * pages, flops=pages)
    if op == "compact":
        live = _live(c)
        moves = sum(p >= len(live) for p in live)
        held = len(live)
        return dict(bytes=2 * moves * c["page"] * c["Hkv"] * D * e * 2 * c["layers"] + 8 * (c["pages"] + held),
                    flops=c["pages"])
    n = c["T"] * D
    if op == "norm":
        o = 1 if c["out"] == "fp8" else e
        scales = 4 * c["T"] * (D // c["group"] if c["group"] else 1) if c["out"] == "fp8" else 0
        return dict(bytes=n * (e + (2 * e if c["residual"] else 0) + o) + scales + 4 * c["T"] + 4 * D, flops=6 * n)
    return dict(bytes=n * e * (3 + c["residual"]) + 4 * c["T"] + 8 * D, flops=10 * n)


# ------------------------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _paged(c, gen, ks):
    """A cache in whose pool the sequences' pages lie in random order, with some pages that nobody holds; page_table
    [sequences, pages], -1 after a sequence's last page."""
    P = c["page"]
    need = [-(-k // P) for k in ks]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    width = max(max(need), 1)
    at = torch.arange(width, device=DEV)[None, :]
    cnt = torch.tensor(need, device=DEV)[:, None]
    start = torch.cumsum(cnt, 0) - cnt
    table = torch.where(at < cnt, perm[(start + at).clamp(max=total - 1)], torch.full_like(perm[:1], -1))
    return total, table.contiguous()


def _inv_freq(c):
    """Angle per position of each feature pair: base 10000, the positions stretched by the case's factor."""
    i = torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64)
    return 10000.0 ** (-i / c["rot"]) / c["factor"]


def _table(c, positions):
    """cos and sin of every position and pair, [positions, rot / 2, 2] fp32: a program builds it once."""
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * _inv_freq(c)[None, :]
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _live(c):
    """The page numbers in use of a cache from which sequences have gone, in ascending order."""
    r = random.Random(c["pages"] * 7919 + c["N"])
    return [p for p in range(c["pages"]) if r.random() < c["live"]]


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, op, D = TYPES[c["dtype"]], c["op"], c["D"]
    s = dict(case=c)
    if op in ("attn", "append"):
        qs, ks = _lengths(c)
        total, s["page_table"] = _paged(c, gen, ks)
        s["kv_lens"] = _ints(ks)
        cu = [0]
        for q in qs:
            cu.append(cu[-1] + q)
        s["cu_q"], s["total"], s["max_q"], s["max_kv"] = _ints(cu), cu[-1], max(qs), max(ks)
        s["k_cache"] = _randn(gen, total, c["page"], c["Hkv"], D, dtype=dt)
        s["v_cache"] = _randn(gen, total, c["page"], c["Hkv"], D, dtype=dt)
        if op == "attn":
            s["q"] = _randn(gen, cu[-1], c["Hkv"] * c["G"], D, dtype=dt)
        else:  # queries, keys and values are slices of one projection's output
            qkv = _randn(gen, cu[-1], c["Hq"] + 2 * c["Hkv"], D, dtype=dt)
            s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
            s["table"] = _table(c, max(ks))
    elif op == "rope":
        s["q"], s["k"] = _randn(gen, c["T"], c["Hq"] + c["Hkv"], D, dtype=dt).split([c["Hq"], c["Hkv"]], 1)
        s["positions"] = torch.arange(c["T"], device=DEV, dtype=torch.int32) % 4096
        s["table"] = _table(c, 4096)
    elif op == "fork":
        ks = _lengths(dict(c, q=0))[1]
        total, table = _paged(c, gen, ks)
        total += c["N"]  # room for the children's last pages
        s["page_table"] = torch.cat([table, torch.full_like(table, -1)])
        s["seq_lens"] = torch.cat([_ints(ks), torch.zeros(c["N"], dtype=torch.int32, device=DEV)])
        s["refcount"] = torch.zeros(total, dtype=torch.int32, device=DEV)
        s["refcount"][table[table >= 0].long()] = 1
        s["pools"] = [_randn(gen, total, c["page"], c["Hkv"], D, dtype=dt) for _ in range(2 * c["layers"])]
        s["states"] = 0.02 * _randn(gen, 2 * c["N"], c["state_heads"], D, D)
        s["parents"] = torch.randperm(c["N"], generator=gen, device=DEV).to(torch.int32)
        s["children"] = (c["N"] + torch.randperm(c["N"], generator=gen, device=DEV)).to(torch.int32)
    elif op == "compact":
        live = _live(c)
        width = max(1, -(-len(live) // c["N"]))
        held = torch.full((c["N"] * width,), -1, dtype=torch.int32, device=DEV)
        if live:
            held[:len(live)] = _ints(live)[torch.randperm(len(live), generator=gen, device=DEV)]
        s["page_table"] = held.view(width, c["N"]).t().contiguous()
        s["refcount"] = torch.zeros(c["pages"], dtype=torch.int32, device=DEV)
        if live:
            s["refcount"][_ints(live).long()] = 1
        s["pools"] = [_randn(gen, c["pages"], c["page"], c["Hkv"], D, dtype=dt) for _ in range(2 * c["layers"])]
    else:
        s["x"] = _randn(gen, c["T"], D, dtype=dt)
        s["weight"] = 1.0 + 0.1 * _randn(gen, D)
        s["residual"] = 2.0 * _randn(gen, c["T"], D, dtype=dt) if c["residual"] else None
        if op == "norm_bwd":  # x is the stored sum of the forward; residual is the gradient that comes down the stream
            s["dy"] = _randn(gen, c["T"], D, dtype=dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + 1e-6)
    return s


# ---------------------------------------------------------------------------------------------- the plain forms
def _plain_attention(s):
    c = s["case"]
    N, Hkv, G, D, P = c["N"], c["Hkv"], c["G"], c["D"], c["page"]
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
    if c["window"]:
        sees = sees & (j > pos[..., None] - c["window"])
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


def _plain_rotate(x, cs, interleaved, inverse):
    """x [T, H, D], cs [T, rot / 2, 2]: the leading features turn by the pairs' angles."""
    rot = 2 * cs.shape[1]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sin = -sin
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    cs = s["table"][s["positions"].long()]
    return dict(q=_plain_rotate(s["q"], cs, c["interleaved"], c["inverse"]),
                k=_plain_rotate(s["k"], cs, c["interleaved"], c["inverse"]))


def _plain_append(s):
    c = s["case"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(s["total"], device=DEV)
    n = torch.bucketize(t, cu[1:], right=True)
    pos = kv[n] - cu[n + 1] + t
    cs = s["table"][pos]
    page, off = s["page_table"][n, pos // c["page"]].long(), pos % c["page"]
    s["k_cache"][page, off] = _plain_rotate(s["k"], cs, c["interleaved"], False)
    s["v_cache"][page, off] = s["v"]
    return dict(q=_plain_rotate(s["q"], cs, c["interleaved"], False), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_fork(s):
    c = s["case"]
    P, table, lens, ref = c["page"], s["page_table"], s["seq_lens"], s["refcount"]
    par, chi = s["parents"].long(), s["children"].long()
    # the branches of the step before end
    gone = table[chi]
    ref.scatter_add_(0, gone.clamp(min=0).long().flatten(), -(gone >= 0).to(torch.int32).flatten())
    # and new ones begin
    n, width = lens[par].long(), table.shape[1]
    part = n % P != 0
    free = torch.argsort((ref != 0).to(torch.int32), stable=True)                  # pages nobody holds first, ascending
    new = torch.where(part, free[(torch.cumsum(part, 0) - 1).clamp(min=0)], torch.full_like(n, -1))
    last = (n // P).clamp(max=width - 1)
    rows = table[par]
    old = torch.gather(rows, 1, last[:, None])[:, 0].clamp(min=0).long()
    dst = torch.where(part, new, old)                                              # nothing to copy: onto itself
    at = torch.arange(width, device=DEV)[None, :]
    shared = at < (n // P)[:, None]
    ref.scatter_add_(0, rows.clamp(min=0).long().flatten(), shared.to(torch.int32).flatten())
    ref.scatter_add_(0, dst, part.to(torch.int32))
    table[chi] = torch.where((at == last[:, None]) & part[:, None], new[:, None].to(torch.int32), rows)
    lens[chi] = lens[par]
    for pool in s["pools"]:
        pool[dst] = pool[old]
    s["states"][chi] = s["states"][par]
    return dict(new=new.to(torch.int32), page_table=table, seq_lens=lens, refcount=ref, pools=s["pools"],
                states=s["states"])


def _plain_compact(s):
    table, ref = s["page_table"], s["refcount"]
    total = ref.numel()
    ids = torch.arange(total, device=DEV)
    live = ref > 0
    count = live.sum()
    high, hole = live & (ids >= count), ~live & (ids < count)
    moves = high.sum()
    src = torch.argsort((~high).to(torch.int32), stable=True)                      # ascending, the moving pages first
    dst = torch.argsort((~hole).to(torch.int32), stable=True)
    new = torch.where(high, dst[(torch.cumsum(high, 0) - 1).clamp(min=0)], ids)
    table = torch.where(table >= 0, new[table.clamp(min=0).long()].to(torch.int32), table)
    counts = torch.zeros_like(ref).scatter_add_(0, new, ref)
    half = total // 2 + 1
    real = ids[:half] < moves
    a = torch.where(real, src[:half], total - 1)                                   # padded with a page that stays
    b = torch.where(real, dst[:half], total - 1)
    for pool in s["pools"]:
        pool[b] = pool[a]
    return dict(page_table=table, refcount=counts, moves=moves.to(torch.int32), pools=s["pools"])


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(-1) + 1e-6)
    y = h * rstd[:, None] * s["weight"]
    got = dict(rstd=rstd)
    if c["residual"]:
        got["h"] = h.to(s["x"].dtype)
    if c["out"] == "same":
        return dict(got, y=y.to(s["x"].dtype))
    g = y.view(c["T"], -1, c["group"] or c["D"])
    scale = g.abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (g / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(torch.float8_e4m3fn)
    return dict(got, y=q, scale=scale)


def _plain_norm_bwd(s):
    c = s["case"]
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"]
    dx = rstd * g - h * rstd.pow(3) * (g * h).mean(-1, keepdim=True)
    if c["residual"]:
        dx = dx + s["residual"].float()
    return dict(dx=dx.to(s["x"].dtype), dw=(dy * h * rstd).sum(0))


# ----------------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return dict(attn=_plain_attention, append=_plain_append, fork=_plain_fork, compact=_plain_compact,
                    norm=_plain_norm, norm_bwd=_plain_norm_bwd, rope=_plain_rope)[op](s)
    import gated_deltanet_linear_15_gb300 as g
    if op == "attn":
        o, lse = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], cu_q=s["cu_q"],
                                   max_q=s["max_q"], window=c["window"], return_lse=True)
        return dict(o=o, lse=lse)
    if op == "append":
        q = g.rotary_append(s["q"], s["k"], s["v"], s["table"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                            cu_q=s["cu_q"], interleaved=c["interleaved"])
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "rope":
        q, k = g.rotary(s["q"], s["k"], s["table"], s["positions"], interleaved=c["interleaved"], inverse=c["inverse"])
        return dict(q=q, k=k)
    if op == "fork":
        g.free_pages(s["page_table"], s["seq_lens"], s["refcount"], s["children"])
        new = g.fork_pages(s["page_table"], s["seq_lens"], s["refcount"], s["parents"], s["children"], s["pools"],
                           page_size=c["page"], states=[s["states"]])
        return dict(new=new, page_table=s["page_table"], seq_lens=s["seq_lens"], refcount=s["refcount"],
                    pools=s["pools"], states=s["states"])
    if op == "compact":
        table, ref, moves = g.compact_pages(s["page_table"], s["refcount"], s["pools"], inplace=False)
        return dict(page_table=table, refcount=ref, moves=moves, pools=s["pools"])
    if op == "norm":
        r = g.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6, fp8=c["out"] == "fp8",
                       group=c.get("group", 0))
        got = dict(y=r.y, rstd=r.rstd)
        if c["residual"]:
            got["h"] = r.h
        if c["out"] == "fp8":
            got["scale"] = r.scale
        return got
    dx, dw = g.rms_norm_bwd(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["residual"])
    return dict(dx=dx, dw=dw)


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_attention(c, s):
    Hkv, G, D, P = c["Hkv"], c["G"], c["D"], c["page"]
    qs, ks = _lengths(c)
    out, lse, at = [], [], 0
    for n, (ql, kl) in enumerate(zip(qs, ks)):
        pages = s["page_table"][n, :-(-kl // P)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:kl].double()
        v = s["v_cache"][pages].flatten(0, 1)[:kl].double()
        for t in range(0, ql, 128):
            q = s["q"][at + t:at + min(ql, t + 128)].double()
            pos = kl - ql + t + torch.arange(q.shape[0], device=DEV)
            key = torch.arange(kl, device=DEV)
            off = key[None] > pos[:, None]
            if c["window"]:
                off = off | (pos[:, None] - key[None] >= c["window"])
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


def _exact_turn(c, x, pos, inverse):
    """Each pair of leading features as a complex number, times exp(+-i angle)."""
    rot, T = c["rot"], x.shape[0]
    # the angles of the table that the program holds: cos and sin as stored
    cs = _table(c, int(pos.max()) + 1 if T else 1)[pos.long()].double()
    w = torch.complex(cs[..., 0], -cs[..., 1] if inverse else cs[..., 1])[:, None]
    y = x.double().clone()
    head = y[..., :rot]
    if c["interleaved"]:
        z = torch.view_as_complex(head.reshape(T, -1, rot // 2, 2).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(c, seed):
    op = c["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers and copies
    if op == "attn":
        qs, ks = _lengths(c)
        if sum(q * k for q, k in zip(qs, ks)) * c["Hkv"] * c["G"] * c["D"] > 1e11 or c["N"] * c["G"] * c["Hkv"] > 4096:
            return None
    s = prepare(c, seed)
    if op == "attn":
        return _exact_attention(c, s)
    if op == "rope":
        return dict(q=_exact_turn(c, s["q"], s["positions"], c["inverse"]),
                    k=_exact_turn(c, s["k"], s["positions"], c["inverse"]))
    if op == "append":
        qs, ks = _lengths(c)
        pos = torch.cat([torch.arange(k - q, k, device=DEV) for q, k in zip(qs, ks)])
        seq = torch.repeat_interleave(torch.arange(c["N"], device=DEV), torch.tensor(qs, device=DEV))
        slot = s["page_table"][seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.view(-1, c["Hkv"], c["D"])[slot] = _exact_turn(c, s["k"], pos, False)
        vc.view(-1, c["Hkv"], c["D"])[slot] = s["v"].double()
        return dict(q=_exact_turn(c, s["q"], pos, False), k_cache=kc, v_cache=vc)
    x, w = s["x"].double(), s["weight"].double()
    if op == "norm":
        if c["residual"]:
            x = x + s["residual"].double()
        got = dict(h=x) if c["residual"] else {}
        rms = (torch.linalg.vector_norm(x, dim=-1).square() / c["D"] + 1e-6).sqrt()
        y = x / rms[:, None] * w
        got["rstd"] = 1 / rms
        if c["out"] == "same":
            return dict(got, y=y)
        b = y.unflatten(-1, (-1, c["group"] or c["D"]))
        scale = b.abs().max(-1).values.clamp(min=AMAX_FLOOR) / E4M3_MAX
        return dict(got, y=(b / scale.unsqueeze(-1)).flatten(-2), scale=scale)
    dy, r = s["dy"].double(), s["rstd"].double()
    # y_i = w_i x_i r with r = (mean x^2 + eps)^(-1/2): dL/dx_i = r w_i dy_i - r^3 x_i <w dy, x> / D
    dot = torch.einsum("td,d,td->t", dy, w, x)
    dx = r[:, None] * w * dy - (r ** 3 * dot / c["D"])[:, None] * x
    if c["residual"]:
        dx = dx + s["residual"].double()
    return dict(dx=dx, dw=torch.einsum("td,td,t->d", dy, x, r))
