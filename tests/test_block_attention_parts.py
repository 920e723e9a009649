"""Attention under a window whose first tokens stay visible, and of sequences that share a prefix, against the definition in
64 bits.

Bounds.  Those of the attention without either (tests/test_block_attention.py): bf16 weights and outputs are rounded, 2^-8 of
sum p |v| and of |o|, 5 % on top for fp32 sums; fp32 by three TF32 parts 3e-5 sum p |v|.  Joining a few more parts adds two
roundings and a power of two each, 2^-21 of sum p |v|, inside that room.  lse as there."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests import block_ref as ref
from tests.test_block_attention import make

gpu = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def attention(x, qs, scale, window=0, sinks=0):
    """o, lse and sum p |v| of every query in 64 bits: query i of a sequence at position p sees the keys j <= p with
    j > p - window or j < sinks."""
    q, kc, vc = (x[n].cpu().to(F64) for n in ("q", "k_cache", "v_cache"))
    table, P, G = x["page_table"].cpu(), kc.shape[1], q.shape[1] // kc.shape[2]
    o, mag, lse = torch.zeros_like(q), torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=F64)
    at = 0
    for n, ql in enumerate(qs):
        kv = int(x["kv_lens"][n])
        slots, rows = torch.arange(kv), slice(at, at + ql)
        at += ql
        if not ql or not kv:
            continue
        pages = table[n, slots // P].long()
        p = torch.arange(kv - ql, kv)[:, None]
        see = slots <= p
        if window:
            see &= (slots > p - window) | (slots < sinks)
        seen = see.any(0)  # what nobody sees may hold anything
        k = torch.where(seen[:, None, None], kc[pages, slots % P], 0.0).repeat_interleave(G, 1)
        v = torch.where(seen[:, None, None], vc[pages, slots % P], 0.0).repeat_interleave(G, 1)
        z = (scale * torch.einsum("ihd,jhd->hij", q[rows], k)).masked_fill(~see, -math.inf)
        l = torch.logsumexp(z, -1)
        w = torch.where(l[..., None] == -math.inf, 0.0, torch.exp(z - l[..., None]))
        lse[rows], o[rows], mag[rows] = l.T, torch.einsum("hij,jhd->ihd", w, v), torch.einsum("hij,jhd->ihd", w, v.abs())
    return o, lse, mag


def close(o, lse, x, qs, scale, window=0, sinks=0):
    ro, rl, mag = attention(x, qs, scale, window, sinks)
    o, lse = o.cpu().to(F64), lse.cpu().to(F64)
    tol = 1.05 * 2 ** -8 * (ro.abs() + mag) + 1e-30 if x["q"].dtype == BF else 3e-5 * mag + 1e-30
    assert torch.isfinite(o).all()
    bad = (o - ro).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((o - ro).abs() / tol).max():.2f} of the bound"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (o[empty] == 0).all()
    if (~empty).any():
        assert ((lse - rl)[~empty].abs() <= 1e-5 + 1e-6 * rl[~empty].abs()).all()


# ------------------------------------------------------------------ sinks
SINKS = [
    # (new, cached) tokens, dtype, D, Hkv, G, page, window, sinks
    ([(1, 1)], BF, 128, 1, 1, 16, 1, 1),
    ([(1, 300)], BF, 64, 2, 3, 16, 17, 1),
    ([(1, 700), (1, 40), (1, 21), (1, 5)], BF, 128, 2, 4, 64, 100, 4),
    ([(1, 3000)], BF, 128, 1, 1, 32, 64, 130),         # sinks end inside the third block
    ([(1, 900)], BF, 128, 1, 2, 16, 256, 600),         # sinks reach almost to the window
    ([(1, 900)], BF, 128, 1, 2, 16, 256, 644),         # and to it
    ([(1, 500)], BF, 64, 1, 2, 16, 30, 5000),          # and past the sequence
    ([(4, 2000), (7, 900), (2, 2)], BF, 128, 2, 4, 64, 200, 20),
    ([(5, 1234)], BF, 64, 1, 8, 128, 77, 33),
    ([(300, 1500)], BF, 128, 2, 2, 64, 128, 4),        # chunks: rows of one tile begin their windows elsewhere
    ([(257, 257), (100, 900), (1, 2000)], BF, 128, 1, 4, 32, 50, 10),
    ([(64, 4000)], BF, 64, 2, 4, 16, 1000, 200),
    ([(200, 1000)], BF, 64, 1, 1, 256, 129, 128),
    ([(513, 700)], BF, 128, 1, 1, 16, 1, 1),
    ([(1, 900), (3, 400), (40, 600), (0, 77), (1, 1)], F32, 64, 2, 2, 16, 100, 21),
    ([(1, 2500)], F32, 128, 1, 4, 64, 333, 7),
    ([(30, 800)], F32, 128, 2, 3, 32, 64, 100),
    ([(1, 40), (2, 3)], F32, 64, 1, 1, 16, 10, 4),
]


@gpu
@pytest.mark.parametrize("seqs,dtype,D,Hkv,G,page,window,sinks", SINKS)
@pytest.mark.parametrize("equal", [False, True])
def test_sinks(seqs, dtype, D, Hkv, G, page, window, sinks, equal):
    import gated_deltanet_linear_15_gb300 as g
    if equal:  # without cu_q: as many new tokens for each
        seqs = [(seqs[0][0], max(kv, seqs[0][0])) for _, kv in seqs]
    x, qs = make(seqs, dtype, D, Hkv, G, page, seed=len(seqs) + D)
    args = dict(cu_q=None if equal else ref.lens_to_cu(qs, DEV), max_q=max(qs), window=window, sinks=sinks, return_lse=True)
    o, lse = g.paged_attention(**x, **args)
    close(o, lse, x, qs, D ** -0.5, window, sinks)
    again = g.paged_attention(**x, **args)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    args["max_q"] = 0
    o, lse = g.paged_attention(**x, **args)  # perhaps another kernel
    close(o, lse, x, qs, D ** -0.5, window, sinks)


@gpu
@pytest.mark.parametrize("dtype,D,G,page,new", [(BF, 128, 4, 64, 1), (BF, 64, 1, 16, 1), (F32, 64, 2, 16, 1), (F32, 128, 4, 32, 1),
                                                (BF, 128, 64, 16, 1)])
def test_keys_between_sinks_and_window_may_hold_anything(dtype, D, G, page, new):
    """One new token: what lies between does not reach it, NaN included; G = 64 takes the chunk kernel."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(new, 1000), (new, 801)], dtype, D, 1, G, page)
    clean = g.paged_attention(**x, max_q=new, window=150, sinks=9)
    P = page
    for n, kv in enumerate((1000, 801)):
        for t in range(9, kv - 150):
            pg = int(x["page_table"][n, t // P])
            x["k_cache"][pg, t % P], x["v_cache"][pg, t % P] = float("nan"), float("nan")
    assert torch.equal(g.paged_attention(**x, max_q=new, window=150, sinks=9), clean)
    o, lse = g.paged_attention(**x, max_q=new, window=150, sinks=9, return_lse=True)
    close(o, lse, x, qs, D ** -0.5, 150, 9)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sinks_without_effect(dtype):
    """Without a window, or with one that reaches the beginning, sinks change no bit; with no sinks neither does the argument."""
    import gated_deltanet_linear_15_gb300 as g
    x, _ = make([(3, 400), (3, 70)], dtype, 64, 2, 2, 16)
    want = g.paged_attention(**x, max_q=3)
    assert torch.equal(g.paged_attention(**x, max_q=3, sinks=10), want)
    assert torch.equal(g.paged_attention(**x, max_q=3, window=1 << 30, sinks=2 ** 31 - 1), want)
    assert torch.equal(g.paged_attention(**x, max_q=3, window=100, sinks=0), g.paged_attention(**x, max_q=3, window=100))


@gpu
@pytest.mark.parametrize("seed", range(6))
def test_sinks_drawn(seed):
    import random
    import gated_deltanet_linear_15_gb300 as g
    r = random.Random(seed)
    D, G, page = r.choice([64, 128]), r.choice([1, 2, 5, 8]), r.choice([16, 64, 128])
    seqs = [(q, max(q, r.randint(1, 1500))) for q in (r.choice([0, 1, 1, r.randint(1, 90)]) for _ in range(5))]
    window, sinks = r.randint(1, 400), r.randint(1, 300)
    x, qs = make(seqs, r.choice([BF, BF, F32]), D, 2, G, page, seed=seed)
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), window=window, sinks=sinks, return_lse=True)
    close(o, lse, x, qs, D ** -0.5, window, sinks)


# ------------------------------------------------------------------ shared prefixes
def shared(groups, dtype, D, Hkv, G, page, seed=0, wide=True):
    """groups: (prefix, [(new, own) tokens of each sequence, own ones with the new]); a group's sequences name the same pages for
    its prefix, up to the end of its last page.  Slots that hold no token are NaN.  wide: the table has room for so many tokens
    that sharing could save a lot, as far as the host knows, and the batch is computed in two parts."""
    gen = torch.Generator().manual_seed(seed)
    lens = [(q, pre + own) for pre, seqs in groups for q, own in seqs]
    full = [-(-pre // page) for pre, seqs in groups for _ in seqs]
    need = [max(-(-kv // page), f) for (_, kv), f in zip(lens, full)]
    pool = sum(-(-pre // page) for pre, _ in groups) + sum(n - f for n, f in zip(need, full)) + 3
    perm, at = torch.randperm(pool, generator=gen).tolist(), 0
    width = max(need) + 1
    if wide and len(lens) > len(groups):
        width = max(width, -(-130 * 10 ** 6 // ((len(lens) - len(groups)) * page * Hkv * D * 4)))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    kc, vc = torch.full((pool, page, Hkv, D), math.nan), torch.full((pool, page, Hkv, D), math.nan)
    n = 0
    for pre, seqs in groups:
        head = perm[at:at + -(-pre // page)]
        at += len(head)
        for q, own in seqs:
            own_pages = perm[at:at + need[n] - len(head)]
            at += len(own_pages)
            row = head + own_pages
            table[n, :len(row)] = torch.tensor(row, dtype=torch.int32)
            kv = pre + own
            for j, pg in enumerate(row):  # a shared page that is not full goes on with the longest sequence's tokens
                m = min(page, max(0, kv - j * page))
                fresh = kc[pg, :m].isnan()
                kc[pg, :m] = torch.where(fresh, torch.randn(m, Hkv, D, generator=gen), kc[pg, :m])
                vc[pg, :m] = torch.where(fresh, torch.randn(m, Hkv, D, generator=gen), vc[pg, :m])
            n += 1
    qs = [q for q, _ in lens]
    cu = [0]
    for _, seqs in groups:
        cu.append(cu[-1] + len(seqs))
    x = dict(q=torch.randn(sum(qs), Hkv * G, D, generator=gen).to(DEV, dtype), k_cache=kc.to(DEV, dtype), v_cache=vc.to(DEV, dtype),
             page_table=table.to(DEV), kv_lens=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=DEV))
    return x, qs, torch.tensor([p for p, _ in groups], dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)


PREFIX = [
    # groups, dtype, D, Hkv, G, page
    ([(32, [(1, 1), (1, 1)])], BF, 128, 1, 1, 16),
    ([(96, [(1, 5), (1, 30), (1, 1)])], BF, 64, 2, 3, 16),
    ([(1000, [(1, 17)] * 4)], BF, 128, 2, 4, 16),                    # the prefix ends inside a page
    ([(700, [(1, 40)] * 40)], BF, 128, 2, 4, 64),                    # 160 rows: the chunk kernel for the prefix
    ([(2000, [(1, 1 + i) for i in range(70)])], BF, 64, 1, 4, 32),   # 280 rows: two tiles
    ([(513, [(5, 5 + i) for i in range(9)]), (0, [(1, 30), (2, 2)]), (64, [(3, 100)]), (129, [(1, 1)] * 3)], BF, 128, 2, 4, 16),
    ([(300, [(70, 90), (1, 3), (0, 5), (200, 200)])], BF, 128, 1, 2, 64),   # the chunk kernel for both
    ([(4096, [(1, 64)] * 2)], BF, 128, 8, 1, 256),
    ([(250, [(1, 7), (4, 9)]), (90, [(1, 1)] * 5)], F32, 64, 2, 2, 16),
    ([(1500, [(2, 33)] * 12)], F32, 128, 1, 4, 32),
    ([(77, [(30, 60)] * 3)], F32, 64, 1, 1, 16),
]


@gpu
@pytest.mark.parametrize("groups,dtype,D,Hkv,G,page", PREFIX)
@pytest.mark.parametrize("wide", [True, False])
def test_prefix(groups, dtype, D, Hkv, G, page, wide):
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu_seqs = shared(groups, dtype, D, Hkv, G, page, seed=D + len(groups), wide=wide)
    per = [sum(q for q, _ in seqs) for _, seqs in groups]
    args = dict(prefix_lens=pre, cu_seqs=cu_seqs, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), max_group=max(per), return_lse=True)
    o, lse = g.prefix_attention(**x, **args)
    close(o, lse, x, qs, D ** -0.5)
    again = g.prefix_attention(**x, **args)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    args.update(max_q=0, max_group=0)
    o, lse = g.prefix_attention(**x, **args)  # perhaps other kernels
    close(o, lse, x, qs, D ** -0.5)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 5], [0, 0], [10000, 10000], [48, 200], [-3, 2 ** 31 - 1]])
def test_prefix_of_any_length(dtype, lens):
    """Shorter than what is shared, negative, or longer than what some sequence has cached: the same attention."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, _, cu_seqs = shared([(48, [(1, 1), (3, 40), (2, 2)]), (200, [(1, 9), (1, 1)])], dtype, 64, 2, 2, 16)
    o, lse = g.prefix_attention(**x, prefix_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqs=cu_seqs,
                                cu_q=ref.lens_to_cu(qs, DEV), return_lse=True)
    close(o, lse, x, qs, 64 ** -0.5)  # what the shortest sequence of a group had cached are the 48 or 200 shared tokens


@gpu
def test_sequences_outside_groups_and_equal_groups():
    """Sequences that cu_seqs leaves out share nothing; without cu_seqs groups are of one size; without cu_q so are the new
    tokens."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(0, [(2, 50)]), (320, [(2, 9)] * 4), (0, [(2, 2), (2, 70)])], BF, 128, 2, 4, 16)
    o, lse = g.prefix_attention(**x, prefix_lens=pre[1:2], cu_seqs=cu[1:3].contiguous(), return_lse=True)
    close(o, lse, x, qs, 128 ** -0.5)
    x, qs, pre, _ = shared([(320, [(2, 9)] * 4), (80, [(2, 30)] * 4)], BF, 128, 2, 4, 16)
    o, lse = g.prefix_attention(**x, prefix_lens=pre, return_lse=True)
    close(o, lse, x, qs, 128 ** -0.5)


@gpu
def test_prefix_empty_batches_and_untouched_rows():
    """No new tokens at all, a group without any, and rows that no sequence names, which keep what they held."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(100, [(0, 5)] * 3), (64, [(1, 2), (0, 1), (2, 4)])], BF, 64, 1, 2, 16)
    cu_q = ref.lens_to_cu(qs, DEV)
    o, lse = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, cu_q=cu_q, return_lse=True)
    close(o, lse, x, qs, 64 ** -0.5)
    more = dict(x, q=torch.cat([x["q"], torch.randn_like(x["q"])]))
    out = torch.full_like(more["q"], 5.0)
    assert g.prefix_attention(**more, prefix_lens=pre, cu_seqs=cu, cu_q=cu_q, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out[:3], o) and (out[3:] == 5).all()
    none = dict(x, q=x["q"][:0])
    assert g.prefix_attention(**none, prefix_lens=pre, cu_seqs=cu, cu_q=torch.zeros_like(cu_q)).shape == (0, 2, 64)


@gpu
@pytest.mark.parametrize("cu_seqs,cu_q", [([0, 3, 1, 6], [0, 1, 2, 3, 4, 5, 6]), ([5, 2, 9, -4], [0, 1, 2, 3, 4, 5, 6]),
                                          ([0, 6, 6, 6], [0, 4, 1, 6, 0, 6, 6]), ([0, 2, 4, 6], [0, 6, 0, 6, 0, 6, 0])])
def test_any_groups_end_within_the_rows(cu_seqs, cu_q):
    """Entries out of order or range: whatever is computed, the call ends and its status is clean."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, _, _ = shared([(100, [(1, 9)] * 6)], BF, 128, 2, 20, 16)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    how = dict(prefix_lens=ints([100, 50, 2 ** 31 - 1]), cu_seqs=ints(cu_seqs), cu_q=ints(cu_q))
    g.prefix_attention(**x, **how, workspace=ws)
    assert g.prefix_attention_status(**x, **how, workspace=ws) == 0


@gpu
@pytest.mark.parametrize("dtype,G,groups", [(BF, 4, 1), (BF, 1, 3), (F32, 2, 2), (BF, 40, 2)])
def test_prefix_right_behind_its_inputs(dtype, G, groups):
    """Queries, caches, lengths and prefixes written by the kernels just before, call after call with one workspace: the bits of
    calls that had the GPU to themselves."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(400 + 16 * k, [(1, 30 + 7 * i) for i in range(12)]) for k in range(groups)], dtype, 128, 2, G, 16)
    ws = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    gen = torch.Generator().manual_seed(9)
    drawn = [dict(q=torch.randn(x["q"].shape, generator=gen).to(DEV, dtype), less=k % 3, shift=16 * (k % 5)) for k in range(12)]
    lens, fixed = x["kv_lens"].clone(), pre.clone()
    caches = [(x["k_cache"] * (1 + 0.1 * k), x["v_cache"] * (1 - 0.1 * k)) for k in range(3)]

    def call(d, k):
        x["q"].copy_(d["q"])
        torch.sub(lens, d["less"], out=x["kv_lens"])
        torch.sub(fixed, d["shift"], out=pre)
        for name, new in zip(("k_cache", "v_cache"), caches[k % 3]):
            x[name].copy_(new)
        return g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, return_lse=True, workspace=ws)

    want = []
    for k, d in enumerate(drawn):
        want.append(call(d, k))
        torch.cuda.synchronize()
    for _ in range(8):
        got = [call(d, k) for k, d in enumerate(drawn)]
        for p, q in zip(got, want):
            assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@gpu
def test_prefix_capture_and_workspaces():
    """Replayed from a graph over new queries and lengths, and on another stream with a workspace of its own: the same bits."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(500, [(1, 20 + i) for i in range(12)])], BF, 128, 2, 4, 16)
    graph = torch.cuda.CUDAGraph()
    g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu)
    with torch.cuda.graph(graph):
        o, lse = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, return_lse=True)
    x["q"].copy_(torch.randn_like(x["q"]))
    x["kv_lens"].sub_(3)
    graph.replay()
    close(o, lse, x, qs, 128 ** -0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        got = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, workspace=ws)
    side.synchronize()
    assert torch.equal(got, o)


def _shape(**kw):
    s = _lib.GdnPagedShape()
    s.num_seqs, s.total_q, s.num_heads, s.num_kv_heads, s.head_dim = 64, 64, 8, 2, 128
    s.page_size, s.num_pages, s.max_pages, s.dtype, s.max_q, s.scale, s.table_stride = 64, 100, 200, _lib.GDN_BF16, 1, 0.1, 200
    s.q_tok, s.q_head, s.o_tok, s.o_head = 1024, 128, 1024, 128
    s.k_page = s.v_page = 64 * 256
    s.k_tok = s.v_tok = 256
    s.k_head = s.v_head = 128
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@gpu
@pytest.mark.parametrize("new,dtype", [(1, BF), (40, BF), (3, F32)])
def test_status_of_an_expired_wait(lib, new, dtype):
    """A call that is made to wait, with a short limit, for what never comes returns, leaves 4 and no output."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(700, [(new, 20 + new)] * 12)], dtype, 128, 2, 4, 16)
    ws, out = torch.empty(256 << 20, dtype=torch.uint8, device=DEV), torch.full_like(x["q"], 7.0)
    s = _shape(num_seqs=12, total_q=12 * new, page_size=16, num_pages=x["k_cache"].shape[0], max_pages=x["page_table"].shape[1], max_q=new,
               table_stride=x["page_table"].shape[1], dtype=_lib.GDN_BF16 if dtype == BF else _lib.GDN_FP32, k_page=16 * 256, v_page=16 * 256)
    p, st = lambda t: t.data_ptr(), torch.cuda.current_stream().cuda_stream  # noqa: E731

    def call():
        return lib.gdn_prefix_attn_fwd(ctypes.byref(s), 1, 0, p(x["q"]), p(x["k_cache"]), p(x["v_cache"]), p(x["page_table"]), None,
                                       p(x["kv_lens"]), p(cu), p(pre), p(out), None, p(ws), ws.numel(), st)

    s.reserved = _lib.GDN_DEBUG_WAIT_TIMEOUT - (1 << 32)
    assert call() == 0
    assert lib.gdn_prefix_attn_status(ctypes.byref(s), 1, 0, p(ws), st) == 4 and (out == 7).all()
    s.reserved = 0
    assert call() == 0 and lib.gdn_prefix_attn_status(ctypes.byref(s), 1, 0, p(ws), st) == 0
    assert torch.equal(out, g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, max_q=new, scale=0.1))


# ------------------------------------------------------------------ refusals
@gpu
def test_binding_refuses():
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(100, [(1, 9)] * 4)], BF, 64, 2, 2, 16)
    for call in (lambda: g.paged_attention(**x, window=5, sinks=-1), lambda: g.paged_attention(**x, window=5, sinks=2 ** 31),
                 lambda: g.prefix_attention(**x, prefix_lens=pre.long()), lambda: g.prefix_attention(**x, prefix_lens=pre[None]),
                 lambda: g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu[:1]), lambda: g.prefix_attention(**x, prefix_lens=pre[:0]),
                 lambda: g.prefix_attention(**x, prefix_lens=torch.cat([pre] * 3)), lambda: g.prefix_attention(**x, prefix_lens=pre.cpu()),
                 lambda: g.prefix_attention(**x, prefix_lens=torch.cat([pre] * 5), cu_seqs=torch.cat([cu] * 3)),
                 lambda: g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, max_group=-1),
                 lambda: g.prefix_attention(**x, prefix_lens=pre, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def test_c_entry_refuses(lib):
    p = {n: 0x10000 * (i + 1) for i, n in enumerate(("q", "k", "v", "table", "cu", "kv", "seqs", "pre", "o", "lse"))}

    def call(groups=4, group=0, ws=0x1000000, nbytes=1 << 40, shape=None, **kw):
        a = dict(p, **kw)
        return lib.gdn_prefix_attn_fwd(ctypes.byref(shape or _shape()), groups, group, *a.values(), ws, nbytes, None)

    need = lib.gdn_prefix_attn_workspace_size(ctypes.byref(_shape()), 4, 0)
    assert need > lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape()))
    for n in ("q", "k", "v", "table", "kv", "pre", "o"):
        assert call(**{n: None}) == 1, n
    assert call(o=p["q"]) == 1 and call(ws=0x1000010) == 1 and call(ws=None) == 3 and call(nbytes=need - 1) == 3
    assert call(groups=0) == 1 and call(groups=65) == 1 and call(group=-1) == 1 and call(groups=3, seqs=None) == 1
    assert call(shape=_shape(window=5)) == 2 and call(shape=_shape(head_dim=96)) == 2 and call(shape=_shape(reserved=1)) == 1
    assert call(shape=_shape(total_q=0)) == 0
    assert lib.gdn_prefix_attn_workspace_size(ctypes.byref(_shape(window=5)), 4, 0) == 0
    big = _shape(num_seqs=2 ** 31 - 1, total_q=2 ** 28, max_pages=2 ** 31 - 1, table_stride=2 ** 31 - 1)
    assert lib.gdn_prefix_attn_workspace_size(ctypes.byref(big), 1, 0) > 2 ** 40
    s = _shape(window=100)
    a = [p[n] for n in ("q", "k", "v", "table", "cu", "kv", "o", "lse")]
    assert lib.gdn_paged_attn_sinks_fwd(ctypes.byref(s), -1, *a, 0x1000000, 1 << 40, None) == 1
    assert lib.gdn_paged_attn_sinks_fwd(ctypes.byref(s), 4, *a, 0x1000000, 100, None) == 3
    assert lib.gdn_paged_attn_sinks_fwd(ctypes.byref(_shape(total_q=0)), 4, *a, 0x1000000, 100, None) == 0
