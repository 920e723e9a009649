"""Attention over a paged cache against the definition in 64 bits, and its refusals.

Bounds.  bf16: the products are exact and the sums fp32; the weights are rounded to bf16 before the second product
(at most 2^-8 of each, so 2^-8 sum p |v|) and the output once (2^-8 |o|); 5 % on top for fp32 sums and the power of two.
fp32: each product loses at most 2^-20 of its magnitude (three TF32 parts), the logits sum D of them:
|ds| <= 2^-20 scale sum |q k|, which is below 8e-6 for the N(0, 1) inputs here; a weight is off by at most twice that,
and the second product adds 2^-20: 3e-5 sum p |v| holds with room for fp32 sums.  lse: |ds| plus fp32 rounding."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests import block_ref as ref

gpu = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def make(seqs, dtype, D, Hkv, G, page, seed=0, head_major=False, spare=3, dev=DEV, fill=float("nan")):
    """seqs: (new, cached) tokens of each.  Every slot that holds no token is `fill` (NaN)."""
    gen = torch.Generator().manual_seed(seed)
    qs, ks = [s[0] for s in seqs], [s[1] for s in seqs]
    need = [-(-k // page) for k in ks]
    width = max(max(need), 1) + 1
    perm = torch.randperm(sum(need) + spare, generator=gen)
    shape = (sum(need) + spare, Hkv, page, D) if head_major else (sum(need) + spare, page, Hkv, D)
    kc, vc = torch.full(shape, fill), torch.full(shape, fill)
    if head_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = torch.full((len(seqs), width), -1, dtype=torch.int32)
    at = 0
    for n, k in enumerate(ks):
        for j in range(need[n]):
            pg = int(perm[at])
            at += 1
            table[n, j] = pg
            m = min(page, k - j * page)
            kc[pg, :m], vc[pg, :m] = torch.randn(m, Hkv, D, generator=gen), torch.randn(m, Hkv, D, generator=gen)
    q = torch.randn(sum(qs), Hkv * G, D, generator=gen)
    kc, vc = kc.to(dev, dtype), vc.to(dev, dtype)  # .to keeps the head-major strides
    return dict(q=q.to(dev, dtype), k_cache=kc, v_cache=vc, page_table=table.to(dev),
                kv_lens=torch.tensor(ks, dtype=torch.int32, device=dev)), qs


def close(o, lse, x, qs, scale, window=0):
    ro, rl, mag = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["kv_lens"], qs, scale, window)
    o, lse = o.cpu().double(), lse.cpu().double()
    if x["q"].dtype == torch.bfloat16:
        tol = 1.05 * 2 ** -8 * (ro.abs() + mag) + 1e-30
    else:
        tol = 3e-5 * mag + 1e-30
    assert torch.isfinite(o).all()
    bad = (o - ro).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((o - ro).abs() / tol).max():.2f} of the bound"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (o[empty] == 0).all()
    if (~empty).any():
        assert ((lse - rl)[~empty].abs() <= 1e-5 + 1e-6 * rl[~empty].abs()).all()


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    # (new, cached) tokens, dtype, D, Hkv, G, page, window
    ([(1, 1)], BF, 128, 1, 1, 16, 0),
    ([(1, 17)], BF, 64, 2, 3, 16, 0),
    ([(1, 100), (1, 1), (1, 64), (1, 333)], BF, 128, 2, 4, 16, 0),
    ([(1, 1000), (1, 129)], BF, 64, 1, 16, 64, 0),
    ([(4, 300), (4, 4), (4, 67)], BF, 128, 2, 4, 32, 0),
    ([(5, 257), (0, 40), (1, 40), (3, 3)], BF, 128, 1, 6, 128, 0),
    ([(70, 200), (1, 90), (33, 33)], BF, 128, 2, 2, 16, 0),
    ([(300, 300)], BF, 64, 1, 4, 64, 0),
    ([(130, 1000)], BF, 128, 1, 1, 256, 0),
    ([(1, 500), (40, 333)], BF, 128, 2, 4, 16, 37),
    ([(1, 500), (200, 400)], BF, 64, 1, 8, 32, 16),
    ([(1, 3000)], BF, 128, 1, 2, 64, 1),
    ([(9, 4), (2, 0), (1, 7)], BF, 128, 2, 4, 16, 0),        # fewer cached tokens than new ones: the first see nothing
    ([(140, 12)], BF, 128, 1, 2, 16, 0),
    ([(1, 0), (1, 0)], BF, 64, 1, 1, 16, 0),
    ([(1, 1)], F32, 64, 1, 1, 16, 0),
    ([(1, 300), (1, 77)], F32, 128, 2, 4, 32, 0),
    ([(40, 100), (1, 50), (0, 9), (17, 17)], F32, 64, 2, 3, 16, 0),
    ([(90, 333)], F32, 128, 1, 2, 64, 50),
    ([(3, 1)], F32, 64, 2, 2, 16, 0),
]


@gpu
@pytest.mark.parametrize("seqs,dtype,D,Hkv,G,page,window", CASES)
@pytest.mark.parametrize("hint", [True, False])
def test_matches_definition(seqs, dtype, D, Hkv, G, page, window, hint):
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make(seqs, dtype, D, Hkv, G, page, seed=len(seqs) + D + G)
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs) if hint else 1, window=window, return_lse=True)
    close(o, lse, x, qs, D ** -0.5, window)


@gpu
@pytest.mark.parametrize("dtype,D,G,q", [(BF, 128, 4, 1), (BF, 64, 2, 40), (F32, 64, 2, 3), (BF, 128, 4, 150)])
def test_strided_inputs_and_scale(dtype, D, G, q):
    """q as a slice of a wider projection, head-major caches, a table that is a slice, an output view, another scale, and
    equal new lengths without cu_q."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(q, q + 31), (q, q + 160)], dtype, D, 2, G, 32, seed=3, head_major=True)
    T, Hq = x["q"].shape[:2]
    assert x["k_cache"].stride(1) == D
    wide = torch.full((T, Hq + 4, D), float("nan"), dtype=dtype, device=DEV)
    wide[:, 2:2 + Hq] = x["q"]
    x["q"] = wide[:, 2:2 + Hq]
    tab = torch.full((2, x["page_table"].shape[1] + 5), 1 << 30, dtype=torch.int32, device=DEV)
    tab[:, 1:-4] = x["page_table"]
    x["page_table"] = tab[:, 1:-4]
    out = torch.full((T, 2 * Hq, D), 7.0, dtype=dtype, device=DEV)
    o, lse = g.paged_attention(**x, max_q=q, scale=0.31, return_lse=True, out=out[:, Hq:])
    assert (out[:, :Hq] == 7).all()
    close(o, lse, x, qs, 0.31)


@gpu
def test_long_context_is_split_and_joined():
    """A single sequence that many CTAs share, decoded and drafted, and a ragged batch; two calls agree bit for bit."""
    import gated_deltanet_linear_15_gb300 as g
    for seqs, G in (([(1, 20001)], 4), ([(4, 9999)], 8), ([(1, 5000), (1, 31), (2, 7777), (1, 0)], 2), ([(150, 4000)], 2)):
        x, qs = make(seqs, BF, 128, 1, G, 64, seed=5)
        a = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), return_lse=True)
        b = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        close(*a, x, qs, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 128)])
@pytest.mark.parametrize("page", [16, 32, 64])
def test_slices_that_end_past_their_pages(dtype, D, page):
    """17 to 32 rows per key head, whose slices may reach over two pages: one that ends with the table, one whose second
    half is a missing page (zeros), windows that begin inside a slice."""
    import gated_deltanet_linear_15_gb300 as g
    for seqs, G, window in (([(3, 97)], 8, 0), ([(3, 97), (4, 33), (2, 17)], 8, 19), ([(30, 353)], 1, 21)):
        x, qs = make(seqs, dtype, D, 2, G, page, seed=page, spare=0)
        x["page_table"] = x["page_table"][:, :-1].contiguous()
        o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), window=window, return_lse=True)
        close(o, lse, x, qs, D ** -0.5, window)
        if page == 16 and not window:
            pg = int(x["page_table"][0, 1])
            x["page_table"][0, 1] = -1
            o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), return_lse=True)
            x["page_table"][0, 1] = pg
            x["k_cache"][pg], x["v_cache"][pg] = 0, 0
            close(o, lse, x, qs, D ** -0.5)


@gpu
@pytest.mark.parametrize("N,q,dtype", [(33, 1, BF), (300, 1, BF), (300, 3, F32), (513, 1, BF), (700, 2, BF), (90, 40, BF), (600, 20, BF),
                                       (3, 1500, F32)])
def test_many_sequences(N, q, dtype):
    """Batches of every size class of the search for a CTA's share, with empty sequences and sequences without new tokens
    among them."""
    import random

    import gated_deltanet_linear_15_gb300 as g
    r = random.Random(N)
    seqs = [(r.choice([q, q, r.randint(0, q)]), r.randint(0, 70)) for _ in range(N)]
    x, qs = make(seqs, dtype, 64, 2, 1, 16, seed=N)
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=q, return_lse=True)
    close(o, lse, x, qs, 0.125)


@gpu
@pytest.mark.parametrize("seqs,Hkv,G", [
    ([(20, 3000), (20, 2500), (19, 1777), (3, 900)], 4, 4),     # a few 256-row items in many pieces, more rows than blocks
    ([(130, 1300), (200, 700), (64, 64), (90, 2222)], 8, 4),    # many items in few pieces
])
def test_joins_of_tall_items(seqs, Hkv, G):
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make(seqs, BF, 128, Hkv, G, 64, seed=Hkv)
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), return_lse=True)
    close(o, lse, x, qs, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("seqs,dtype", [([(8, 3)], BF), ([(9, 4), (1, 30)], BF), ([(140, 12), (200, 300)], BF), ([(9, 4)], F32)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 1 << 30, 40])
def test_windows_longer_than_the_context(seqs, dtype, window):
    """Also where the first queries lie before the first key."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make(seqs, dtype, 128, 1, 2, 16, seed=18)
    if window == 40:   # 40 is longer than the contexts here, and shorter than the table's row
        seqs, window = [(min(a, 40), min(b, 40)) for a, b in seqs], 40
        x, qs = make(seqs + [(1, 200)], dtype, 128, 1, 2, 16, seed=18)
        close(*g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), window=window, return_lse=True), x, qs,
              128 ** -0.5, window)
        return
    cu = ref.lens_to_cu(qs, DEV)
    o, lse = g.paged_attention(**x, cu_q=cu, max_q=max(qs), window=window, return_lse=True)
    want = g.paged_attention(**x, cu_q=cu, max_q=max(qs), return_lse=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    close(o, lse, x, qs, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("seqs,Hkv,window", [
    ([(200, 300)] * 25, 1, 16),              # items in three pieces of a block, the last rows see keys in the third only
    ([(256, 1000)] * 39, 1, 64),
    ([(256, 900), (250, 700)], 2, 20),       # a few items in many pieces
    ([(30, 800), (17, 400), (9, 1000)], 1, 12),
])
@pytest.mark.parametrize("level", [-100.0, -1000.0])
def test_joins_of_rows_that_see_nothing_in_the_first_pieces(seqs, Hkv, window, level):
    """Under a window the last rows of a tile see nothing of its first key blocks; with all logits far below zero, what they
    do see must not be measured against a maximum of zero.  Bound: the logits' fp32 sums pass |level| / scale, and each of
    their 8 steps may lose 2^-23 of 2 of that: 16 * 2^-23 |level| in a logit, twice that in a weight."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make(seqs, BF, 128, Hkv, 1, 16, seed=17, fill=0.0)
    scale = 128 ** -0.5
    a = (-level / (128 * scale)) ** 0.5
    x["q"] = (a + 0.02 * x["q"]).to(BF)
    x["k_cache"] = (-a + 0.02 * x["k_cache"]).to(BF)
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), window=window, return_lse=True)
    ro, rl, mag = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["kv_lens"], qs, scale, window)
    assert (rl < level / 2).all()
    slack = 16 * 2 ** -23 * 2 * abs(level)
    assert ((lse.cpu().double() - rl).abs() <= slack + 1e-5 + 1e-6 * rl.abs()).all()
    assert ((o.cpu().double() - ro).abs() <= 1.05 * 2 ** -8 * (ro.abs() + mag) + 2 * slack * mag).all()


@gpu
def test_peaked_and_growing_logits():
    """Logits that grow along the context (the maximum rises at every step) and by far more than fp32's exponent range
    would bear without it."""
    import gated_deltanet_linear_15_gb300 as g
    for q in (1, 140):
        x, qs = make([(q, 900)], BF, 128, 1, 2, 64, seed=7)
        P = x["k_cache"].shape[1]
        for j in range(-(-900 // P)):
            pg = int(x["page_table"][0, j])
            ramp = torch.linspace(j, j + 1, P, device=DEV)[:, None, None]
            x["k_cache"][pg] = (x["q"][-1, 0] * ramp * 0.7).to(BF)
        o, lse = g.paged_attention(**x, max_q=q, return_lse=True)
        ro, rl, mag = ref.attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["kv_lens"], qs, 128 ** -0.5)
        # the logits reach several hundred: fp32 sums are off by up to 128 * 2^-24 of their magnitude
        slack = 128 * 2 ** -24 * 128 ** -0.5 * float((x["q"].float().abs().max() ** 2) * 0.7 * 15 * 128)
        assert ((o.cpu().double() - ro).abs() <= (2.1 * 2 ** -8 + 2 * slack) * mag).all()
        assert ((lse.cpu().double() - rl).abs() <= slack + 1e-6 * rl.abs()).all()


@gpu
def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and more than 2^31 elements, its last pages in use."""
    import gated_deltanet_linear_15_gb300 as g
    pages, P, H, D = 66000, 64, 4, 128
    kc = torch.empty(pages, P, H, D, dtype=BF, device=DEV)
    vc = torch.empty(pages, P, H, D, dtype=BF, device=DEV)
    assert kc.numel() > 1 << 31
    for q in (1, 70):
        x, qs = make([(q, 300)], BF, D, H, 2, P, seed=9, spare=0)
        far = pages - 1 - torch.arange(5, device=DEV) * 3
        near = x["page_table"][0, :5].long()
        kc[far], vc[far] = x["k_cache"][near], x["v_cache"][near]
        table = far.to(torch.int32)[None].contiguous()
        o, lse = g.paged_attention(x["q"], kc, vc, table, x["kv_lens"], max_q=q, return_lse=True)
        close(o, lse, x, qs, D ** -0.5)


@gpu
def test_bad_device_data_stays_in_bounds():
    """Page numbers outside the pool count as pages of zeros, lengths are cut to the table, cu_q to the tokens."""
    import gated_deltanet_linear_15_gb300 as g
    for q in (2, 140):
        x, qs = make([(q, 200)], BF, 128, 1, 2, 64, seed=11)
        bad = dict(x, page_table=x["page_table"].clone())
        bad["page_table"][0, 1] = 1 << 30
        zero = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
        zero["k_cache"][int(x["page_table"][0, 1])] = 0
        zero["v_cache"][int(x["page_table"][0, 1])] = 0
        a, b = g.paged_attention(**bad, max_q=q), g.paged_attention(**zero, max_q=q)
        assert torch.equal(a, b)
        long = dict(x, kv_lens=torch.full_like(x["kv_lens"], 2 ** 31 - 1))
        g.paged_attention(**long, max_q=q)
        g.paged_attention(**dict(x, kv_lens=torch.full_like(x["kv_lens"], -5)), max_q=q)
        g.paged_attention(**x, cu_q=torch.tensor([-7, 10 ** 6], dtype=torch.int32, device=DEV), max_q=q)
        torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("N,T,max_q", [((1 << 18) + 2, 1 << 18, 1), (700, 3000, 1), (700, 3000, 3000)])
def test_cu_q_that_names_tokens_many_times(N, T, max_q):
    """cu_q goes to and fro, which in the first case makes more tiles than 31 bits hold: the call ends at once without touching
    anything, and the next one is right."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(1, 20)], BF, 64, 1, 1, 16)
    cu = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    cu[1::2] = T
    out = torch.full((T, 1, 64), 7.0, dtype=BF, device=DEV)
    lens, table = torch.full((N,), 20, dtype=torch.int32, device=DEV), x["page_table"].repeat(N, 1)
    g.paged_attention(torch.zeros(T, 1, 64, dtype=BF, device=DEV), x["k_cache"], x["v_cache"], table, lens, cu_q=cu, max_q=max_q,
                      out=out)
    assert (out == 7).all()
    close(*g.paged_attention(**x, max_q=1, return_lse=True), x, qs, 0.125)


@gpu
@pytest.mark.parametrize("N,q", [(5, 1), (40, 3), (3, 90)])
def test_one_table_row_for_all_sequences(N, q):
    """An expanded row is read with its stride of 0.  The rows behind it hold other pages of the pool, so that reading them
    instead would stay in bounds and show."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(q, 200 + n) for n in range(N)], BF, 128, 1, 2, 16, seed=N)
    x["kv_lens"] = torch.clamp(x["kv_lens"], max=x["kv_lens"][0])
    full = x["page_table"]
    for row in (full[:1], full[1:2]):
        want = g.paged_attention(**dict(x, page_table=row.repeat(N, 1)), max_q=q)
        assert torch.equal(g.paged_attention(**dict(x, page_table=row.expand(N, -1)), max_q=q), want)
    close(*g.paged_attention(**dict(x, page_table=full[:1].expand(N, -1)), max_q=q, return_lse=True),
          dict(x, page_table=full[:1].expand(N, -1)), qs, 128 ** -0.5)
    with pytest.raises(RuntimeError):   # rows that overlap one another
        g.paged_attention(**dict(x, page_table=full.as_strided((2, full.shape[1]), (1, 1)), kv_lens=x["kv_lens"][:2], q=x["q"][:2 * q]), max_q=q)


@gpu
def test_non_finite_values_reach_only_their_readers():
    """A NaN in one cached value of an early token reaches every query; infinities and NaN behind a window, in later
    tokens' tiles or in free slots reach none."""
    import gated_deltanet_linear_15_gb300 as g
    for q in (1, 150):
        x, qs = make([(q, 1200)], BF, 128, 1, 2, 64, seed=13)
        lo = 1200 - q - 200 + 1
        for t in range(0, lo - 1, 7):
            pg = int(x["page_table"][0, t // 64])
            x["k_cache"][pg, t % 64] = float("inf")
            x["v_cache"][pg, t % 64] = float("nan")
        o, lse = g.paged_attention(**x, max_q=q, window=200, return_lse=True)
        close(o, lse, dict(x, k_cache=x["k_cache"].nan_to_num(0, 0, 0), v_cache=x["v_cache"].nan_to_num(0, 0, 0)), qs, 128 ** -0.5, 200)
        y, qs = make([(q, 300)], BF, 128, 1, 2, 64, seed=14)
        y["v_cache"][int(y["page_table"][0, 0]), 3, 0, 5] = float("nan")
        o = g.paged_attention(**y, max_q=q)
        assert torch.isnan(o[:, :, 5]).all() and torch.isfinite(o[:, :, :5]).all()


@gpu
@pytest.mark.parametrize("seqs", [[(1, 5)], [(1, 20001)], [(40, 40)], [(150, 4000)], [(9, 4), (2, 30)], [(140, 12), (1, 0)]])
def test_scores_that_are_all_nan(seqs):
    """o and lse are NaN, whether the item is whole or cut into pieces; only a query without keys has lse = -inf."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make(seqs, BF, 128, 1, 2, 16, seed=19)
    x["k_cache"].fill_(float("nan"))
    o, lse = g.paged_attention(**x, cu_q=ref.lens_to_cu(qs, DEV), max_q=max(qs), return_lse=True)
    blind = torch.cat([torch.arange(k - q, k) < 0 for q, k in seqs])
    assert torch.isnan(o[~blind]).all() and torch.isnan(lse[~blind]).all()
    assert (o[blind] == 0).all() and (lse[blind] == -math.inf).all()


NANS = [0x7fffffff, 0x7fc00000, 0x7f800001, 0xffffffff, 0xff800001]   # the first is what fp32 arithmetic makes on the GPU


def _bits(u):
    return torch.tensor([u - (1 << 32) if u >> 31 else u], dtype=torch.int32, device=DEV).view(torch.float32)


@gpu
@pytest.mark.parametrize("nan", NANS + [None])
@pytest.mark.parametrize("D,G,q", [(64, 1, 1), (64, 2, 20), (128, 1, 1), (128, 2, 20)])
def test_fp32_nan_reaches_its_readers(nan, D, G, q):
    """Every bit pattern of a NaN, and one that the GPU computes, in a value, a key and a query."""
    import gated_deltanet_linear_15_gb300 as g
    nan = _bits(nan) if nan else torch.full((1,), math.inf, device=DEV) - math.inf
    x, qs = make([(q, 300)], F32, D, 1, G, 64, seed=20)
    clean = g.paged_attention(**x, max_q=q)
    pg = int(x["page_table"][0, 1])
    y = dict(x, v_cache=x["v_cache"].clone())
    y["v_cache"][pg, 5, 0, 7] = nan
    o = g.paged_attention(**y, max_q=q)
    assert torch.isnan(o[:, :, 7]).all()
    o[:, :, 7] = clean[:, :, 7]
    assert torch.equal(o, clean)
    y = dict(x, k_cache=x["k_cache"].clone())
    y["k_cache"][pg, 5, 0, D - 3] = nan
    o, lse = g.paged_attention(**y, max_q=q, return_lse=True)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    y = dict(x, q=x["q"].clone())
    y["q"][q - 1, G - 1, 9] = nan
    o, lse = g.paged_attention(**y, max_q=q, return_lse=True)
    assert torch.isnan(o[q - 1, G - 1]).all() and torch.isnan(lse[q - 1, G - 1])
    o[q - 1, G - 1] = clean[q - 1, G - 1]
    assert torch.equal(o, clean)


@gpu
@pytest.mark.parametrize("D,q", [(64, 1), (128, 1), (128, 30)])
def test_fp32_largest_values(D, q):
    """The largest finite values of either sign do not become infinite on the way, and infinities are as good as any value.  All queries see one key, so o is its
    value row (weight 1, the three parts of a product leave 2^-21); then keys near the top with queries of 2^-96 and a scale that undo
    them (parts below 2^-126 would lose their low bits)."""
    import gated_deltanet_linear_15_gb300 as g
    top = float(torch.finfo(F32).max)
    x, qs = make([(q, q)], F32, D, 1, 1, 64, seed=21, fill=0.0)
    v = torch.tensor([top, -top, top * (1 - 2.0 ** -13), 3.3e38, 1.0, -2.5, 1e-30, 0.0], device=DEV).repeat(D // 8)
    x["v_cache"][:] = v
    o = g.paged_attention(**x, max_q=q, window=1)
    assert torch.isfinite(o).all() and ((o - v).abs() <= 2.0 ** -20 * v.abs()).all()
    for inf in (math.inf, -math.inf):   # an infinite value, and a key that is infinitely far away
        y, qs = make([(q, 50)], F32, D, 1, 1, 64, seed=23)
        want = g.paged_attention(**y, max_q=q)
        pg = int(y["page_table"][0, 0])
        y["v_cache"][pg, 3, 0, 6] = inf
        o = g.paged_attention(**y, max_q=q)
        assert (o[:, :, 6] == inf).all()
        o[:, :, 6] = want[:, :, 6]
        assert torch.equal(o, want)
        y["q"][..., 5] = -1.7
        y["k_cache"][pg, 3, 0, 5], y["v_cache"][pg, 3, 0, 6] = math.inf, 0.25
        o, lse = g.paged_attention(**y, max_q=q, return_lse=True)
        y["k_cache"][pg, 3, 0, 5] = 1e4      # 1e4 * 1.7 / sqrt(D) below the others: a weight of zero too
        assert torch.isfinite(o).all() and torch.equal(o, g.paged_attention(**y, max_q=q))
    x, qs = make([(q, 50)], F32, D, 1, 1, 64, seed=22, fill=0.0)
    k, qq = x["k_cache"].clone(), x["q"].clone()
    k[..., 3], qq[..., 3] = top, 2.0 ** -96
    k[..., 4], qq[..., 4] = -top, 1.3 * 2.0 ** -96
    k[..., :3], k[..., 5:] = k[..., :3] * 2.0 ** 31, k[..., 5:] * 2.0 ** 31
    x["k_cache"], x["q"] = k, qq
    close(*g.paged_attention(**x, max_q=q, scale=D ** -0.5 * 2.0 ** -31, return_lse=True), x, qs, D ** -0.5 * 2.0 ** -31)


@gpu
def test_runs_on_the_current_stream():
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(1, 3000)], BF, 128, 2, 4, 64, seed=15)
    want = g.paged_attention(**x, max_q=1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = {k: v.clone() for k, v in x.items()}
        got = g.paged_attention(**y, max_q=1)
    side.synchronize()
    assert torch.equal(got, want)


@gpu
def test_captured_in_a_graph():
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(1, 700), (1, 20)], BF, 128, 2, 4, 64, seed=16)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x["q"])
    g.paged_attention(**x, max_q=1, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.paged_attention(**x, max_q=1, out=out, workspace=ws)
    x["kv_lens"][0] -= 100  # the graph reads the lengths of the replay
    x["q"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, g.paged_attention(**x, max_q=1))


def _raw(x, o, ws, q, **kw):
    """The C entry's arguments for a batch of equal new lengths."""
    s = _lib.GdnPagedShape()
    n, (t, hq, d), kc, vc = x["kv_lens"].numel(), x["q"].shape, x["k_cache"], x["v_cache"]
    s.num_seqs, s.total_q, s.num_heads, s.num_kv_heads, s.head_dim, s.page_size = n, t, hq, kc.shape[2], d, kc.shape[1]
    s.num_pages, s.max_pages, s.table_stride = kc.shape[0], x["page_table"].shape[1], x["page_table"].stride(0)
    s.dtype, s.max_q, s.scale = _lib.GDN_BF16 if x["q"].dtype == BF else _lib.GDN_FP32, q, d ** -0.5
    (s.q_tok, s.q_head), (s.o_tok, s.o_head) = x["q"].stride()[:2], o.stride()[:2]
    (s.k_page, s.k_tok, s.k_head), (s.v_page, s.v_tok, s.v_head) = kc.stride()[:3], vc.stride()[:3]
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s), [t.data_ptr() for t in (x["q"], kc, vc, x["page_table"])] + [None, x["kv_lens"].data_ptr(), o.data_ptr(),
                                                                                        None, ws.data_ptr(), ws.numel()]


@gpu
@pytest.mark.parametrize("q,dtype", [(1, BF), (40, BF), (3, F32)])
def test_status_of_a_clean_call_and_of_an_expired_wait(lib, q, dtype):
    """A call that is made to wait, with a short limit, for what never comes returns and leaves 4; the next call is clean."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(q, 300), (q, 77 + q)], dtype, 128, 2, 2, 16, seed=q)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    args = (x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["kv_lens"])
    o, lse = g.paged_attention(**x, max_q=q, return_lse=True, workspace=ws)
    assert g.paged_attention_status(*args, ws, max_q=q) == 0
    close(o, lse, x, qs, 128 ** -0.5)
    stream = torch.cuda.current_stream().cuda_stream
    out = torch.full_like(o, 7.0)
    ws.fill_(255)
    shape, raw = _raw(x, out, ws, q, reserved=_lib.GDN_DEBUG_WAIT_TIMEOUT - (1 << 32))
    assert lib.gdn_paged_attn_fwd(shape, *raw, stream) == 0
    torch.cuda.synchronize()
    word = lib.gdn_paged_attn_status(shape, ws.data_ptr(), stream)
    assert word == 4 and g.gdn_device_status_code(word) == _lib.GDN_ERR_TIMEOUT and (out == 7).all()
    assert g.paged_attention_status(*args, ws, max_q=q) == 4
    assert torch.equal(g.paged_attention(**x, max_q=q, workspace=ws), o)
    assert g.paged_attention_status(*args, ws, max_q=q) == 0


@gpu
def test_workspaces_too_small_are_refused(lib):
    """Both calls name the bytes that are needed, instead of working with other memory or reading behind the tensor."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(1, 300)], BF, 128, 2, 2, 16)
    args = (x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["kv_lens"])
    need = lib.gdn_paged_attn_workspace_size(_raw(x, x["q"], x["q"], 1)[0])
    ws = torch.zeros(2 * need, dtype=torch.uint8, device=DEV)
    for bad in (ws[:need - 1], ws[:0], ws[::2], ws.cpu()):
        with pytest.raises(ValueError, match="workspace"):
            g.paged_attention(**x, max_q=1, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            g.paged_attention_status(*args, bad, max_q=1)
    with pytest.raises(RuntimeError, match="32-byte"):
        g.paged_attention(**x, max_q=1, workspace=ws[16:])
    want = g.paged_attention(**x, max_q=1)
    assert torch.equal(g.paged_attention(**x, max_q=1, workspace=ws[:need]), want)
    assert g.paged_attention_status(*args, ws[:need], max_q=1) == 0


@gpu
@pytest.mark.parametrize("change", [
    dict(q=lambda t: t.half()), dict(q=lambda t: t[:, :3]), dict(q=lambda t: t.cpu()), dict(kv_lens=lambda t: t.long()),
    dict(page_table=lambda t: t[:, ::2]), dict(page_table=lambda t: t.long()), dict(k_cache=lambda t: t[..., :64]),
    dict(v_cache=lambda t: t.float()), dict(q=lambda t: t[..., :100]), dict(kv_lens=lambda t: t[:1]),
])
def test_binding_refuses(change):
    import gated_deltanet_linear_15_gb300 as g
    x, qs = make([(1, 20), (1, 30)], BF, 128, 2, 2, 16)
    for k, f in change.items():
        x[k] = f(x[k])
    with pytest.raises((ValueError, RuntimeError)):
        g.paged_attention(**x, max_q=1)


# ------------------------------------------------------------------ refusals of the C entry point (no GPU needed)
def _shape(**kw):
    s = _lib.GdnPagedShape()
    s.num_seqs, s.total_q, s.num_heads, s.num_kv_heads, s.head_dim = 2, 4, 8, 2, 128
    s.page_size, s.num_pages, s.max_pages, s.dtype, s.max_q, s.scale, s.table_stride = 16, 100, 10, _lib.GDN_BF16, 2, 0.1, 10
    s.q_tok, s.q_head, s.o_tok, s.o_head = 1024, 128, 1024, 128
    s.k_page = s.v_page = 16 * 256
    s.k_tok = s.v_tok = 256
    s.k_head = s.v_head = 128
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call(lib, s, ws=1 << 40, **p):
    a = dict(q=0x10000, k=0x10000, v=0x10000, table=0x10000, cu=0x10000, kv=0x10000, o=0x10000, lse=None, w=0x10000)
    a.update(p)
    return lib.gdn_paged_attn_fwd(ctypes.byref(s), a["q"], a["k"], a["v"], a["table"], a["cu"], a["kv"], a["o"], a["lse"],
                                  a["w"], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(num_heads=7), 1), (dict(num_kv_heads=0), 1), (dict(dtype=5), 1),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=8192), 2), (dict(num_pages=0), 1), (dict(total_q=-1), 1),
    (dict(window=-1), 1), (dict(max_q=-1), 1), (dict(scale=math.inf), 1), (dict(reserved=1), 1), (dict(q_tok=1020), 1),
    (dict(k_head=-128), 1), (dict(v_tok=4), 1), (dict(table_stride=9), 1), (dict(total_q=1 << 30), 2),
])
def test_c_entry_refuses_shapes(lib, kw, code):
    s = _shape(**kw)
    assert _call(lib, s) == code
    assert lib.gdn_last_error_string() != b""
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(s)) == 0


def test_plan_of_the_largest_counts(lib):
    """2^31 - 1 tokens in a few sequences take the kernel, and the scratch memory, of other long chunks; in as many sequences
    as tokens those of a decode step."""
    def need(t, n):
        return lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(num_heads=2, total_q=t, num_seqs=n, max_q=0)))

    most = 2 ** 31 - 1
    assert need(most, 2) == need(1 << 20, 2) > 0
    assert need(most, most) == need(8, 8) > 0


def test_c_entry_knows_the_debug_hook(lib):
    hook = _lib.GDN_DEBUG_WAIT_TIMEOUT - (1 << 32)
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(reserved=hook))) > 0
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(reserved=hook + 1))) == 0
    s = _shape(reserved=hook, rot=128, table_rows=10)
    assert lib.gdn_rotary_append(ctypes.byref(s), *[0x10000] * 10, None) == 1


def test_c_entry_takes_one_row_for_all(lib):
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(table_stride=0))) > 0
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(table_stride=-10))) == 0


def test_c_entry_refuses_pointers(lib):
    s = _shape()
    need = lib.gdn_paged_attn_workspace_size(ctypes.byref(s))
    assert need > 0
    for name in ("q", "k", "v", "table", "kv", "o"):
        assert _call(lib, s, **{name: None}) == 1, name
    for name in ("q", "k", "v", "o", "w"):
        assert _call(lib, s, **{name: 0x10008}) == 1, name
    assert _call(lib, s, ws=need - 1) == 3 and b"workspace" in lib.gdn_last_error_string()
    assert _call(lib, s, w=None) == 3
    assert _call(lib, _shape(total_q=5), cu=None) == 1   # not the same number for each of two sequences
    assert lib.gdn_paged_attn_fwd(None, *[0x10000] * 9, 1 << 40, None) == 1
    assert _call(lib, _shape(total_q=0)) == 0            # nothing to do: no launch


@pytest.mark.parametrize("at", [0x10004, 0x10010, 0x10030])
def test_c_entry_refuses_workspace_off_32_bytes(lib, at):
    """The records of cut items are written 32 bytes at a time."""
    for s in (_shape(), _shape(total_q=200, max_q=100)):   # the row kernel and the chunk kernel
        assert _call(lib, s, w=at) == 1 and b"32-byte" in lib.gdn_last_error_string()


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_c_entry_refuses_output_over_input(lib, name):
    """Other CTAs still read what one has written over."""
    assert _call(lib, _shape(), **{"o": 0x50000, "q": 0x20000, "k": 0x30000, "v": 0x40000, name: 0x50000}) == 1
    assert b"inputs" in lib.gdn_last_error_string()


def test_c_entry_refuses_group_beyond_16_bits(lib):
    s = _shape(num_heads=65536, num_kv_heads=1, total_q=2)
    assert _call(lib, s) == 2 and lib.gdn_paged_attn_workspace_size(ctypes.byref(s)) == 0
    assert lib.gdn_paged_attn_workspace_size(ctypes.byref(_shape(num_heads=65535, num_kv_heads=1, total_q=2))) > 0


def _can_stall(threads, programs):
    """Whether warps that run `programs`, lists of ("sync" | "arrive", barrier), can come to stand: every order is tried.  A
    barrier's generation ends when `threads[barrier]` have arrived, whoever they are; a sync leaves with its generation."""
    start = (tuple((0, False) for _ in programs), tuple(0 for _ in threads))
    seen, todo = {start}, [start]
    while todo:
        warps, count = todo.pop()
        moved = False
        for w, (pc, blocked) in enumerate(warps):
            if blocked or pc == len(programs[w]):
                continue
            moved = True
            kind, b = programs[w][pc]
            now, full = list(warps), count[b] + 32 == threads[b]
            now[w] = (pc + 1, False) if kind == "arrive" or full else (pc, True)
            if full:
                now = [(p + 1, False) if held and programs[v][p][1] == b else (p, held) for v, (p, held) in enumerate(now)]
            state = (tuple(now), tuple(0 if i == b and full else c + 32 * (i == b) for i, c in enumerate(count)))
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(pc < len(p) for (pc, _), p in zip(warps, programs)):
            return True
    return False


def test_barriers_hold_after_an_expired_wait():
    """The chunk kernel's hand-overs by hardware barrier, with the bounded waits between them run out (so that nothing else
    orders the warps): no order of the warps may leave one waiting for ever."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(_lib.__file__), "csrc", "attn_chunk_tc.cu")).read()
    op = {n: (k, int(c)) for n, k, c in
          re.findall(r"void (weights_ready|weights_wait|turn_wait|turn_give)\(int x\) \{ asm volatile\(\"bar\.(\w+) %0, (\d+);", src)}
    assert len(op) == 4 and op["weights_ready"][1] == op["weights_wait"][1] and op["turn_wait"][1] == op["turn_give"][1]
    assert _can_stall([160], [[("arrive", 0)] * 3] * 4 + [[("sync", 0)] * 3])   # the model sees a second arrival
    ready, wait = op["weights_ready"][0], op["weights_wait"][0]
    assert not _can_stall([op["weights_wait"][1]], [[(ready, 0)] * 3] * 4 + [[(wait, 0)] * 3])
    give, turn = op["turn_give"][0], op["turn_wait"][0]
    first = [(turn, 0), (give, 1)] * 4 + [(turn, 0)]
    assert not _can_stall([op["turn_wait"][1]] * 2, [first, [(give, 0)] + [(turn, 1), (give, 0)] * 4])


def test_header_and_binding_agree(lib):
    import os
    import re
    src = open(os.path.join(os.path.dirname(_lib.__file__), "..", "include", "gdn_block.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = sorted(set(re.findall(r"\b(gdn_[a-z_]+)\s*\(", src)))
    assert declared == sorted(_lib.BLOCK_EXPORTS)
    for name in declared:
        assert hasattr(lib, name)
