"""Rotary positions, their gradient and the append to a paged cache, against the definition in 64 bits.

Bounds.  A turned feature is a c - b s: two fp32 products and a sum (3 * 2^-24 of |a| + |b| at most, the table being
given), rounded once to the output type: 2^-8 of its value in bf16."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests import block_ref as ref

gpu = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def close(got, want, x):
    got = got.cpu().double()
    big = x.cpu().double().abs().amax(-1, keepdim=True)
    half = 2 ** -8 * want.abs() if x.dtype == BF else 0
    assert ((got - want).abs() <= half + 6 * 2 ** -24 * big + 1e-37).all()


def table_ref(rows, rot, base=10000.0, f=1.0):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / f)
    return torch.stack([a.cos(), a.sin()], -1)


@gpu
@pytest.mark.parametrize("rot,scaling,kw", [
    (64, None, {}), (128, "linear", dict(factor=4.0)), (32, "base", dict(factor=8.0)), (2, None, {}),
    (128, "parts", dict(factor=8.0, context=4096)), (64, None, dict(base=500000.0)),
])
def test_table(rot, scaling, kw):
    """Far positions keep fp32 accuracy: one rounding of the fp64 cos and sin."""
    import gated_deltanet_linear_15_gb300 as g
    rows = 70001
    t = g.rotary_table(rows, rot, scaling=scaling, **kw).cpu().double()
    freq, amp = g.rotary_frequencies(rot, scaling=scaling, **kw)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    want = amp * torch.stack([a.cos(), a.sin()], -1)
    assert ((t - want).abs() <= 2 ** -25 * 2 * amp).all()


def test_frequencies():
    from gated_deltanet_linear_15_gb300 import rotary_frequencies as f
    plain, amp = f(64)
    assert amp == 1.0 and plain[0] == 1.0 and torch.allclose(plain[-1], torch.tensor(10000.0 ** (-62 / 64), dtype=torch.float64))
    assert torch.allclose(f(64, scaling="linear", factor=4.0)[0] * 4, plain)
    by_base = f(64, scaling="base", factor=4.0)[0]
    assert by_base[0] == 1.0 and torch.allclose(by_base[-1] * 4, plain[-1])      # fastest kept, slowest stretched
    parts, amp = f(64, scaling="parts", factor=4.0, context=4096)
    assert parts[0] == plain[0] and torch.allclose(parts[-1] * 4, plain[-1]) and amp == 0.1 * math.log(4.0) + 1
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32]) and torch.allclose(parts[turns <= 1] * 4, plain[turns <= 1])
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.0), dict(rot=8, scaling="nope"), dict(rot=2, scaling="base"),
                dict(rot=8, scaling="parts"), dict(rot=8, base=1.0)):
        with pytest.raises(ValueError):
            f(**bad)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 1, 1, 64, 64), (7, 4, 2, 128, 64), (33, 3, 0, 128, 32), (5, 2, 1, 80, 80),
                                           (9, 2, 2, 10, 6), (300, 8, 2, 128, 128), (3, 1, 1, 2, 2), (4, 5, 1, 96, 16)])
def test_rotary(dtype, interleaved, inverse, T, Hq, Hk, D, rot):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(T + D)
    q, k = torch.randn(T, Hq, D, generator=gen).to(DEV, dtype), torch.randn(T, Hk, D, generator=gen).to(DEV, dtype)
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32)
    pos[0] = 0
    table = table_ref(4500, rot).float().to(DEV)   # positions past it are left unturned
    a, b = g.rotary(q, k if Hk else None, table, pos.to(DEV), interleaved, inverse)
    close(a, ref.rotate(q, table, pos, interleaved, inverse), q)
    if Hk:
        close(b, ref.rotate(k, table, pos, interleaved, inverse), k)
        a2, b2 = g.rotary(q.clone(), k.clone(), table, pos.to(DEV), interleaved, inverse, inplace=True)
        assert torch.equal(a, a2) and torch.equal(b, b2)


@gpu
@pytest.mark.parametrize("dtype,D", [(BF, 2048), (BF, 2064), (BF, 4096), (F32, 1024), (F32, 1032), (F32, 2048)])
def test_heads_as_wide_as_a_block_and_wider(dtype, D):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(D)
    qkv = torch.randn(3, 4, D, generator=gen).to(DEV, dtype)
    q, k, v = qkv.split([2, 1, 1], 1)
    cs, pos = table_ref(16, D).float().to(DEV), torch.tensor([4, 5, 6], dtype=torch.int32)
    want_q, want_k = ref.rotate(q, cs, pos), ref.rotate(k, cs, pos)
    a, b = g.rotary(q, k, cs, pos.to(DEV))
    close(a, want_q, q)
    close(b, want_k, k)
    kc, vc = torch.zeros(1, 16, 1, D, dtype=dtype, device=DEV), torch.zeros(1, 16, 1, D, dtype=dtype, device=DEV)
    o = g.rotary_append(q, k, v, cs, kc, vc, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                        torch.tensor([7], dtype=torch.int32, device=DEV))
    assert torch.equal(o, a) and torch.equal(kc[0, 4:7], b) and torch.equal(vc[0, 4:7], v)
    assert not kc[0, :4].any() and not kc[0, 7:].any()


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1])
def test_rotary_strided_and_unaligned(dtype, shift):
    """q and k as slices of one projection; with shift, features that start off any 16-byte boundary.  What lies between
    the heads stays as it is."""
    import gated_deltanet_linear_15_gb300 as g
    T, D = 21, 64
    gen = torch.Generator().manual_seed(4)
    flat = torch.randn(T, 8 * D + 5, generator=gen).to(DEV, dtype)
    q = flat[:, shift:shift + 4 * D].unflatten(1, (4, D))
    k = flat[:, shift + 5 * D:shift + 7 * D].unflatten(1, (2, D))
    pos = torch.arange(T, dtype=torch.int32)
    table = table_ref(64, 32).float().to(DEV)
    want_q, want_k = ref.rotate(q, table, pos), ref.rotate(k, table, pos)
    before = flat.clone()
    a, b = g.rotary(q, k, table, pos.to(DEV))
    close(a, want_q, before[:, shift:shift + 4 * D].unflatten(1, (4, D)))
    close(b, want_k, before[:, shift + 5 * D:shift + 7 * D].unflatten(1, (2, D)))
    assert torch.equal(flat, before)
    g.rotary(q, k, table, pos.to(DEV), inplace=True)
    assert torch.equal(q, a) and torch.equal(k, b)
    gap = torch.ones_like(flat, dtype=torch.bool)
    gap[:, shift:shift + 4 * D] = False
    gap[:, shift + 5 * D:shift + 7 * D] = False
    assert torch.equal(flat[gap], before[gap])


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_by_formula_and_differences(interleaved):
    """The turn is linear, so <turn(x + u) - turn(x), g> = <u, gradient> up to fp32 rounding, for any step u."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(8)
    T, D, rot = 19, 64, 48
    q, k = torch.randn(T, 4, D, generator=gen).to(DEV), torch.randn(T, 2, D, generator=gen).to(DEV)
    table, pos = table_ref(512, rot).float().to(DEV), torch.randint(0, 512, (T,), generator=gen, dtype=torch.int32).to(DEV)
    q.requires_grad_(), k.requires_grad_()
    gq, gk = torch.randn(T, 4, D, generator=gen).to(DEV), torch.randn(T, 2, D, generator=gen).to(DEV)
    a, b = g.rotary_embedding(q, k, table, pos, interleaved)
    ((a * gq).sum() + (b * gk).sum()).backward()
    close(q.grad, ref.rotate(gq, table, pos, interleaved, inverse=True), gq)
    close(k.grad, ref.rotate(gk, table, pos, interleaved, inverse=True), gk)
    u = torch.randn(T, 4, D, generator=gen).to(DEV)
    up = g.rotary(q.detach() + u, None, table, pos, interleaved)[0].double()
    lhs = float(((up - a.detach().double()) * gq.double()).sum())
    rhs = float((u.double() * q.grad.double()).sum())
    # every term is off by at most 8 roundings of values below 8; they add like a walk of T * 4 * D steps, times 10
    assert abs(lhs - rhs) <= 10 * math.sqrt(T * 4 * D) * 8 * 2 ** -24 * 8


@gpu
@pytest.mark.parametrize("with_k", [False, True])
def test_second_derivatives(with_k):
    """<gradient of q for v, u> is linear in v, and its derivative is u turned; so is that of a gradient of a gradient."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(12)
    q, v, u = (torch.randn(7, 3, 32, generator=gen).to(DEV) for _ in range(3))
    k = torch.randn(7, 1, 32, generator=gen).to(DEV).requires_grad_() if with_k else None
    table, pos = table_ref(64, 24).float().to(DEV), torch.arange(7, dtype=torch.int32, device=DEV)
    q.requires_grad_(), v.requires_grad_()
    a, b = g.rotary_embedding(q, k, table, pos)
    outs, gouts = ([a, b], [v, torch.ones_like(b)]) if with_k else ([a], [v])
    dq = torch.autograd.grad(outs, q, gouts, create_graph=True)[0]
    close(dq.detach(), ref.rotate(v.detach(), table, pos, inverse=True), v.detach())
    dv = torch.autograd.grad((dq * u).sum(), v)[0]
    close(dv, ref.rotate(u, table, pos), u)


@gpu
def test_gradient_of_queries_alone():
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(9)
    q, gq = torch.randn(7, 3, 32, generator=gen).to(DEV).requires_grad_(), torch.randn(7, 3, 32, generator=gen).to(DEV)
    table, pos = table_ref(64, 32).float().to(DEV), torch.arange(7, dtype=torch.int32, device=DEV)
    out, none = g.rotary_embedding(q, None, table, pos)
    assert none is None
    out.backward(gq)
    close(q.grad, ref.rotate(gq, table, pos, False, inverse=True), gq)


def _append_case(seqs, dtype, D, Hq, Hkv, page, head_major, seed):
    gen = torch.Generator().manual_seed(seed)
    qs, ks = [s[0] for s in seqs], [s[1] for s in seqs]
    need = [-(-max(k, 0) // page) for k in ks]
    total, width = sum(need) + 2, max(max(need), 1) + 1
    perm = torch.randperm(total, generator=gen)
    table = torch.full((len(seqs), width), -1, dtype=torch.int32)
    at = 0
    for n in range(len(seqs)):
        for j in range(need[n]):
            table[n, j] = perm[at]
            at += 1
    shape = (total, Hkv, page, D) if head_major else (total, page, Hkv, D)
    kc, vc = torch.randn(shape, generator=gen), torch.randn(shape, generator=gen)
    if head_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    qkv = torch.randn(sum(qs), Hq + 2 * Hkv, D, generator=gen)
    return qs, ks, table, kc.to(DEV, dtype), vc.to(DEV, dtype), qkv.to(DEV, dtype)


@gpu
@pytest.mark.parametrize("seqs,dtype,D,Hq,Hkv,page,rot,interleaved,head_major", [
    ([(1, 1)], BF, 128, 4, 1, 16, 128, False, False),
    ([(1, 65), (1, 17), (1, 16)], BF, 128, 8, 2, 16, 64, False, True),
    ([(40, 77), (0, 3), (1, 30), (5, 5)], BF, 64, 4, 4, 32, 64, True, False),
    ([(300, 300)], BF, 128, 8, 2, 64, 128, False, False),
    ([(9, 100), (2, 40)], F32, 64, 2, 1, 16, 16, False, True),
    ([(6, 6), (3, 9)], F32, 24, 2, 1, 16, 10, True, False),
    ([(9, 4), (4, 20)], BF, 64, 2, 2, 16, 64, False, False),     # positions below 0 are not written
])
def test_append(seqs, dtype, D, Hq, Hkv, page, rot, interleaved, head_major):
    import gated_deltanet_linear_15_gb300 as g
    qs, ks, table, kc, vc, qkv = _append_case(seqs, dtype, D, Hq, Hkv, page, head_major, seed=D + page)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    pos = torch.cat([torch.arange(b - a, b, dtype=torch.int32) for a, b in zip(qs, ks)])
    cs = table_ref(max(ks) + 1, rot).float().to(DEV)
    want_q, want_k = ref.rotate(q, cs, pos, interleaved), ref.rotate(k, cs, pos, interleaved)
    kc0, vc0 = kc.clone(), vc.clone()
    o = g.rotary_append(q, k, v, cs, kc, vc, table.to(DEV), torch.tensor(ks, dtype=torch.int32, device=DEV),
                        cu_q=ref.lens_to_cu(qs, DEV), interleaved=interleaved)
    close(o, want_q, q)
    written = torch.zeros(kc.shape[:2], dtype=torch.bool)
    t = 0
    for n, ql in enumerate(qs):
        for i in range(ql):
            p = int(pos[t])
            if p >= 0:
                pg, off = int(table[n, p // page]), p % page
                close(kc[pg, off], want_k[t], k[t])
                assert torch.equal(vc[pg, off], v[t])
                written[pg, off] = True
            t += 1
    assert torch.equal(kc[~written], kc0[~written]) and torch.equal(vc[~written], vc0[~written])


@gpu
def test_append_leaves_out_what_has_no_place():
    """Missing pages, positions past the table row or the rotary table, tokens that no sequence claims."""
    import gated_deltanet_linear_15_gb300 as g
    qs, ks, table, kc, vc, qkv = _append_case([(40, 40), (3, 3)], BF, 64, 2, 1, 16, False, seed=2)
    q, k, v = qkv.split([2, 1, 1], 1)
    cs = table_ref(20, 64).float().to(DEV)
    kc0, vc0 = kc.clone(), vc.clone()
    bad = table.clone()
    bad[0, 1], bad[0, 2] = 10 ** 6, -3
    o = g.rotary_append(q, k, v, cs, kc, vc, bad.to(DEV), torch.tensor([40, 10 ** 6], dtype=torch.int32, device=DEV),
                        cu_q=torch.tensor([0, 40, 42], dtype=torch.int32, device=DEV))
    pos = torch.arange(40, dtype=torch.int32)
    close(o[:40], ref.rotate(q[:40], cs, pos), q[:40])
    assert torch.equal(o[40:42], q[40:42])
    first = int(table[0, 0])
    assert torch.equal(vc[first], v[:16])
    keep = torch.ones(kc.shape[0], dtype=torch.bool)
    keep[first] = False
    assert torch.equal(kc[keep], kc0[keep]) and torch.equal(vc[keep], vc0[keep])


@gpu
def test_append_through_one_table_row():
    """Sequences that share one (expanded) table row, at positions of their own; the rows behind it are other pages."""
    import gated_deltanet_linear_15_gb300 as g
    qs, ks, table, kc, vc, qkv = _append_case([(2, 2 + 5 * n) for n in range(9)], BF, 64, 2, 1, 16, False, seed=3)
    q, k, v = qkv.split([2, 1, 1], 1)
    cs, table = table_ref(64, 64).float().to(DEV), table.to(DEV)
    lens = torch.tensor(ks, dtype=torch.int32, device=DEV)
    kc2, vc2 = kc.clone(), vc.clone()
    a = g.rotary_append(q, k, v, cs, kc, vc, table[-1:].repeat(9, 1), lens)
    b = g.rotary_append(q, k, v, cs, kc2, vc2, table[-1:].expand(9, -1), lens)
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


@gpu
def test_expanded_tensors_are_read_but_not_written():
    """Heads that share memory may be turned into new tensors; in place, or as an output or a cache, they are refused."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(13)
    one, q = torch.randn(5, 1, 64, generator=gen).to(DEV), torch.randn(5, 4, 64, generator=gen).to(DEV)
    wide, table, pos = one.expand(-1, 4, -1), table_ref(8, 64).float().to(DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    a, b = g.rotary(wide, wide, table, pos)
    close(a, ref.rotate(wide, table, pos), wide)
    assert torch.equal(a, b)
    kc, cache = torch.zeros(2, 16, 1, 64, device=DEV), torch.zeros(2, 16, 4, 64, device=DEV)
    pages, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([5], dtype=torch.int32, device=DEV)
    for call in (lambda: g.rotary(wide, None, table, pos, inplace=True), lambda: g.rotary(q, wide, table, pos, inplace=True),
                 lambda: g.rotary_append(q, q, q, table, kc.expand(-1, -1, 4, -1), cache, pages, lens),
                 lambda: g.rotary_append(q, q, q, table, cache, kc.expand(-1, -1, 4, -1), pages, lens),
                 lambda: g.rotary_append(q, q, q, table, cache, cache.clone(), pages, lens, out=torch.empty_like(one).expand(-1, 4, -1)),
                 lambda: g.paged_attention(q, cache, cache, pages, lens, out=torch.empty_like(one).expand(-1, 4, -1))):
        with pytest.raises(ValueError, match="expanded"):
            call()


@gpu
def test_lack_of_memory_is_named():
    """An output of 2 TB for an expanded input."""
    import gated_deltanet_linear_15_gb300 as g
    q = torch.zeros(4, 1, 128, dtype=BF, device=DEV).expand(-1, 2 ** 31 - 1, -1)
    with pytest.raises(torch.OutOfMemoryError):
        g.rotary(q, None, table_ref(8, 128).float().to(DEV), torch.arange(4, dtype=torch.int32, device=DEV))


@gpu
def test_many_equal_sequences_without_cu():
    import gated_deltanet_linear_15_gb300 as g
    seqs = [(2, 2 + 3 * n) for n in range(50)]
    qs, ks, table, kc, vc, qkv = _append_case(seqs, BF, 128, 4, 2, 32, False, seed=6)
    q, k, v = qkv.split([4, 2, 2], 1)
    cs = table_ref(200, 128).float().to(DEV)
    lens = torch.tensor(ks, dtype=torch.int32, device=DEV)
    kc2, vc2 = kc.clone(), vc.clone()
    a = g.rotary_append(q, k, v, cs, kc, vc, table.to(DEV), lens)
    b = g.rotary_append(q, k, v, cs, kc2, vc2, table.to(DEV), lens, cu_q=ref.lens_to_cu(qs, DEV))
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


# ------------------------------------------------------------------ refusals (no GPU needed)
def _shape(**kw):
    s = _lib.GdnRotaryShape()
    s.tokens, s.q_heads, s.k_heads, s.head_dim, s.rot, s.table_rows, s.dtype = 4, 2, 1, 64, 32, 100, _lib.GDN_BF16
    s.q_tok = s.qo_tok = 128
    s.q_head = s.qo_head = s.k_head = s.ko_head = s.k_tok = s.ko_tok = 64
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _call(lib, s, **p):
    a = dict(q=0x10000, k=0x10000, table=0x10000, pos=0x10000, qo=0x10000, ko=0x10000)
    a.update(p)
    return lib.gdn_rotary(ctypes.byref(s), a["q"], a["k"], a["table"], a["pos"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("kw", [dict(rot=33), dict(rot=0), dict(rot=66), dict(head_dim=1), dict(tokens=-1), dict(q_heads=-1),
                                dict(dtype=9), dict(interleaved=2), dict(inverse=-1), dict(table_rows=-1), dict(reserved=1)])
def test_c_entry_refuses_shapes(lib, kw):
    assert _call(lib, _shape(**kw)) == 1
    assert lib.gdn_last_error_string() != b""


def test_c_entry_refuses_pointers(lib):
    for name in ("q", "k", "table", "pos", "qo", "ko"):
        assert _call(lib, _shape(), **{name: None}) == 1, name
    assert _call(lib, _shape(), table=0x10004) == 1
    assert _call(lib, _shape(tokens=0), q=None) == 0
    assert lib.gdn_rotary_table(None, 4, 10, 1.0, 0x10000, None) == 1
    assert lib.gdn_rotary_table(0x10000, 0, 10, 1.0, 0x10000, None) == 1
    assert lib.gdn_rotary_table(0x10000, 4, 10, math.nan, 0x10000, None) == 1


def test_append_refuses(lib):
    s = _lib.GdnPagedShape()
    s.num_seqs, s.total_q, s.num_heads, s.num_kv_heads, s.head_dim, s.page_size = 2, 4, 4, 2, 64, 16
    s.num_pages, s.max_pages, s.dtype, s.table_stride, s.rot, s.table_rows = 10, 4, _lib.GDN_BF16, 4, 64, 100
    s.k_page = s.v_page = 16 * 128

    def call(**p):
        a = dict(zip(("q", "k", "v", "table", "kc", "vc", "pt", "cu", "kv", "o"), [0x10000] * 10))
        a.update(p)
        return lib.gdn_rotary_append(ctypes.byref(s), *a.values(), None)

    for name in ("q", "k", "v", "table", "kc", "vc", "pt", "kv", "o"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(rot=7), dict(rot=128), dict(interleaved=3), dict(k_page=0), dict(page_size=24), dict(num_kv_heads=3)):
        old = {k: getattr(s, k) for k in kw}
        for k, v in kw.items():
            setattr(s, k, v)
        assert call() != 0, kw
        for k, v in old.items():
            setattr(s, k, v)
