"""The norm of each head with its rotary turn, forward, backward and into the cache, against the definition in 64 bits.

Bounds.  A head's sum of squares is formed in chains of at most 32 products and a tree: off by at most 2^-19 of itself, half of
that in the reciprocal root, which is off by 2^-22 more; the products with it and the weight, and the turn's two products and
sum, round six times: in all below 2^-19 of |a c| + |b s| for an output a c - b s.  The backward's products have one sum more,
over terms of both signs: 2^-18 of the sum of magnitudes.  dw adds T H terms, each off by 2^-19, in chains that cannot be
longer than their number: (2^-19 + T H 2^-24) of the sum of magnitudes.  A bf16 output adds half a step, 2^-8 of the value."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests import block_ref as ref

gpu = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


# ------------------------------------------------------------------ the definition, in 64 bits on the CPU
def rotate(x, table, positions, interleaved, inverse=False):
    """x [T, H, D] fp64 turned by its positions' angles; a position outside the table leaves its token as it is."""
    x, table, positions = x.cpu().to(F64), table.cpu().to(F64), positions.cpu().long()
    rot, inside = 2 * table.shape[1], (positions >= 0) & (positions < table.shape[0])
    cs = table[positions.clamp(0, table.shape[0] - 1)][:, None]
    c, s = cs[..., 0], cs[..., 1] * (-1 if inverse else 1)
    first = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return torch.where(inside[:, None, None], y, x)


def turn_size(x, table, positions, interleaved):
    """The magnitudes |a c| + |b s| of every output of rotate."""
    t = table.cpu().to(F64).abs()
    t = torch.stack([t[..., 0], -t[..., 1]], -1)  # c, -s: both outputs become sums
    a = rotate(x.abs(), t, positions, interleaved)
    b = rotate(x.abs(), t * torch.tensor([1.0, -1.0], dtype=F64), positions, interleaved)
    return torch.maximum(a, b)


def forward(x, w, table, positions, eps, off, interleaved):
    """(y, its magnitude)"""
    x, w = x.cpu().to(F64), w.cpu().to(F64) + off
    y = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w
    return rotate(y, table, positions, interleaved), turn_size(y, table, positions, interleaved)


def backward(dy, x, w, table, positions, eps, off, interleaved):
    """(dx, its magnitude, dw, its magnitude)"""
    dy, x, w = dy.cpu().to(F64), x.cpu().to(F64), w.cpu().to(F64) + off
    u, um = rotate(dy, table, positions, interleaved, True), turn_size(dy, table, positions, interleaved)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = x * r
    dx = r * (u * w - h * (u * w * h).mean(-1, keepdim=True))
    size = r * (um * w.abs() + h.abs() * (um * w.abs() * h.abs()).mean(-1, keepdim=True))
    return dx, size, (u * h).sum((0, 1)), (um * h.abs()).sum((0, 1))


def near(got, want, tol, what, dtype):
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    err = (got.cpu().to(F64) - want).abs()
    bad = ~(err <= half * want.abs() + tol + 1e-37)
    assert not bad.any(), f"{what}: {int(bad.sum())} values, worst {float(err[bad].max()):.3g}"


def inputs(T, Hq, Hk, D, rot, dtype, off=0.0, rows=300, seed=0):
    gen = torch.Generator().manual_seed(seed + T * 7 + D + rot)

    def rand(*shape, dtype=F32):
        return torch.randn(*shape, generator=gen).to(DEV, dtype)

    freq, amp = __import__("gated_deltanet_linear_15_gb300").rotary_frequencies(rot, factor=4.0, scaling="linear")
    angle = torch.arange(rows, dtype=F64)[:, None] * freq
    table = torch.stack([angle.cos(), angle.sin()], -1).float().to(DEV)
    pos = torch.randint(0, rows, (T,), generator=gen).to(torch.int32)
    if T > 2:
        pos[1], pos[2] = -1, rows  # outside the table: not turned
    qk = rand(T, Hq + Hk, D, dtype=dtype)
    return dict(q=qk[:, :Hq], k=qk[:, Hq:] if Hk else None, dq=rand(T, Hq, D, dtype=dtype), dk=rand(T, Hk, D, dtype=dtype) if Hk else None,
                wq=1 - off + 0.2 * rand(D), wk=1 - off + 0.2 * rand(D) if Hk else None, table=table, pos=pos.to(DEV))


# D, rot: units of a head that are a power of two, others, odd ones, and more than a warp holds
SIZES = [(1, 1, 1, 64, 64), (7, 4, 2, 128, 128), (33, 3, 1, 128, 64), (5, 16, 16, 64, 32), (9, 2, 0, 256, 64), (300, 8, 2, 128, 32),
         (6, 5, 2, 96, 96), (4, 3, 3, 80, 20), (5, 2, 1, 7, 6), (3, 2, 2, 2, 2), (4, 1, 1, 1024, 512), (3, 40, 8, 512, 512),
         (2, 70, 30, 128, 128), (1, 1, 1, 1023, 1022), (2000, 1, 1, 64, 64)]


@gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_and_backward(T, Hq, Hk, D, rot, dtype, interleaved):
    import gated_deltanet_linear_15_gb300 as g
    off = 1.0 if interleaved else 0.0
    i = inputs(T, Hq, Hk, D, rot, dtype, off)
    how = dict(eps=1e-5, weight_offset=off, interleaved=interleaved)
    q, k = g.norm_rotary(i["q"], i["k"], i["wq"], i["wk"], i["table"], i["pos"], **how)
    got = g.norm_rotary_bwd(i["dq"], i["dk"], i["q"], i["k"], i["wq"], i["wk"], i["table"], i["pos"], **how)
    again = g.norm_rotary_bwd(i["dq"], i["dk"], i["q"], i["k"], i["wq"], i["wk"], i["table"], i["pos"], **how)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
    if not Hk:
        assert k is None and got[1] is None and got[3] is None
    for x, w, y, dy, dx, dw in ((i["q"], i["wq"], q, i["dq"], got[0], got[2]), (i["k"], i["wk"], k, i["dk"], got[1], got[3])):
        if x is None:
            continue
        want, size = forward(x, w, i["table"], i["pos"], 1e-5, off, interleaved)
        near(y, want, 2.0 ** -19 * size, "y", dtype)
        want, size, ww, wsize = backward(dy, x, w, i["table"], i["pos"], 1e-5, off, interleaved)
        near(dx, want, 2.0 ** -18 * size, "dx", dtype)
        near(dw, ww, (2.0 ** -18 + x.shape[0] * x.shape[1] * 2.0 ** -24) * wsize, "dw", F32)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 4, 8])
def test_strides_and_odd_alignment(dtype, off):
    """Heads inside wider rows, from any element on: the numbers of contiguous ones, to the sums' order."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(9, 4, 2, 64, 32, dtype)

    def moved(t):
        big = torch.full((9, t.shape[1], 64 + 13), float("nan"), device=DEV, dtype=dtype)
        big[..., off:off + 64] = t
        return big[..., off:off + 64]

    a = (i["wq"], i["wk"], i["table"], i["pos"])
    q, k = g.norm_rotary(moved(i["q"]), moved(i["k"]), *a)
    back = g.norm_rotary_bwd(moved(i["dq"]), moved(i["dk"]), moved(i["q"]), moved(i["k"]), *a)
    for x, w, y, dy, dx, dw in ((i["q"], i["wq"], q, i["dq"], back[0], back[2]), (i["k"], i["wk"], k, i["dk"], back[1], back[3])):
        want, size = forward(x, w, i["table"], i["pos"], 1e-6, 0.0, False)
        near(y, want, 2.0 ** -19 * size, "y", dtype)
        want, size, ww, wsize = backward(dy, x, w, i["table"], i["pos"], 1e-6, 0.0, False)
        near(dx, want, 2.0 ** -18 * size, "dx", dtype)
        near(dw, ww, (2.0 ** -18 + 36 * 2.0 ** -24) * wsize, "dw", F32)


@gpu
@pytest.mark.parametrize("D", [128, 96])
def test_zero_heads_and_nan(D):
    """A head of zeros stays zero with gradient u w / sqrt(eps), a NaN stays in its head (and in dw)."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(6, 4, 2, D, D, F32)
    q = i["q"].clone()
    q[3, 1] = 0
    q[4, 2, 5] = float("nan")
    a = (i["wq"], i["wk"], i["table"], i["pos"])
    y, _ = g.norm_rotary(q, i["k"], *a)
    assert (y[3, 1] == 0).all() and y[4, 2].isnan().all()
    keep = torch.ones(6, 4, dtype=torch.bool, device=DEV)
    keep[4, 2] = False
    assert torch.isfinite(y[keep]).all()
    dq, _, _, dwk = g.norm_rotary_bwd(i["dq"], i["dk"], q, i["k"], *a)
    u = rotate(i["dq"], i["table"], i["pos"], False, True)[3, 1] * i["wq"].cpu().to(F64) * 1e3
    near(dq[3, 1], u, 2.0 ** -18 * 1e3 * 8, "dq of a zero head", F32)
    assert torch.isfinite(dq[keep]).all() and torch.isfinite(dwk).all()


@gpu
@pytest.mark.parametrize("T,Hq", [(0, 4), (3, 0)])
def test_empty(T, Hq):
    import gated_deltanet_linear_15_gb300 as g
    q, w = torch.zeros(T, Hq, 64, device=DEV), torch.ones(64, device=DEV)
    table, pos = torch.zeros(4, 32, 2, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    assert g.norm_rotary(q, None, w, None, table, pos)[0].shape == q.shape
    got = g.norm_rotary_bwd(q, q, q, q, w, w, table, pos)
    assert got[0].shape == q.shape and (got[2] == 0).all() and (got[3] == 0).all()


# ------------------------------------------------------------------ gradients through autograd
@gpu
def test_gradient_by_differences():
    """Central differences of the definition in 64 bits, step 2^-12: an error of order 2^-24 of the third derivative, below
    2^-12 of the gradient's size here; the kernel's own is 2^-18 of a magnitude that is a few times the gradient's."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(5, 3, 2, 64, 32, F32)
    gen = torch.Generator().manual_seed(3)
    leaves = [i[k].clone().requires_grad_() for k in ("q", "k", "wq", "wk")]
    gq, gk = torch.randn(5, 3, 64, generator=gen, dtype=F64), torch.randn(5, 2, 64, generator=gen, dtype=F64)
    q, k = g.norm_rotary_embedding(*leaves, i["table"], i["pos"])
    ((q * gq.to(DEV)).sum() + (k * gk.to(DEV)).sum()).backward()

    def loss(q, k, wq, wk):
        a = (i["table"], i["pos"], 1e-6, 0.0, False)
        return float((forward(q, wq, *a)[0] * gq).sum() + (forward(k, wk, *a)[0] * gk).sum())

    base, e = [t.detach().cpu().to(F64) for t in leaves], 2.0 ** -12
    for n in range(4):
        u = torch.randn(base[n].shape, generator=gen, dtype=F64)
        up, down = list(base), list(base)
        up[n], down[n] = base[n] + e * u, base[n] - e * u
        num, grad = (loss(*up) - loss(*down)) / (2 * e), leaves[n].grad.cpu().to(F64)
        assert abs(num - float((grad * u).sum())) <= 2.0 ** -10 * float((grad * u).norm())


@gpu
def test_one_weight_for_both_and_no_k():
    """A weight that q and k share gets both gradients; without k there are none of it; second derivatives are refused."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(5, 3, 2, 64, 64, BF)
    w = i["wq"].clone().requires_grad_()
    q, k = g.norm_rotary_embedding(i["q"], i["k"], w, w, i["table"], i["pos"])
    torch.autograd.backward([q, k], [i["dq"], i["dk"]])
    want = g.norm_rotary_bwd(i["dq"], i["dk"], i["q"], i["k"], i["wq"], i["wq"], i["table"], i["pos"])
    assert torch.equal(w.grad, want[2] + want[3])
    x = i["q"].clone().requires_grad_()
    q, k = g.norm_rotary_embedding(x, None, i["wq"], None, i["table"], i["pos"])
    assert k is None
    q.backward(i["dq"])
    want = g.norm_rotary_bwd(i["dq"], i["dk"], i["q"], i["k"], i["wq"], i["wq"], i["table"], i["pos"])
    assert torch.equal(x.grad, want[0])
    y, _ = g.norm_rotary_embedding(x, None, i["wq"], None, i["table"], i["pos"])
    dx = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


# ------------------------------------------------------------------ into the cache
@gpu
@pytest.mark.parametrize("D,rot,page,Hq,Hkv", [(128, 128, 16, 8, 2), (64, 32, 64, 4, 4), (96, 40, 32, 3, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(D, rot, page, Hq, Hkv, dtype, interleaved):
    """Queries as the forward gives them, keys in their slots, values as they are; other slots, missing pages and tokens that no
    sequence names stay as they were."""
    import gated_deltanet_linear_15_gb300 as g
    qs, kv = [3, 0, 1, 20], [70, 5, 1, 90]
    i = inputs(26, Hq, Hkv, D, rot, dtype, rows=200)
    q, k, v = i["q"], i["k"], torch.randn(26, Hkv, D, device=DEV).to(dtype)
    width = -(-90 // page)
    table = torch.randperm(4 * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(4, width).to(DEV)
    table[3, 84 // page] = -1
    kc, vc = torch.full((4 * width, page, Hkv, D), 3.0, device=DEV, dtype=dtype), torch.full((4 * width, page, Hkv, D), 4.0, device=DEV, dtype=dtype)
    cu = ref.lens_to_cu(qs, DEV)
    out = g.norm_rotary_append(q, k, v, i["wq"], i["wk"], i["table"], kc, vc, table, torch.tensor(kv, dtype=torch.int32, device=DEV),
                               cu_q=cu, eps=1e-5, interleaved=interleaved)
    pos = torch.cat([torch.arange(b - a, b) for a, b in zip(qs, kv)]).to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(4), torch.tensor(qs))
    wk, wv = torch.full(kc.shape, 3.0, dtype=F64), torch.full(vc.shape, 4.0, dtype=F64)
    sk = torch.zeros_like(wk)
    key, size = forward(k[:24], i["wk"], i["table"], pos, 1e-5, 0.0, interleaved)
    for t in range(24):
        pg = int(table[seq[t], int(pos[t]) // page])
        if pg >= 0:
            wk[pg, int(pos[t]) % page], sk[pg, int(pos[t]) % page] = key[t], size[t]
            wv[pg, int(pos[t]) % page] = v[t].cpu().to(F64)
    near(kc, wk, 2.0 ** -19 * sk, "keys", dtype)
    assert torch.equal(vc.cpu().to(F64), wv)
    want, size = forward(q[:24], i["wq"], i["table"], pos, 1e-5, 0.0, interleaved)
    near(out[:24], want, 2.0 ** -19 * size, "queries", dtype)


@gpu
def test_append_is_forward_and_copy():
    """Bit for bit the forward at the same positions; the cache's version moves on; an output of the caller's is used."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(8, 8, 2, 128, 128, BF, rows=64)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    q, k = g.norm_rotary(i["q"], i["k"], i["wq"], i["wk"], i["table"], pos)
    kc, vc = torch.zeros(2, 16, 2, 128, device=DEV, dtype=BF), torch.zeros(2, 16, 2, 128, device=DEV, dtype=BF)
    table, lens, v = torch.tensor([[1]], dtype=torch.int32, device=DEV), torch.tensor([8], dtype=torch.int32, device=DEV), i["dk"]
    before, out = kc._version, torch.empty_like(i["dq"])
    got = g.norm_rotary_append(i["q"], i["k"], v, i["wq"], i["wk"], i["table"], kc, vc, table, lens, out=out)
    assert got is out or got.data_ptr() == out.data_ptr()
    assert torch.equal(got, q) and torch.equal(kc[1, :8], k) and torch.equal(vc[1, :8], v) and kc._version > before


# ------------------------------------------------------------------ refusals
@gpu
def test_binding_refuses():
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(4, 2, 1, 64, 32, F32)
    q, k, wq, wk, table, pos = (i[n] for n in ("q", "k", "wq", "wk", "table", "pos"))
    for call in (lambda: g.norm_rotary(q.half(), k.half(), wq, wk, table, pos), lambda: g.norm_rotary(q, k.bfloat16(), wq, wk, table, pos),
                 lambda: g.norm_rotary(q, k, wq[:32], wk, table, pos), lambda: g.norm_rotary(q, k, wq, None, table, pos),
                 lambda: g.norm_rotary(q, k, wq.bfloat16(), wk, table, pos), lambda: g.norm_rotary(q, k, wq, wk, table, pos[:2]),
                 lambda: g.norm_rotary(q, k[:2], wq, wk, table, pos), lambda: g.norm_rotary(q, k, wq, wk, table, pos, eps=0.0),
                 lambda: g.norm_rotary(q, k, wq, wk, table, pos, eps=math.nan), lambda: g.norm_rotary(q.cpu(), k, wq, wk, table, pos),
                 lambda: g.norm_rotary_bwd(q[:2], k, q, k, wq, wk, table, pos), lambda: g.norm_rotary_bwd(q, None, q, k, wq, wk, table, pos),
                 lambda: g.norm_rotary_bwd(q, q, q, k, wq, wk, table, pos),
                 lambda: g.norm_rotary(torch.zeros(1, 1, 1026, device=DEV), None, torch.ones(1026, device=DEV), None, table, pos[:1])):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def _shape(**kw):
    s = _lib.GdnRotaryShape(tokens=4, q_heads=2, k_heads=1, head_dim=64, rot=32, table_rows=10, dtype=_lib.GDN_BF16)
    for n in ("q_tok", "qo_tok", "k_tok", "ko_tok"):
        setattr(s, n, 128)
    for n in ("q_head", "qo_head", "k_head", "ko_head"):
        setattr(s, n, 64)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_c_entry_refuses(lib):
    p = [0x10000 * (i + 1) for i in range(14)]

    def fwd(eps=1e-6, off=0.0, drop=None, **kw):
        a = list(p[:8])
        if drop is not None:
            a[drop] = None
        return lib.gdn_norm_rotary(ctypes.byref(_shape(**kw)), eps, off, *a, None)

    for kw, code in ((dict(inverse=1), 1), (dict(eps=0.0), 1), (dict(eps=math.inf), 1), (dict(off=math.nan), 1), (dict(head_dim=1026), 2),
                     (dict(rot=3), 1), (dict(rot=66), 1), (dict(tokens=-1), 1), (dict(dtype=9), 1), (dict(reserved=1), 1)):
        assert fwd(**kw) == code, kw
    for i in range(8):
        assert fwd(drop=i) == 1, i
    s = _shape()
    need = lib.gdn_norm_rotary_bwd_workspace_size(ctypes.byref(s))
    assert need > 0 and lib.gdn_norm_rotary_bwd_workspace_size(ctypes.byref(_shape(rot=3))) == 0

    def bwd(nbytes=need, ws=0x1000000, drop=None, same=False):
        a = list(p[:12])
        if same:
            a[11] = a[10]
        if drop is not None:
            a[drop] = None
        return lib.gdn_norm_rotary_bwd(ctypes.byref(s), 1e-6, 0.0, *a, ws, nbytes, None)

    for i in range(12):
        assert bwd(drop=i) == 1, i
    assert bwd(nbytes=need - 1) == 3 and bwd(ws=None) == 3 and bwd(ws=0x1000008) == 1 and bwd(same=True) == 1
    t = _lib.GdnPagedShape(num_seqs=1, total_q=4, num_heads=2, num_kv_heads=1, head_dim=64, page_size=16, num_pages=4, max_pages=2,
                           dtype=_lib.GDN_BF16, k_page=1024, v_page=1024, rot=32, table_rows=10)
    a = list(p[:12])
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11):   # all but cu_q
        b = list(a)
        b[i] = None
        assert lib.gdn_norm_rotary_append(ctypes.byref(t), 1e-6, 0.0, *b, None) == 1, i
    assert lib.gdn_norm_rotary_append(ctypes.byref(t), 0.0, 0.0, *a, None) == 1
