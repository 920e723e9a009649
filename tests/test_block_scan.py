"""The gated linear recurrence, forward, backward and by single tokens, against a token loop in 64 bits.

Bounds.  M is the recurrence of the magnitudes, M_t = a_t M_{t-1} + |x_t|.  In a segment of 16 tokens each step multiplies by
a gate that is off by at most 2^-22 of itself (ex2.approx; expf has 2^-23), with the argument's rounding |g| exp(g) 2^-24 <=
2^-25, and rounds once (2^-24): at most 16 * 2.75 * 2^-23 = 44 * 2^-23 of M.  A state that
passes a whole segment is multiplied by the exponential of a sum of 16 gates, off by 16 * 2^-24 |sum| exp(sum) <= 3 * 2^-23 and
by 2^-23 of itself, and added to (two roundings where maps meet): 5 * 2^-23, and as much again where the maps of eight segments
are joined before they are applied.  So (44 + 10 n) 2^-23 M for n segments.  Gradients are the same recurrence of the other
direction; that of the gate is a product of both, so both bounds add up.  A bf16 output adds half a step, 2^-8 of the value."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib

gpu = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


# ------------------------------------------------------------------ the definition, in 64 bits on the CPU
def loop(x, g, h0, cu):
    """(h, M, final, final's M, state before each token, its M) of the line x, g [tokens, D]; h0 [N, D]."""
    x, a = x.cpu().to(F64), g.cpu().to(F64).exp()
    h0 = torch.zeros(len(cu) - 1, x.shape[1], dtype=F64) if h0 is None else h0.cpu().to(F64)
    h, m, hp, mp = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    final, mf = h0.clone(), h0.abs()
    for n, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
        s, ms = h0[n], h0[n].abs()
        for t in range(b, e):
            hp[t], mp[t] = s, ms
            s, ms = a[t] * s + x[t], a[t] * ms + x[t].abs()
            h[t], m[t] = s, ms
        if e > b:
            final[n], mf[n] = s, ms
    return h, m, final, mf, hp, mp


def loop_bwd(dy, g, d_final, cu):
    """(d, magnitude, what reaches the state before each token, its magnitude, dh0, its magnitude)."""
    dy, a = dy.cpu().to(F64), g.cpu().to(F64).exp()
    dT = torch.zeros(len(cu) - 1, dy.shape[1], dtype=F64) if d_final is None else d_final.cpu().to(F64)
    d, m, f, mf = torch.zeros_like(dy), torch.zeros_like(dy), torch.zeros_like(dy), torch.zeros_like(dy)
    d0, m0 = dT.clone(), dT.abs()
    for n, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
        s, ms = dT[n], dT[n].abs()
        for t in range(e - 1, b - 1, -1):
            d[t], m[t] = s + dy[t], ms + dy[t].abs()
            s, ms = a[t] * d[t], a[t] * m[t]
            f[t], mf[t] = s, ms
        if e > b:
            d0[n], m0[n] = s, ms
    return d, m, f, mf, d0, m0


def bound(longest):
    return (44 + 10 * (longest // 16 + 2)) * 2.0 ** -23


def near(got, want, tol, what):
    got = got.cpu().to(F64).reshape(want.shape)
    half = 2.0 ** -8 if what.endswith("bf16") else 2.0 ** -24
    bad = ~((got - want).abs() <= half * want.abs() + tol + 1e-37)
    assert not bad.any(), f"{what}: {int(bad.sum())} values, worst {float((got - want).abs()[bad].max()):.3g}"


def inputs(lens, D, dtype, gate, packed, h0=True, seed=0):
    gen = torch.Generator().manual_seed(seed + D + 7 * sum(lens))
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])

    def rand(*shape, dtype=F32):
        return torch.randn(*shape, generator=gen).to(DEV, dtype)

    x, dy = rand(*lead, D, dtype=dtype), rand(*lead, D, dtype=dtype)
    rate = 10 ** (-3.5 * torch.rand(D, generator=gen))
    g = (-rate * torch.nn.functional.softplus(torch.randn(*lead, D, generator=gen))).to(DEV, gate)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return dict(x=x, dy=dy, g=g, h0=rand(len(lens), D) if h0 else None, dT=rand(len(lens), D) if h0 else None, cu=cu,
                dev=torch.tensor(cu, dtype=torch.int32, device=DEV) if packed else None)


def check(i, D, both=True):
    """Forward and backward of inputs i against the loops."""
    import gated_deltanet_linear_15_gb300 as g
    kind = "bf16" if i["x"].dtype == BF else "fp32"
    gkind = "bf16" if i["g"].dtype == BF else "fp32"
    longest = max(b - a for a, b in zip(i["cu"][:-1], i["cu"][1:]))
    tol = bound(longest)
    y, final, states = g.gated_scan(i["x"], i["g"], i["h0"], cu_seqlens=i["dev"], save_states=True)
    line = {k: i[k].reshape(-1, D) for k in ("x", "g", "dy")}
    h, m, hT, mT, hp, mp = loop(line["x"], line["g"], i["h0"], i["cu"])
    near(y, h, tol * m, "y " + kind)
    near(final, hT, tol * mT, "final")
    again = g.gated_scan(i["x"], i["g"], i["h0"], cu_seqlens=i["dev"])
    assert torch.equal(again[0], y) and torch.equal(again[1], final)
    if not both:
        return
    got = g.gated_scan_bwd(i["dy"], i["x"], i["g"], states, i["h0"], i["dT"], cu_seqlens=i["dev"])
    d, md, f, mf, d0, m0 = loop_bwd(line["dy"], line["g"], i["dT"], i["cu"])
    near(got[0], d, tol * md, "dx " + kind)
    near(got[1], f * hp, 2 * tol * mf * mp, "dg " + gkind)
    if i["h0"] is None:
        assert got[2] is None
    else:
        near(got[2], d0, tol * m0, "dh0")
    again = g.gated_scan_bwd(i["dy"], i["x"], i["g"], states, i["h0"], i["dT"], cu_seqlens=i["dev"])
    assert all(p is q is None or torch.equal(p, q) for p, q in zip(again, got))


# ------------------------------------------------------------------ sizes, types, packing
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@gpu
@pytest.mark.parametrize("N,T,D", [(1, 1, 64), (1, 15, 1), (3, 16, 100), (2, 17, 64), (1, 300, 130), (5, 129, 101), (4, 1000, 256),
                                   (1, 5000, 64), (70, 3, 33), (300, 1, 8), (2, 2049, 72), (1, 700, 1000)])
@pytest.mark.parametrize("dtype,gate", TYPES)
def test_equal_sequences(N, T, D, dtype, gate):
    check(inputs([T] * N, D, dtype, gate, False, h0=T % 2 == 1), D)


PACKED = {"empties": [0, 5, 0, 0, 1, 1, 1, 200, 16, 0, 33, 0], "one": [777], "singles": [1] * 150, "long_and_short": [3] * 20 + [2500] + [2] * 40,
          "many_empty": [0] * 100 + [7] + [0] * 90 + [9, 0], "aligned": [16, 32, 128, 16, 64], "all_empty_but_last": [0] * 5 + [40]}


@gpu
@pytest.mark.parametrize("lens", PACKED.values(), ids=PACKED.keys())
@pytest.mark.parametrize("D", [64, 130, 37])
@pytest.mark.parametrize("dtype,gate", TYPES)
def test_packed_sequences(lens, D, dtype, gate):
    check(inputs(lens, D, dtype, gate, True), D)


@gpu
def test_packed_without_states():
    check(inputs(PACKED["empties"], 64, BF, BF, True, h0=False), 64)


@gpu
@pytest.mark.parametrize("packed", [False, True])
def test_wide(packed):
    """More channel blocks than SMs, more sequences than parts."""
    check(inputs([40] * 9, 20000, BF, BF, packed), 20000, both=False)
    check(inputs([3, 0, 50, 17], 10000, F32, F32, True), 10000)


@gpu
@pytest.mark.parametrize("lens,D", [([3000, 100, 2700, 0, 2500, 900], 2001), ([431, 0, 1716, 4325, 3411, 55, 6939, 233], 1001),
                                    ([200, 300, 15000, 1, 0, 700], 1001), ([1, 9000], 2001), ([0, 0, 8500, 0, 0], 2001)])
def test_long_packed_sequences(lens, D):
    """Few packed sequences and many rounds: parts that are evened out, or cannot be."""
    check(inputs(lens, D, F32, F32, True), D, both=False)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 2, 4, 8])
def test_rows_with_strides_and_odd_alignment(dtype, off):
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([50, 9, 41], 64, dtype, dtype, True)
    want = g.gated_scan(i["x"], i["g"], i["h0"], cu_seqlens=i["dev"], save_states=True)
    back = g.gated_scan_bwd(i["dy"], i["x"], i["g"], want[2], i["h0"], i["dT"], cu_seqlens=i["dev"])

    def moved(t):
        big = torch.full((1, 100, 3 * 64 + 11), float("nan"), device=DEV, dtype=dtype)
        big[..., off:off + 64] = t
        return big[..., off:off + 64]

    x, gt, dy = moved(i["x"]), moved(i["g"]), moved(i["dy"])
    got = g.gated_scan(x, gt, i["h0"], cu_seqlens=i["dev"], save_states=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(p, q) for p, q in zip(g.gated_scan_bwd(dy, x, gt, got[2], i["h0"], i["dT"], cu_seqlens=i["dev"]), back))


@gpu
@pytest.mark.parametrize("T", [0, 1])
def test_no_and_single_tokens(T):
    import gated_deltanet_linear_15_gb300 as g
    x, h0 = torch.randn(3, T, 40, device=DEV), torch.randn(3, 40, device=DEV)
    y, final, states = g.gated_scan(x, x - 5, h0, save_states=True)
    assert y.shape == x.shape
    if T == 0:
        assert torch.equal(final, h0) and (g.gated_scan(x, x)[1] == 0).all()
        dx, dg, dh0 = g.gated_scan_bwd(x, x, x, states, h0, final)
        assert torch.equal(dh0, final) and dx.shape == x.shape
    else:
        assert torch.equal(y[:, 0], final)


@gpu
def test_no_sequences():
    import gated_deltanet_linear_15_gb300 as g
    x, h0 = torch.zeros(0, 7, 40, device=DEV), torch.zeros(0, 40, device=DEV)
    y, final, states = g.gated_scan(x, x, h0, save_states=True)
    dx, dg, dh0 = g.gated_scan_bwd(x, x, x, states, h0, final)
    assert y.shape == dx.shape == dg.shape == x.shape and final.shape == dh0.shape == h0.shape
    assert g.gated_scan_step(h0, h0, final)[0].shape == h0.shape


# ------------------------------------------------------------------ what gates and states may hold
@gpu
def test_a_gate_of_minus_infinity_forgets():
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([100], 64, F32, F32, False)
    i["g"][:, 57] = -float("inf")
    y, final, states = g.gated_scan(i["x"], i["g"], i["h0"], save_states=True)
    assert torch.equal(y[:, 57], i["x"][:, 57])
    check(i, 64)


@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_in_their_sequence_and_channel(bad):
    import gated_deltanet_linear_15_gb300 as g
    lens = [130, 3, 200, 64]
    i = inputs(lens, 64, F32, F32, True)
    want = g.gated_scan(i["x"], i["g"], i["h0"], cu_seqlens=i["dev"], save_states=True)
    back = g.gated_scan_bwd(i["dy"], i["x"], i["g"], want[2], i["h0"], i["dT"], cu_seqlens=i["dev"])
    x, dy = i["x"].clone(), i["dy"].clone()
    x[0, 133 + 20, 5] = bad
    dy[0, 133 + 90, 6] = bad
    got = g.gated_scan(x, i["g"], i["h0"], cu_seqlens=i["dev"], save_states=True)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[0, 133 + 20:333, 5] = False
    assert torch.equal(got[0][keep], want[0][keep]) and not torch.isfinite(got[0][~keep]).any()
    assert torch.equal(got[1][[0, 1, 3]], want[1][[0, 1, 3]])
    b = g.gated_scan_bwd(dy, i["x"], i["g"], want[2], i["h0"], i["dT"], cu_seqlens=i["dev"])
    keep[:] = True
    keep[0, 133:133 + 91, 6] = False
    assert torch.equal(b[0][keep], back[0][keep]) and not torch.isfinite(b[0][~keep]).any()
    assert torch.equal(b[2][[0, 1, 3]], back[2][[0, 1, 3]])


@gpu
@pytest.mark.parametrize("cu", [[5, 20, 40], [0, 20, 40], [0, 0, 0], [30, 60, 90]])
def test_rows_that_no_sequence_names_stay(cu):
    """Through the C entry: the outputs' other rows keep what they held."""
    import gated_deltanet_linear_15_gb300 as g
    D, T = 64, 90
    i = inputs([T], D, F32, F32, True)
    s = _lib.GdnScanShape(num_seqs=2, tokens=T, dim=D, dtype=_lib.GDN_FP32, gate_dtype=_lib.GDN_FP32,
                          x_row=D, g_row=D, y_row=D, dy_row=D, dg_row=D)
    dev, h0 = torch.tensor(cu, dtype=torch.int32, device=DEV), torch.randn(2, D, device=DEV)
    y, dx, dg = (torch.full((T, D), 7.0, device=DEV) for _ in range(3))
    final, dh0 = torch.zeros(2, D, device=DEV), torch.zeros(2, D, device=DEV)
    states = torch.zeros((T + 15) // 16, D, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    lib, p = _lib.load(), lambda t: t.data_ptr()
    assert lib.gdn_scan_fwd(ctypes.byref(s), p(i["x"]), p(i["g"]), p(h0), p(dev), p(y), p(final), p(states), st) == 0
    assert lib.gdn_scan_bwd(ctypes.byref(s), p(i["dy"]), p(i["x"]), p(i["g"]), p(states), p(h0), p(final), p(dev), p(dx), p(dg), p(dh0),
                            st) == 0
    torch.cuda.synchronize()
    line = {k: i[k][0] for k in ("x", "g", "dy")}
    h, m, hT, mT, hp, mp = loop(line["x"], line["g"], h0, cu)
    d, md, f, mf, d0, m0 = loop_bwd(line["dy"], line["g"], final, cu)
    for got in (y, dx, dg):
        assert (got[:cu[0]] == 7).all() and (got[cu[-1]:] == 7).all()
    w, tol = slice(cu[0], cu[-1]), bound(90)
    near(y[w], h[w], tol * m[w], "y")
    near(final, hT, tol * mT, "final")
    near(dx[w], d[w], tol * md[w], "dx")
    near(dg[w], (f * hp)[w], 2 * tol * (mf * mp)[w], "dg")
    near(dh0, d0, tol * m0, "dh0")


@gpu
@pytest.mark.parametrize("cu", [[0, 50, 20, 90], [90, 0, 90, 0], [-5, 1000, 3, 2 ** 31 - 1], [40, 30, 20, 10], [0] * 40 + [90, 3] * 60])
def test_any_cu_seqlens_ends_within_the_rows(cu):
    """Entries out of order or range: whatever is computed, the call ends and nothing outside the outputs is written."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([90], 64, F32, F32, True)
    dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
    h0 = torch.randn(len(cu) - 1, 64, device=DEV)
    y, final, states = g.gated_scan(i["x"], i["g"], h0, cu_seqlens=dev, save_states=True)
    g.gated_scan_bwd(i["dy"], i["x"], i["g"], states, h0, final, cu_seqlens=dev)
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("cu", [[0, 5000, 2000, 8300], [8300, 0, 8300, 0], [-5, 1000000, 3, 2 ** 31 - 1], [4000, 3000, 2000, 1000], [8300, 8300, 9]])
def test_any_cu_seqlens_of_many_rounds_ends(cu):
    """The same where parts are evened out."""
    import gated_deltanet_linear_15_gb300 as g
    x = torch.ones(1, 8300, 2001, device=DEV)
    dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y, final, states = g.gated_scan(x, -x, cu_seqlens=dev, save_states=True)
    g.gated_scan_bwd(x, x, -x, states, None, final, cu_seqlens=dev)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ gradients
@gpu
def test_gradient_by_differences():
    """Central differences of the loop in 64 bits along random directions, step 2^-12: an error of order 2^-24 of the third
    derivative, below 2^-12 of the gradient's size here; the kernel's own is at most bound(70) of it."""
    import gated_deltanet_linear_15_gb300 as g
    lens, D, e = [70, 0, 25], 24, 2.0 ** -12
    i = inputs(lens, D, F32, F32, True)
    gy, gf = torch.randn(95, D, dtype=F64), torch.randn(3, D, dtype=F64)
    leaves = [i[k].clone().requires_grad_() for k in ("x", "g", "h0")]
    y, final = g.gated_linear_recurrence(*leaves, cu_seqlens=i["dev"])
    ((y[0] * gy.to(DEV)).sum() + (final * gf.to(DEV)).sum()).backward()

    def loss(x, gt, h0):
        r = loop(x, gt, h0, i["cu"])
        return float((r[0] * gy).sum() + (r[2] * gf).sum())

    base = [i["x"][0].cpu().to(F64), i["g"][0].cpu().to(F64), i["h0"].cpu().to(F64)]
    for k in range(3):
        u = torch.randn(base[k].shape, dtype=F64)
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + e * u, base[k] - e * u
        num = (loss(*up) - loss(*down)) / (2 * e)
        grad = leaves[k].grad.cpu().to(F64).reshape(u.shape)
        assert abs(num - float((grad * u).sum())) <= 2.0 ** -10 * float((grad * u).norm())


@gpu
@pytest.mark.parametrize("dtype,gate", TYPES)
def test_autograd(dtype, gate):
    """The gradients are the backward's; an output that nothing depends on counts as zero."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([40, 40], 48, dtype, gate, False)
    leaves = [i[k].clone().requires_grad_() for k in ("x", "g", "h0")]
    y, final = g.gated_linear_recurrence(*leaves)
    y.backward(i["dy"], retain_graph=True)
    states = g.gated_scan(i["x"], i["g"], i["h0"], save_states=True)[2]
    want = g.gated_scan_bwd(i["dy"], i["x"], i["g"], states, i["h0"])
    assert all(torch.equal(p.grad, q) for p, q in zip(leaves, want))
    for p in leaves:
        p.grad = None
    final.backward(i["dT"])
    want = g.gated_scan_bwd(torch.zeros_like(i["dy"]), i["x"], i["g"], states, i["h0"], i["dT"])
    assert all(torch.equal(p.grad, q) for p, q in zip(leaves, want))
    x = i["x"].clone().requires_grad_()
    g.gated_linear_recurrence(x, i["g"])[0].sum().backward()
    assert x.grad is not None and i["g"].grad is None


@gpu
def test_second_derivatives_are_refused():
    import gated_deltanet_linear_15_gb300 as g
    x = torch.randn(2, 20, 16, device=DEV, requires_grad=True)
    y, _ = g.gated_linear_recurrence(x, -x.detach().abs())
    dx = torch.autograd.grad(y.square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


# ------------------------------------------------------------------ single tokens and continuation
@gpu
@pytest.mark.parametrize("N,D", [(1, 1), (3, 64), (5, 101), (256, 1024), (2, 2050), (70000, 4)])
@pytest.mark.parametrize("dtype,gate", TYPES)
def test_step(N, D, dtype, gate):
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([1] * N, D, dtype, gate, False)
    x, gt, h0 = i["x"][:, 0], i["g"][:, 0], i["h0"]
    pool = torch.full((N, D + 8), 3.0, device=DEV)
    state = pool[:, 4:4 + D]
    state.copy_(h0)
    y, out = g.gated_scan_step(x, gt, state)
    assert out is state and (pool[:, :4] == 3).all() and (pool[:, 4 + D:] == 3).all()
    a = gt.cpu().to(F64).exp()
    want = a * h0.cpu().to(F64) + x.cpu().to(F64)
    tol = 2.0 ** -22 * (a * h0.cpu().to(F64).abs() + x.cpu().to(F64).abs())
    near(state, want, tol, "state")
    near(y, want, tol, "y " + ("bf16" if dtype == BF else "fp32"))


@gpu
def test_prefill_goes_on_in_steps():
    """A sequence in two calls and a step: as in one call, to the bound."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([301, 301], 96, F32, F32, False)
    x, gt = i["x"], i["g"]
    h, m, hT, mT, _, _ = loop(x.reshape(-1, 96), gt.reshape(-1, 96), i["h0"], i["cu"])
    _, s = g.gated_scan(x[:, :200].contiguous(), gt[:, :200].contiguous(), i["h0"])
    _, s = g.gated_scan(x[:, 200:300].contiguous(), gt[:, 200:300].contiguous(), s)
    y, s = g.gated_scan_step(x[:, 300], gt[:, 300], s)
    near(s, hT, 2 * bound(301) * mT, "state")
    assert torch.equal(y, s)


@gpu
def test_capture_and_streams():
    """Replayed from a graph, and on a stream of its own: the same bits."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([500, 0, 33, 700], 256, BF, BF, True)

    def run():
        y, final, states = g.gated_scan(i["x"], i["g"], i["h0"], cu_seqlens=i["dev"], save_states=True)
        return (y, final) + tuple(g.gated_scan_bwd(i["dy"], i["x"], i["g"], states, i["h0"], i["dT"], cu_seqlens=i["dev"]))

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------------ refusals
@gpu
def test_binding_refuses():
    import gated_deltanet_linear_15_gb300 as g
    x, s = torch.zeros(2, 10, 64, device=DEV), torch.zeros(2, 64, device=DEV)
    cu = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    st = g.gated_scan(x, x, save_states=True)[2]
    for call in (lambda: g.gated_scan(x.half(), x.half()), lambda: g.gated_scan(x, x.bfloat16()), lambda: g.gated_scan(x, x[:1]),
                 lambda: g.gated_scan(x.cpu(), x), lambda: g.gated_scan(x[0], x[0]), lambda: g.gated_scan(x, x, s[:1]),
                 lambda: g.gated_scan(x, x, s.bfloat16()), lambda: g.gated_scan(x, x, cu_seqlens=cu), lambda: g.gated_scan(x[:1], x[:1], cu_seqlens=cu.long()),
                 lambda: g.gated_scan(x[:1], x[:1], cu_seqlens=cu[:1]), lambda: g.gated_scan(x.transpose(0, 1), x.transpose(0, 1)),
                 lambda: g.gated_scan(x.transpose(1, 2), x.transpose(1, 2)), lambda: g.gated_scan_bwd(x, x, x, st[:1]),
                 lambda: g.gated_scan_bwd(x[:1], x, x, st), lambda: g.gated_scan_bwd(x, x, x, st, d_final=s[:1]),
                 lambda: g.gated_scan_bwd(x, x, x, st.bfloat16()), lambda: g.gated_scan_step(x[0], x[0], s),
                 lambda: g.gated_scan_step(s, s, s.bfloat16()), lambda: g.gated_scan_step(s, s, s[:1].expand(2, 64)), lambda: g.gated_scan_step(s, s, s)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def _shape(**kw):
    s = _lib.GdnScanShape(num_seqs=2, tokens=20, dim=64, dtype=_lib.GDN_BF16, gate_dtype=_lib.GDN_FP32,
                          x_row=64, g_row=64, y_row=64, dy_row=64, dg_row=64, state_row=64)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), 1), (dict(tokens=-1), 1), (dict(tokens=21), 1), (dict(tokens=2 ** 31 - 2), 2), (dict(dim=0), 2),
    (dict(dim=(1 << 20) + 1), 2), (dict(dtype=5), 1), (dict(dtype=_lib.GDN_FP32, gate_dtype=_lib.GDN_BF16), 1), (dict(reserved=1), 1),
    (dict(x_row=-1), 1), (dict(y_row=63), 1),
])
def test_c_entry_refuses_shapes(lib, kw, code):
    a = [0x10000, 0x20000, None, None, 0x30000, None, None]
    assert lib.gdn_scan_fwd(ctypes.byref(_shape(**kw)), *a, None) == code
    assert lib.gdn_last_error_string() != b""


def test_c_entry_refuses_arguments(lib):
    s = _shape()
    p = [0x10000 * (i + 1) for i in range(11)]

    def fwd(**kw):
        a = dict(zip(("x", "g", "h0", "cu", "y", "final", "states"), p))
        a.update(cu=None, **kw)
        return lib.gdn_scan_fwd(ctypes.byref(s), *a.values(), None)

    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(y=p[0]), dict(y=p[1]), dict(final=p[2])):
        assert fwd(**kw) == 1, kw

    def bwd(shape=s, **kw):
        a = dict(zip(("dy", "x", "g", "states", "h0", "dT", "cu", "dx", "dg", "dh0"), p))
        a.update(cu=None)
        a.update(**kw)
        return lib.gdn_scan_bwd(ctypes.byref(shape), *a.values(), None)

    for kw in (dict(dy=None), dict(x=None), dict(g=None), dict(states=None), dict(dx=None), dict(dg=None), dict(dx=p[8]), dict(dx=p[0]),
               dict(dg=p[2]), dict(dh0=p[5]), dict(dh0=p[4]), dict(shape=_shape(dg_row=10))):
        assert bwd(**kw) == 1, kw
    for kw in (dict(tokens=4), dict(state_row=63)):
        assert lib.gdn_scan_step(ctypes.byref(_shape(**dict(dict(tokens=2), **kw))), *p[:4], None) == 1
    for i in range(4):
        a = p[:4]
        a[i] = None
        assert lib.gdn_scan_step(ctypes.byref(_shape(tokens=2)), *a, None) == 1
    assert lib.gdn_scan_states_rows(ctypes.byref(s)) == 2
    assert lib.gdn_scan_states_rows(ctypes.byref(_shape(dim=0))) == -1
    assert lib.gdn_scan_fwd(ctypes.byref(_shape(tokens=0)), *[None] * 7, None) == 0
