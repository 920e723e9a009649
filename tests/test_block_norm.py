"""The residual stream's root-mean-square norm, forward and backward, against the definition in 64 bits.

Bounds.  Sums of D squares in fp32 are off by at most D 2^-24 of their value in theory and a few 2^-24 as they are formed
here (trees of partial sums); 2^-20 is allowed for rstd, which carries to y.  A bf16 output adds its rounding, 2^-8 of the
value; e4m3 has 3 mantissa bits, so half an ulp is 2^-4 of the value, or 2^-10 of the largest scaled value (448 maps to
the top) below the normal range: 2^-10 * scale in absolute terms."""
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


def near(got, want, rel, what):
    got = got.cpu().double()
    assert ((got - want).abs() <= rel * want.abs() + 1e-30).all(), \
        f"{what}: {float(((got - want).abs() / (want.abs() + 1e-30)).max()):.3g} of the value"


def rand(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen).to(DEV, dtype)


SHAPES = [(1, 64), (3, 8), (5, 1), (7, 100), (2, 1000), (300, 128), (9, 1024), (4, 1032), (3, 2048), (200, 2048), (5, 4096),
          (161, 4096), (2, 5120), (3, 8192), (2, 16384), (2, 20000)]


@gpu
@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, D, dtype, residual):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(T * 7 + D)
    x, w = rand(gen, T, D, dtype=dtype), 1 + 0.2 * rand(gen, D)
    r = rand(gen, T, D, dtype=dtype) if residual else None
    got = g.rms_norm(x, w, r, eps=1e-5, weight_offset=0.5)
    h, rstd, y = ref.norm(x, w, r, 1e-5, 0.5)
    half = 2 ** -8 if dtype == BF else 0
    near(got.rstd, rstd, 2 ** -20, "rstd")
    near(got.h, h, half + 2 ** -23, "h")
    # h in fp32 is off by 2^-24 of |x| + |r|, which cancellation can make large against h itself
    slack = 2 ** -23 * (x.cpu().double().abs() + (0 if r is None else r.cpu().double().abs())) * rstd[:, None] * 3
    assert ((got.y.cpu().double() - y).abs() <= (half + 2 ** -20) * y.abs() + slack).all()
    if residual:
        again = g.rms_norm(x, w, r.clone(), eps=1e-5, weight_offset=0.5, inplace=True)
        assert torch.equal(again.h, got.h) and torch.equal(again.y, got.y)
    else:
        assert got.h is x


@gpu
@pytest.mark.parametrize("T,D,group", [(1, 128, 128), (3, 1024, 128), (70, 4096, 128), (5, 2048, 0), (4, 1000, 0), (2, 8192, 128),
                                       (3, 7, 0), (2, 20096, 128), (2, 65536, 0), (200, 128, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_fp8(T, D, group, dtype):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(T + D)
    x, r, w = rand(gen, T, D, dtype=dtype), rand(gen, T, D, dtype=dtype), 1 + 0.2 * rand(gen, D)
    got = g.rms_norm(x, w, r, fp8=True, group=group)
    h, rstd, y = ref.norm(x, w, r)
    b = y.view(T, -1, group or D)
    scale = b.abs().amax(-1) / 448
    assert got.y.dtype == torch.float8_e4m3fn and got.scale.shape == scale.shape
    near(got.scale, scale, 2 ** -19, "scale")
    back = got.y.cpu().float().double().view_as(b) * got.scale.cpu().double()[..., None]
    assert ((back - b).abs() <= (2 ** -4 + 2 ** -18) * b.abs() + 2 ** -10 * scale[..., None]).all()
    near(got.h, h, (2 ** -8 if dtype == BF else 0) + 2 ** -23, "h")


@gpu
@pytest.mark.parametrize("D,group", [(256, 128), (256, 0), (257, 0)])
def test_fp8_is_the_product_with_the_reciprocal_scale(D, group):
    """With rstd = 1 and a weight of 1, y is x: the 8-bit output is fp32 x * (448 / amax), rounded to e4m3, bit for bit."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(D + group)
    x = rand(gen, 400, D)
    x = x / x.double().square().mean(-1, keepdim=True).sqrt().float()
    w = torch.ones(D, device=DEV)
    got = g.rms_norm(x, w, fp8=True, group=group)
    y = x * got.rstd[:, None]
    b = y.view(400, -1, group or D)
    inv = torch.full((), 448.0, device=DEV) / b.abs().amax(-1, keepdim=True).clamp(min=1e-30)
    assert torch.equal(got.y.float().view_as(b), (b * inv).clamp(-448, 448).to(torch.float8_e4m3fn).float())


@gpu
def test_fp8_edges():
    """A row of zeros gives zeros and the floor's scale, a group of tiny values keeps its precision, NaN stays NaN in its
    row only, one huge value leaves the others at zero or nearly."""
    import gated_deltanet_linear_15_gb300 as g
    x = torch.randn(5, 256, device=DEV)
    x[0] = 0
    x[1, :128] *= 1e-12
    x[2, 3] = float("nan")
    x[3, 5] = 1e15
    w = torch.ones(256, device=DEV)
    r = g.rms_norm(x, w, fp8=True, group=128)
    q, s = r.y.float(), r.scale
    assert (q[0] == 0).all() and torch.allclose(s[0], torch.full_like(s[0], 1e-30 / 448))
    assert torch.isnan(q[2]).all() and not torch.isnan(q[[0, 1, 3, 4]]).any()
    _, _, y = ref.norm(x, w)
    assert ((q[1].cpu().double() * s[1].cpu().double().repeat_interleave(128) - y[1]).abs()
            <= (2 ** -4 + 2 ** -18) * y[1].abs() + 2 ** -10 * s[1].cpu().double().repeat_interleave(128)).all()
    assert q[3, 5].abs() == 448


@gpu
@pytest.mark.parametrize("T,D,group", [(700, 256, 128), (300, 512, 128), (50, 20096, 128), (300, 640, 128), (300, 257, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_fp8_in_place_off_the_16_byte_path(T, D, group, dtype):
    """Rows that begin one element off a 16-byte boundary, h in residual's place: the same bits as with an h of its own."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(D)
    x, w = rand(gen, T, D + 1, dtype=dtype)[:, 1:], 1 + 0.2 * rand(gen, D)
    r = rand(gen, T, D + 1, dtype=dtype)
    want = g.rms_norm(x, w, r[:, 1:], fp8=True, group=group)
    for _ in range(5):
        again = r.clone()[:, 1:]
        got = g.rms_norm(x, w, again, fp8=True, group=group, inplace=True)
        assert torch.equal(again, want.h) and torch.equal(got.scale, want.scale)
        assert torch.equal(got.y.view(torch.uint8), want.y.view(torch.uint8))


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_with_strides_and_odd_alignment(dtype):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(1)
    big = rand(gen, 9, 300, dtype=dtype)
    w = 1 + 0.1 * rand(gen, 256)
    for off in (0, 1, 8):
        x, r = big[:, off:off + 256], rand(gen, 9, 280, dtype=dtype)[:, :256]
        got, want = g.rms_norm(x, w, r), g.rms_norm(x.contiguous(), w, r.contiguous())
        near(got.y, want.y.cpu().double(), 2 ** -7 if dtype == BF else 2 ** -20, "y")
        assert torch.equal(got.h, want.h)
    x = rand(gen, 3, 4, 5, 64, dtype=dtype)
    got = g.rms_norm(x, w[:64].contiguous())
    assert got.y.shape == x.shape and got.rstd.shape == (3, 4, 5)
    assert torch.equal(got.y.view(-1, 64), g.rms_norm(x.view(-1, 64), w[:64].contiguous()).y)


@gpu
@pytest.mark.parametrize("T,D", SHAPES + [(0, 64), (1000, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("stream", [False, True])
def test_backward(T, D, dtype, stream):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(T + 3 * D)
    h, dy, w = rand(gen, T, D, dtype=dtype), rand(gen, T, D, dtype=dtype), 1 + 0.2 * rand(gen, D)
    dh = rand(gen, T, D, dtype=dtype) if stream else None
    rstd = ref.norm(h, w)[1].float().to(DEV)
    dx, dw = g.rms_norm_bwd(dy, h, w, rstd, dh, weight_offset=0.25)
    rx, rw = ref.norm_grads(dy, h, w, rstd, dh, 0.25)
    mag = (rstd.cpu().double()[:, None] * (w.cpu().double() + 0.25) * dy.cpu().double()).abs()
    mag = mag + (0 if dh is None else dh.cpu().double().abs()) + h.cpu().double().abs()
    assert ((dx.cpu().double() - rx).abs() <= (2 ** -8 if dtype == BF else 0) * rx.abs() + 2 ** -19 * mag).all()
    # fp32 sums of T terms in chains of at most T / 300 + 60: far below 2^-16 of the magnitude sum for these T
    wmag = (dy.cpu().double() * h.cpu().double() * rstd.cpu().double()[:, None]).abs().sum(0)
    assert ((dw.cpu().double() - rw).abs() <= 2 ** -18 * wmag + 1e-30).all()
    again = g.rms_norm_bwd(dy, h, w, rstd, dh, weight_offset=0.25)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@gpu
def test_gradient_by_differences():
    """Central differences of the fp32 forward along random directions: with a step of 2^-6 the second-order error is
    below 2^-10 of the derivative's scale here, fp32 noise (about 2^-22 * sqrt(elements) / step) below that."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(5)
    T, D, e = 6, 512, 2.0 ** -6
    x, r, w = rand(gen, T, D), rand(gen, T, D), 1 + 0.2 * rand(gen, D)
    gy, gh = rand(gen, T, D), rand(gen, T, D)

    def loss(x, r, w):
        o = g.rms_norm(x, w, r)
        return float((o.y.double() * gy.double()).sum() + (o.h.double() * gh.double()).sum())

    leaves = [t.clone().requires_grad_() for t in (x, r, w)]
    y, h = g.residual_rms_norm(leaves[0], leaves[2], leaves[1])
    ((y * gy).sum() + (h * gh).sum()).backward()
    assert torch.equal(leaves[0].grad, leaves[1].grad)
    for i, name in enumerate(("x", "residual", "weight")):
        u = rand(gen, *leaves[i].shape)
        up, down = [x, r, w], [x, r, w]
        up[i], down[i] = up[i] + e * u, down[i] - e * u
        num = (loss(*up) - loss(*down)) / (2 * e)
        ana = float((leaves[i].grad.double() * u.double()).sum())
        size = float((leaves[i].grad.double() * u.double()).norm())
        assert abs(num - ana) <= 2 ** -6 * size, (name, num, ana, size)


@gpu
def test_gradient_without_a_residual():
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(6)
    x, w, gy = rand(gen, 11, 96, dtype=BF), 1 + 0.2 * rand(gen, 96), rand(gen, 11, 96, dtype=BF)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    g.residual_rms_norm(a, b).backward(gy)
    rstd = g.rms_norm(x, w).rstd
    dx, dw = g.rms_norm_bwd(gy, x, w, rstd)
    assert torch.equal(a.grad, dx) and torch.equal(b.grad, dw)


@gpu
@pytest.mark.parametrize("residual", [False, True])
def test_second_derivatives_are_refused(residual):
    """The backward is a kernel that autograd does not see into: a second derivative raises instead of missing terms."""
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator().manual_seed(7)
    x, w, r = rand(gen, 5, 64).requires_grad_(), (1 + 0.2 * rand(gen, 64)).requires_grad_(), rand(gen, 5, 64)
    out = g.residual_rms_norm(x, w, r if residual else None)
    y = out[0] if residual else out
    dx = torch.autograd.grad(y.square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


@gpu
def test_binding_refuses():
    import gated_deltanet_linear_15_gb300 as g
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    for call in (lambda: g.rms_norm(x.half(), w), lambda: g.rms_norm(x, w.bfloat16()), lambda: g.rms_norm(x, w[:32]),
                 lambda: g.rms_norm(x, w, x[:2]), lambda: g.rms_norm(x, w, x.bfloat16()), lambda: g.rms_norm(x.cpu(), w),
                 lambda: g.rms_norm(x.t(), w[:4].contiguous()), lambda: g.rms_norm(x, w, eps=0.0),
                 lambda: g.rms_norm(x, w, fp8=True, group=128), lambda: g.rms_norm(x, w, fp8=True, group=32),
                 lambda: g.rms_norm(x, w, group=128), lambda: g.rms_norm_bwd(x, x, w, torch.ones(3, device=DEV)),
                 lambda: g.rms_norm_bwd(x, x[:2], w, torch.ones(4, device=DEV))):
        with pytest.raises((ValueError, RuntimeError)):
            call()


# ------------------------------------------------------------------ refusals of the C entry points (no GPU needed)
def _shape(**kw):
    s = _lib.GdnNormShape()
    s.rows, s.dim, s.dtype, s.eps = 4, 256, _lib.GDN_BF16, 1e-6
    s.x_row = s.r_row = s.h_row = s.y_row = 256
    for k, v in kw.items():
        if k == "reserved":
            s.reserved[0] = v
        else:
            setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(dim=0), 2), (dict(dim=65537), 2), (dict(rows=-1), 1), (dict(dtype=3), 1), (dict(eps=0.0), 1), (dict(eps=math.nan), 1),
    (dict(fp8=2), 1), (dict(group=128), 2), (dict(fp8=1, group=64), 2), (dict(fp8=1, group=128, dim=200), 2),
    (dict(weight_offset=math.inf), 1), (dict(x_row=-1), 1), (dict(y_row=255), 1), (dict(h_row=100), 1), (dict(reserved=1), 1),
])
def test_c_entry_refuses_shapes(lib, kw, code):
    p = 0x10000
    assert lib.gdn_rmsnorm_fwd(ctypes.byref(_shape(**kw)), p, p, p, p, p, p, p, None) == code
    assert lib.gdn_last_error_string() != b""


def test_c_entry_refuses_arguments(lib):
    p, big = 0x10000, 1 << 40
    s = _shape(fp8=1)
    for i in (0, 2, 4, 5):   # x, weight, y, scale
        a = [p] * 7
        a[i] = None
        assert lib.gdn_rmsnorm_fwd(ctypes.byref(s), *a, None) == 1, i
    assert lib.gdn_rmsnorm_fwd(ctypes.byref(_shape(rows=0)), *[None] * 7, None) == 0
    s = _shape()
    need = lib.gdn_rmsnorm_bwd_workspace_size(ctypes.byref(s))
    assert need > 0
    for i in (0, 1, 2, 3, 5, 6):   # dy, h, weight, rstd, dx, dw
        a = [p] * 7
        a[i] = None
        assert lib.gdn_rmsnorm_bwd(ctypes.byref(s), *a, p, big, None) == 1, i
    assert lib.gdn_rmsnorm_bwd(ctypes.byref(s), *[p] * 7, p, need - 1, None) == 3
    assert lib.gdn_rmsnorm_bwd(ctypes.byref(s), *[p] * 7, None, big, None) == 3
    assert lib.gdn_rmsnorm_bwd(ctypes.byref(_shape(h_row=10)), *[p] * 7, p, big, None) == 1
    assert lib.gdn_rmsnorm_bwd_workspace_size(ctypes.byref(_shape(dim=0))) == 0
