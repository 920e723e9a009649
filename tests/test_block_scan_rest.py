"""Packed batches with rows that no sequence names (padding before the first or behind the last one): through the gated linear
recurrence with gradients they are zeros in the output and in both gradients, so that what is summed over all rows, the gradient
of a projection before or behind it, takes nothing from them."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests.test_block_scan import BF, DEV, F32, TYPES, bound, inputs, lib, loop, loop_bwd, near  # noqa: F401

gpu = pytest.mark.gpu
CU = [[5, 20, 40], [0, 20, 40], [0, 0, 0], [30, 60, 90], [16, 16, 48], [90, 90, 90], [17, 18, 89]]


def dirty(*tensors):
    """Memory that the allocator hands out next for tensors of these sizes holds NaN."""
    held = [torch.full_like(t, float("nan")) for t in tensors for _ in range(3)]
    torch.cuda.synchronize()
    del held


def named(cu, tokens):
    keep = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    keep[cu[0]:cu[-1]] = True
    return keep


@gpu
@pytest.mark.parametrize("cu", CU)
@pytest.mark.parametrize("D", [64, 130, 37])  # rows by 16 bytes, by pairs (bf16), and from anywhere
@pytest.mark.parametrize("dtype,gate", TYPES)
def test_gradients_of_rows_that_no_sequence_names(cu, D, dtype, gate):
    import gated_deltanet_linear_15_gb300 as g
    i = inputs([90], D, dtype, gate, True)
    dev, h0, keep = torch.tensor(cu, dtype=torch.int32, device=DEV), torch.randn(2, D, device=DEV), named(cu, 90)
    leaves = [i["x"].clone().requires_grad_(), i["g"].clone().requires_grad_(), h0.requires_grad_()]
    dirty(i["x"], i["g"])
    y, final = g.gated_linear_recurrence(*leaves, cu_seqlens=dev)
    dirty(i["x"], i["g"])
    dT = torch.randn(2, D, device=DEV)
    dx, dg, dh0 = torch.autograd.grad((y, final), leaves, (i["dy"], dT))
    for t in (y, dx, dg):
        assert (t[0, ~keep] == 0).all()
    line = {k: i[k][0] for k in ("x", "g", "dy")}
    h, m, hT, mT, hp, mp = loop(line["x"], line["g"], h0.detach(), cu)
    d, md, f, mf, d0, m0 = loop_bwd(line["dy"], line["g"], dT, cu)
    w, tol, kind, gkind = slice(cu[0], cu[-1]), bound(90), "bf16" if dtype == BF else "fp32", "bf16" if gate == BF else "fp32"
    near(y[0, w], h[w], tol * m[w], "y " + kind)
    near(dx[0, w], d[w], tol * md[w], "dx " + kind)
    near(dg[0, w], (f * hp)[w], 2 * tol * (mf * mp)[w], "dg " + gkind)
    near(final, hT, tol * mT, "final")
    near(dh0, d0, tol * m0, "dh0")


@gpu
def test_gradients_of_projections_around_a_padded_batch():
    """x = u A before and z = y B behind, with rows behind the last sequence that hold anything finite: the gradients of A and B are
    those of the batch without them."""
    import gated_deltanet_linear_15_gb300 as g
    gen, D, T, n = torch.Generator().manual_seed(3), 64, 200, 150
    u, gates = torch.randn(T, D, generator=gen).to(DEV), -torch.rand(1, T, D, generator=gen).to(DEV)
    dz = torch.randn(T, D, generator=gen).to(DEV)
    dz[n:] = 0
    cu = torch.tensor([0, 70, n], dtype=torch.int32, device=DEV)

    def grads(rows):
        A, B = (torch.randn(D, D, generator=torch.Generator().manual_seed(s)).to(DEV).requires_grad_() for s in (1, 2))
        x = (u[:rows] @ A)[None]
        dirty(x)
        y, _ = g.gated_linear_recurrence(x, gates[:, :rows].contiguous(), cu_seqlens=cu)
        z = y[0] @ B
        dirty(x)
        return torch.autograd.grad(z, (A, B), dz[:rows])

    for got, want in zip(grads(T), grads(n)):
        assert torch.isfinite(got).all()
        # values of some bound(80) < 2^-16 of ten times their size, in sums of 150 whose size is some sqrt(150) terms
        assert (got - want).abs().max() <= 2.0 ** -8 * want.abs().max()


@gpu
@pytest.mark.parametrize("cu", [[0, 3000, 5000], [1000, 5000, 7000], [8300, 8300, 8300]])
def test_long_padding(cu):
    """More rows of padding than one warp clears, many channel blocks."""
    import gated_deltanet_linear_15_gb300 as g
    x = torch.ones(1, 8300, 2001, device=DEV)
    dev, keep = torch.tensor(cu, dtype=torch.int32, device=DEV), named(cu, 8300)
    dirty(x)
    y, final, states = g.gated_scan(x, -x, cu_seqlens=dev, save_states=True)
    dirty(x)
    dx, dg, _ = g.gated_scan_bwd(x, x, -x, states, None, final, cu_seqlens=dev)
    for t in (y, dx, dg):
        assert (t[0, ~keep] == 0).all() and torch.isfinite(t).all() and (t[0, keep] != 0).any() == keep.any()


def test_c_entry_refuses(lib):  # noqa: F811
    shape = dict(num_seqs=2, tokens=20, dim=64, dtype=_lib.GDN_BF16, gate_dtype=_lib.GDN_FP32, x_row=64, g_row=64, y_row=64, dy_row=64,
                 dg_row=64, state_row=64)
    p = [0x10000 * (i + 1) for i in range(10)]
    for kw in (dict(zero_rest=2), dict(zero_rest=-1), dict(reserved1=1)):
        s = _lib.GdnScanShape(**shape, **kw)
        assert lib.gdn_scan_fwd(ctypes.byref(s), p[0], p[1], None, p[2], p[3], None, None, None) == 1, kw
        assert lib.gdn_scan_bwd(ctypes.byref(s), *p[:4], None, None, p[4], p[5], p[6], None, None) == 1, kw
        assert lib.gdn_scan_states_rows(ctypes.byref(s)) == -1, kw
