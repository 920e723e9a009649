"""The norm of heads with its turn where eps is as small as its type allows: r = 1 / sqrt(mean(x^2) + eps) is large then, and
its powers leave fp32 long before the gradients do.  Against the definition in 64 bits with the bounds of
tests/test_block_norm_rotary.py."""
import pytest
import torch

from tests.test_block_norm_rotary import BF, DEV, F32, F64, backward, forward, inputs, lib, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 96, 7])  # heads by units, and a warp to a head
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eps", [1e-20, 1e-28, 1e-36, 1e-42])
def test_heads_of_zeros_and_small_ones(D, dtype, eps):
    """A head of zeros has the gradient r u w; one of some 1e-15 has what the definition says."""
    import gated_deltanet_linear_15_gb300 as g
    i = inputs(6, 2, 1, D, D // 2 * 2, dtype)
    q, k = i["q"].clone(), i["k"].clone()
    q[1], k[3], q[4] = 0, 0, q[4] * 2.0 ** -50  # exact in both types
    args = (q, k, i["wq"], i["wk"], i["table"], i["pos"])
    y = g.norm_rotary(*args, eps=eps)
    got = g.norm_rotary_bwd(i["dq"], i["dk"], *args, eps=eps)
    eps = float(torch.tensor(eps, dtype=F32))  # as the kernel has it
    for x, w, dy, out, dx, dw in ((q, i["wq"], i["dq"], y[0], got[0], got[2]), (k, i["wk"], i["dk"], y[1], got[1], got[3])):
        want, size = forward(x, w, i["table"], i["pos"], eps, 0.0, False)
        near(out, want, 2.0 ** -19 * size, "y", dtype)
        wx, sx, ww, sw = backward(dy, x, w, i["table"], i["pos"], eps, 0.0, False)
        assert torch.isfinite(dx).all()
        near(dx, wx, 2.0 ** -18 * sx, "dx", dtype)
        near(dw, ww, (2.0 ** -18 + x.shape[0] * x.shape[1] * 2.0 ** -24) * sw, "dw", F32)
