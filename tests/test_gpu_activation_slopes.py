"""Gradients of the sigmoid activations in fp32 against 64 bits, as near as their roundings leave them."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from oracle import activations as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of fp32, relative


def deviation(z, d, p, angle):
    """Standard deviation of act'(z) = p + t, t = z p (1 - p) a'(z), with every rounding at most its half unit and at random:
    a rounding of k half units of c has the variance (k U c)^2 / 3.  In order: the angle's two constants, sum and product, and
    the product with log2(e), each moving a by U a, so act' by da = p (1 - p) + t (1 - 2 p) times that; exp2 (a unit); 1 + e
    and its reciprocal (a unit), p being in act' once and in t twice; e p, z p, the slope's constants and sum (one each, halves
    of two constants), the product with the slope; the last sum."""
    t = d - p
    da = p * (1 - p) + t * (1 - 2 * p)
    squares = 5 * (da * angle) ** 2 + 4 * da ** 2 + 5 * (p + 2 * t) ** 2 + 5 * t ** 2 + d ** 2
    return U * np.sqrt(squares / 3)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_slopes_in_fp32(kind):
    """All values that a checkpoint holds exactly from 2^-6 to 6: the deviations' mean square is 1 at most (2 with the
    spread of some 140 values, of which a tenth is one deviation of that mean), and none of them is 6.  A slope whose constant
    is off by 64 steps has a mean square of 4.6."""
    z = (np.arange(8, 16) * 2.0 ** np.arange(-9, 0)[:, None]).ravel()
    z = np.concatenate([-z[z <= 6], z[z <= 6]])
    n = len(z)
    c, dx = zp.Checkpoint(n, 1), torch.empty(n, 1, device="cuda")
    c.store(torch.from_numpy(z[:, None]).float().cuda())
    c.load(dx)
    assert np.array_equal(dx.double().cpu().numpy()[:, 0], z)
    zp.activation_grad(kind, torch.ones(n, 1, device="cuda"), c, dx)
    d, a = A.act(kind, z)[1], A.angle(kind, z)
    off = (dx.double().cpu().numpy()[:, 0] - d) / deviation(z, d, 1 / (1 + np.exp(-a)), np.abs(a))
    assert (off ** 2).mean() <= 2 and np.abs(off).max() <= 6, ((off ** 2).mean(), np.abs(off).max())
