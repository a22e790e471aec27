"""The rounding of an 8-bit momentum in the numpy oracle: where to nearest it decays, that the random one keeps its mean,
and that no step of a row without gradient grows."""

import numpy as np
import pytest
import torch

from oracle import tensor_set as T

F = np.float32


@pytest.fixture(scope="module")
def zp():
    import os
    from sharded_zero_partition_amd import build as zbuild
    if not os.path.exists(zbuild.LIB):
        zbuild.build()
    import sharded_zero_partition_amd as z
    return z


def test_to_nearest_every_code_falls_up_to_the_limit():
    """beta1 times a code, for every one above 2^-6 (the block's largest holds the scale): below it up to the limit; at
    0.945 (past 17/18) 1.125 stays."""
    m = T.E4M3[9:127].astype(np.float32)
    top = np.float32(256)                                       # keeps the scale at 2^0 in blocks of one code and itself
    for beta1, falls in ((T.NEAREST_BETA1, True), (0.9, True), (0.5, True), (0.945, False), (0.99, False)):
        pairs = np.zeros((m.size, T.BLOCK), np.float32)
        pairs[:, 0], pairs[:, 1] = top, m * F(beta1)
        code, s = T.encode(pairs.ravel(), False)
        assert (s == 127).all()
        after = T.E4M3[code.reshape(-1, T.BLOCK)[:, 1]]
        assert (after < m).all() == falls, beta1
        if not falls:
            assert (after[m == 1.125 * 2.0 ** np.floor(np.log2(m))] == m[m == 1.125 * 2.0 ** np.floor(np.log2(m))]).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_random_rounding_of_m_keeps_the_mean_down_to_zero(sign):
    """As for v, but with signs, and values below the least number go to zero or to it.  A value's deviation is half the
    gap at most, so 6 gap / 2 / sqrt(N); the 16-bit chances add gap 2^-17."""
    x = (sign * np.concatenate([[1.0], np.linspace(1e-6, 1.0, 25), 2.0 ** -8 / 448 * np.array([.01, .1, .3, .5, .9, 1.7])])).astype(np.float32)
    N = 4000
    got = np.array([T.decode(*T.encode(x, False, T.chances(32, 7, 3, t, of_m=True))) for t in range(N)], np.float64)
    power = 2.0 ** (float(T.encode(x, False)[1][0]) - 127)
    grid, a = T.E4M3[:127] * power, np.abs(x.astype(np.float64))
    hi = np.searchsorted(grid, a, side="left")
    lo = np.where(grid[hi] == a, hi, hi - 1)
    for k in range(32):
        assert set(np.unique(np.abs(got[:, k]))) <= {grid[lo[k]], grid[hi[k]]}
        assert (got[:, k] * sign >= 0).all()
    gap = grid[hi] - grid[lo]
    assert (np.abs(got.mean(0) - x) <= 6 * gap / 2 / np.sqrt(N) + gap * 2.0 ** -17).all()


def test_m_and_v_take_other_bits():
    """16 bits each: N pairs of independent ones are equal in N 2^-16 of the cases, give or take 6 of its roots."""
    n = 1 << 20
    a, b = T.chances(n, 5, 2, 9), T.chances(n, 5, 2, 9, of_m=True)
    assert abs(int((a == b).sum()) - n / 65536) <= 6 * np.sqrt(n / 65536)
    x, y = a / 65536 - 0.5, b / 65536 - 0.5
    assert abs((x * y).mean()) <= 6 / 12 / np.sqrt(n)            # each of variance 1/12


@pytest.mark.parametrize("beta1,beta2,always", [(0.9, 0.95, False), (0.9, 0.95, True), (0.95, 0.95, False), (0.95, 0.999, False), (0.99, 0.999, False)])
def test_rows_whose_gradients_end_stop_moving(beta1, beta2, always):
    """200 steps of noise, then none.  |m| / sqrt(v) falls by 0.9775 a step at least in the mean over the rounding
    where beta2 is 0.95 (beta1 0.95 over v's root 0.9747, and 1.003 for v's random error: its variance is v^2 / 256 a step
    at most, 3/8 of that, doubled, for the curve of 1 / sqrt), and by 0.9905 1.003 = 0.9935 for 0.99 and 0.999.  From 4 at
    most, 1200 steps after the last gradient the way that is left is 4 0.9935^1200 / 0.0065 lr = 0.25 lr in the mean, and
    1e-9 lr in the other cases.  A step is 10 lr only where an element is 6000 times the mean of what is left then."""
    n, end, lr = 1024, 2600, 1e-4
    rng = np.random.default_rng(1)
    h, c = T.HParams(lr=lr, beta1=beta1, beta2=beta2), T.Control()
    p = np.zeros(n, np.float32)
    m, ms = T.encode(p, False)
    v, vs = T.encode(p, True)
    at = {}
    for step in range(end):
        g = (rng.standard_normal(n) * 1e-3).astype(np.float32) if step < 200 else np.zeros(n, np.float32)
        assert c.begin([h], check=False)
        p, mw, vw = T.adamw(c.consts[0], g, 1.0, p, T.decode(m, ms), T.decode(v, vs))
        m, ms = T.encode_m(mw, h.beta1, 3, 0, c.t, always)
        v, vs = T.encode(vw, True, T.chances(n, 3, 0, c.t))
        if step == 1399:
            at = p.copy()
    assert np.isfinite(p).all() and np.abs(p - at).max() <= 10 * lr


def test_m_rounding_refusals(zp):
    assert zp.lib.zero_tensor_set_m_rounding(None, 0) == -1
    z = torch.zeros(4)
    for name in ("nearest", None, 1):
        with pytest.raises(ValueError, match="m_rounding"):
            zp.TensorSet(m=[z], v=[z.clone()], m_rounding=name)


def test_a_variance_of_negative_zeros_is_zero():
    v = np.array([-0.0, 1e-6, 0.0, 3e-7] + [-0.0] * 28, np.float32)
    code, s = T.encode(v, True)
    same, t = T.encode(np.abs(v), True)
    assert np.array_equal(code, same) and np.array_equal(s, t) and not (code & 128).any()
