"""Conversion of states on the GPU: zeros of either sign."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from oracle import tensor_set as T

pytestmark = pytest.mark.gpu


def codes(sizes):
    return [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]


@pytest.mark.parametrize("gap", [0, 1, 32])
def test_negative_zeros_are_zeros(gap):
    """-0.0 is not negative: a v that holds one has its block's scale from the others, and becomes zero."""
    rng = np.random.default_rng(gap)
    sizes = [1, 5, 32, 33, 64, 1024, 1025, 5000]
    v = [np.square(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in sizes]
    for k, x in enumerate(v):
        x[rng.random(x.size) < 0.3] = -0.0
        x[: 32 if k % 2 else 0] = -0.0                         # whole blocks of them
    m = [np.where(rng.random(n) < 0.5, np.float32(-0.0), rng.standard_normal(n).astype(np.float32)) for n in sizes]
    wide = [[torch.cat([torch.zeros(gap), torch.from_numpy(x)]).cuda()[gap:] for x in lst] for lst in (m, v)]
    src = zp.TensorSet(m=wide[0], v=wide[1])
    blocks = [-(-n // 32) for n in sizes]
    cm, cv, sm, sv = codes(sizes), codes(sizes), codes(blocks), codes(blocks)
    zp.TensorSet(m=cm, v=cv, m_scale=sm, v_scale=sv).states_from(src)
    for i in range(len(sizes)):
        for x, c, s, positive in ((m[i], cm[i], sm[i], False), (v[i], cv[i], sv[i], True)):
            code, scale = T.encode(x, positive)
            assert np.array_equal(s.cpu().numpy(), scale), (i, positive)
            assert np.array_equal(c.cpu().numpy(), code), (i, positive)
    back = [[torch.empty(n, device="cuda") for n in sizes] for _ in range(2)]
    zp.TensorSet(m=back[0], v=back[1]).states_from(zp.TensorSet(m=cm, v=cv, m_scale=sm, v_scale=sv))
    for x, y in zip(back[1], v):
        assert np.array_equal(x.cpu().numpy() > 0, y > 0)
        # a unit is at most an eighth of the value, or 2^-9 of a scale whose block's largest is above 224
        top = np.repeat(np.abs(T._blocks(y)).max(1), 32)[:y.size].astype(np.float64)
        assert (np.abs(x.cpu().numpy().astype(np.float64) - y) <= np.maximum(np.abs(y) / 8, top * 2.0 ** -9 / 224)).all()
