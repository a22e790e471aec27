"""relu of a negative zero is z > 0 ? z : 0, so zero: in the oracle, and bit for bit on the GPU."""

import numpy as np
import pytest
import torch

from oracle import activations as A


def test_the_oracle():
    a, d, _ = A.act("relu", np.array([-0.0, 0.0, -1.0, 2.0, np.nan]))
    assert not np.signbit(a[:4]).any() and a[:4].tolist() == [0, 0, 0, 2] and np.isnan(a[4]) and np.isnan(d[4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_the_kernels(dtype):
    import sharded_zero_partition_amd as zp
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    x = torch.tensor([[-0.0, 0.0, -2.0, 3.0] * 10, [-0.0] * 40], device="cuda").to(dtype)
    want = torch.tensor([[0.0, 0.0, 0.0, 3.0] * 10, [0.0] * 40], device="cuda").to(dtype)
    ones, h = torch.ones_like(x), torch.empty_like(x)
    cx, cu, ch = (zp.Checkpoint(2, 40) for _ in range(3))
    for gate in ({}, dict(up=ones, up_checkpoint=cu)):
        zp.activation("relu", x, h, cx, out_checkpoint=ch, **gate)
        assert torch.equal(h.view(bits), want.view(bits))
        assert bool((ch.code[:, :40].view(2, 10, 4)[..., :3] == 0).all())
        assert bool((cx.code[1, :40] == 0x80).all())                    # what is kept of x keeps its sign
    dx, du = torch.empty_like(x), torch.empty_like(x)
    zp.activation_grad("relu", ones, cx, dx, up_checkpoint=cu, dup=du)
    assert torch.equal(du.view(bits), want.view(bits)) and torch.equal(dx, (want > 0).to(dtype))
    x[0, 0] = float("nan")
    zp.activation("relu", x, h)
    assert bool(h[0, 0].isnan())
