"""Matrices on the device whose surroundings are guarded: any start, any distance between rows."""

import numpy as np
import torch

import sharded_zero_partition_amd as zp
from oracle import activations as A

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
GUARD = 0x5A


class Guarded:
    """A [rows, cols] view, `off` elements into a buffer, rows `cols + pad` apart; all around it bytes of 0x5A.  `values`
    (fp32 or what the dtype holds) are rounded by torch."""

    def __init__(self, rows, cols, dtype, off=0, pad=0, values=None):
        size = torch.empty(0, dtype=dtype).element_size()
        n = off + rows * (cols + pad) + 64
        self.buf = torch.full((n * size,), GUARD, dtype=torch.uint8, device="cuda")
        self.t = self.buf.view(dtype).as_strided((rows, cols), (cols + pad, 1), off)
        if values is not None:
            self.t.copy_(torch.as_tensor(values).to(dtype))
        inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        inside.as_strided((rows, cols), (cols + pad, 1), off).fill_(True)
        self.outside = ~inside.repeat_interleave(size)

    def untouched(self):
        return bool((self.buf[self.outside] == GUARD).all())

    def wide(self):
        return self.t.to(torch.float64).cpu().numpy()


class Kept:
    """A checkpoint with guards behind its codes and scales, which may start anywhere they are allowed to."""

    def __init__(self, rows, cols, scale_off=0):
        b = A.blocks(cols)
        self.code = torch.full((rows * b * 32 + 96,), GUARD, dtype=torch.uint8, device="cuda")
        self.scale = torch.full((rows * b + 96,), GUARD, dtype=torch.uint8, device="cuda")
        self.n, self.m, self.off = rows * b * 32, rows * b, scale_off
        self.c = zp.Checkpoint(code=self.code[32:32 + self.n].view(rows, b * 32),
                               scale=self.scale[scale_off:scale_off + self.m].view(rows, b), cols=cols)

    def fill(self, code, scale):
        self.c.code.copy_(torch.from_numpy(code))
        self.c.scale.copy_(torch.from_numpy(scale))
        return self

    def host(self):
        return self.c.code.cpu().numpy(), self.c.scale.cpu().numpy()

    def untouched(self):
        outside = [self.code[:32], self.code[32 + self.n:], self.scale[:self.off], self.scale[self.off + self.m:]]
        return all(bool((x == GUARD).all()) for x in outside)


def held(x, dtype):
    """fp32 values as the dtype holds them, in fp32."""
    return torch.as_tensor(x).to(dtype).to(torch.float32).numpy()


def half_unit(x, dtype):
    """The most that rounding to the dtype moves a value: half a step of its own, or of the smallest numbers."""
    f = torch.finfo(dtype)
    return np.maximum(np.abs(x) * f.eps / 2, f.smallest_normal * f.eps / 2)


def activations(rng, rows, cols):
    """Values of every size a layer may see, with blocks of zeros and negative zeros."""
    x = (rng.standard_normal((rows, cols)) * 2.0 ** rng.uniform(-8, 3, (rows, 1))).astype(np.float32)
    x[:, rng.random(cols) < 0.03] *= 50
    x[rng.random((rows, cols)) < 0.02] = 0
    x[rng.random((rows, cols)) < 0.02] = -0.0
    x[rows // 2, : 40] = 0
    return x
