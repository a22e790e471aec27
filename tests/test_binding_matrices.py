"""How the binding takes tensors as matrices, on the CPU (whose tensors are on device -1)."""

import pytest
import torch

from test_activations_host import zp   # noqa: F401


@pytest.mark.parametrize("shape,strides,rows,cols,stride", [
    ((2, 3, 5), None, 6, 5, 5), ((7,), None, 1, 7, 7), ((2, 3, 1), None, 6, 1, 1), ((2, 3, 5), (36, 12, 1), 6, 5, 12),
    ((4, 3, 5), (0, 0, 1), 12, 5, 0), ((2, 0, 5), None, 0, 5, None), ((2, 3, 0), None, 6, 0, None), ((0, 3, 0), None, 0, 0, None),
    ((6, 0), None, 6, 0, None)])
def test_shapes(zp, shape, strides, rows, cols, stride):   # noqa: F811
    t = torch.zeros(200)
    t = torch.zeros(shape) if strides is None else t.as_strided(shape, strides)
    m = zp.binding._matrix(t, "x", -1)
    assert (m.rows, m.cols) == (rows, cols) and stride in (None, m.stride)


def test_refusals(zp):   # noqa: F811
    for t in (torch.zeros(()), torch.zeros(200).as_strided((2, 3, 5), (40, 12, 1)), torch.zeros(4, 6)[:, ::2], torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            zp.binding._matrix(t, "x", -1)
