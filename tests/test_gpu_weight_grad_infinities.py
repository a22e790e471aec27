"""Infinite and NaN gradients in the weight gradient: what the sums of the definition are, in every type and kernel."""

import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES

pytestmark = pytest.mark.gpu


# small tiles, large ones, and those split by tokens; aligned rows of dy and others
@pytest.mark.parametrize("T,n,k", [(70, 60, 40), (200, 150, 300), (1003, 1030, 520), (300, 4100, 4090), (4099, 2049, 70)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sums_with_infinities(dtype, T, n, k):
    """Whole numbers, so finite sums are exact; with an infinity a sum is infinite, or NaN where it meets a zero, the other
    infinity or a NaN."""
    t = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randint(-3, 4, (T, n), device="cuda", generator=g).to(t)
    x = torch.randint(-8, 9, (T, k), device="cuda", generator=g).float()
    inf = float("inf")
    dy[7, 20], dy[T - 1, 30], dy[11, 40], dy[12, 40], dy[13, 50] = inf, -inf, inf, -inf, float("nan")
    if dtype == "fp32":     # a NaN whose upper half is an infinity's
        dy.view(torch.int32)[13, 50] = 0x7F800001
    c, dw, db = zp.Checkpoint(T, k), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    c.store(x)
    zp.weight_grad(dy, c, dw, bias=db)
    assert db[20] == inf and db[30] == -inf and db[40].isnan() and db[50].isnan()
    for row, token, sign in ((20, 7, 1), (30, T - 1, -1)):
        assert torch.equal(dw[row] == inf, sign * x[token] > 0) and torch.equal(dw[row] == -inf, sign * x[token] < 0)
        assert torch.equal(dw[row].isnan(), x[token] == 0)
    both = torch.where(x[11] * x[12] < 0, x[11] * inf, inf - inf)       # inf x11 - inf x12
    assert torch.equal(dw[40].isnan(), both.isnan()) and torch.equal(dw[40].nan_to_num(), both.nan_to_num())
    assert bool(dw[50].isnan().all())
    clean = torch.ones(n, dtype=torch.bool, device="cuda")
    clean[[20, 30, 40, 50]] = False
    wide = dy.double()[:, clean].t().contiguous()
    assert torch.equal(dw[clean].double(), wide @ x.double()) and torch.equal(db[clean].double(), wide.sum(1))
