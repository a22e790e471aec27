"""The weight gradient in large tiles, whole and split by tokens, and in small ones: whole numbers exactly, common scales
of fp16 products against their bound."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES, Guarded
from oracle import activations as A

pytestmark = pytest.mark.gpu

# tokens, outputs n, inputs k, elements behind a row of dy: aligned rows and others, tokens that end inside a turn of ten
# phases, whole rounds of tiles and some over, one to many tiles along k
SHAPES = [(193, 4352, 4096, 0), (200, 4100, 4090, 4), (257, 4096, 4111, 1), (333, 4098, 4000, 6), (1003, 70002, 200, 6),
          (1290, 20000, 500, 0), (1283, 4252, 4096, 4), (2500, 2560, 1600, 0), (4099, 2050, 2040, 6), (4099, 2049, 2040, 7),
          (130, 5120, 5000, 0), (64, 5000, 5120, 3), (1000, 777, 555, 0), (3333, 768, 768, 0), (9000, 130, 70, 6)]


def whole(T, n, k, dtype, pad, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = Guarded(T, n, dtype, 0, pad, torch.randint(-3, 4, (T, n), device="cuda", generator=g, dtype=torch.int8))
    x = torch.randint(-8, 9, (T, k), device="cuda", generator=g, dtype=torch.int8).float()
    c = zp.Checkpoint(T, k)
    c.store(x)
    return dy, x, c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k,pad", SHAPES)
def test_whole_numbers(dtype, T, n, k, pad):
    """Sums of magnitudes stay below 9000 * 24 < 2^24, so every partial sum is exact in fp32."""
    t = DTYPES[dtype]
    if dtype == "fp32" and T * n * k > 2 ** 34:
        T = T // 4 + 1
    dy, x, c = whole(T, n, k, t, pad, T + n)
    want = dy.t.double().t() @ x.double()
    bias = dy.t.double().sum(0)
    w, b = Guarded(n, k, torch.float32, 0, 0), Guarded(1, n, torch.float32)
    zp.weight_grad(dy.t, c, w.t, bias=b.t[0])
    assert torch.equal(w.t.double(), want) and torch.equal(b.t[0].double(), bias)
    zp.weight_grad(dy.t, c, w.t, bias=b.t[0], accumulate=True)
    assert torch.equal(w.t.double(), 2 * want) and torch.equal(b.t[0].double(), 2 * bias)
    assert w.untouched() and b.untouched() and dy.untouched()
    other = Guarded(k, n, t, 0, 2)
    zp.weight_grad(dy.t, c, other.t.t())
    assert torch.equal(other.t.t(), want.to(torch.float32).to(t)) and other.untouched()


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_bits_at_any_alignment(dtype):
    t = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(5)
    T, n, k = 1100, 4098, 2040
    dy = torch.randn(T, n, device="cuda", generator=g).to(t)
    c = zp.Checkpoint(T, k)
    c.store(torch.randn(T, k, device="cuda", generator=g) * 2.0 ** torch.randint(-9, 3, (T, 1), device="cuda", generator=g))
    out = []
    for off, pad in ((0, 6), (1, 6), (8, 14), (0, 1)):
        other, w, b = Guarded(T, n, t, off, pad, dy), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        zp.weight_grad(other.t, c, w, bias=b)
        out.append((w, b))
    for w, b in out[1:]:
        assert torch.equal(w, out[0][0]) and torch.equal(b, out[0][1])


@pytest.mark.parametrize("T,n,k", [(70, 40, 70), (700, 300, 65), (200, 4100, 4090), (4099, 2050, 2040)])
def test_scales_of_every_size(T, n, k):
    """With fp16 gradients a value is rounded to a multiple of 2^-24, half of that off, in a scale where the columns' largest
    block has at most 57344 = 448 2^7 for 448 2^(top - 127): 2^(top - 127) 2^-32 off.  Blocks that are NaN count for no
    scale and stay in their columns."""
    g = torch.Generator(device="cuda").manual_seed(T)
    b = A.blocks(k)
    x = torch.randn(T, k, device="cuda", generator=g)
    power = torch.randint(-60, 30, (T, b), device="cuda", generator=g).float()
    power[:, 1::2] = torch.randint(-30, -20, (T, 1), device="cuda", generator=g).float()       # near each other, and small
    x *= torch.exp2(power).repeat_interleave(32, 1)[:, :k]
    c, x64 = zp.Checkpoint(T, k), torch.empty(T, k, device="cuda")
    c.store(x)
    c.load(x64)
    x64 = x64.double()
    dy = torch.randn(T, n, device="cuda", generator=g).half()
    top = c.scale.max(0).values.double().repeat_interleave(32)[:k]
    w = torch.empty(n, k, device="cuda")
    zp.weight_grad(dy, c, w)
    want, mag, most = dy.double().t() @ x64, dy.double().abs().t() @ x64.abs(), dy.double().abs().sum(0)[:, None]
    # the sums' own roundings, as for equal scales: a unit of fp32 for each, of the magnitudes so far
    bound = (T + 2) * 2.0 ** -23 * mag + most * torch.exp2(top - 127 - 32)
    assert bool(((w.double() - want).abs() <= bound).all())
    c.code[T // 2, 32:64] = 0x7F
    c.scale[T // 2, 1] = 255
    again = torch.empty_like(w)
    zp.weight_grad(dy, c, again)
    bad = torch.zeros(k, dtype=torch.bool, device="cuda")
    bad[32:64] = True
    assert bool(again[:, bad].isnan().all())
    assert torch.equal(again[:, ~bad], w[:, ~bad])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(1003, 70000), (200, 4096), (40, 100), (9000, 64)])
def test_a_bias_alone(dtype, T, n):
    """A layer of no inputs, whose gradient is that of its bias."""
    dy = Guarded(T, n, DTYPES[dtype], 0, 0, torch.randint(-3, 4, (T, n), device="cuda", dtype=torch.int8))
    b = torch.ones(n, device="cuda")
    zp.weight_grad(dy.t, zp.Checkpoint(T, 0), torch.empty(n, 0, device="cuda"), bias=b, accumulate=True)
    assert torch.equal(b.double(), dy.t.double().sum(0) + 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", [(40, 24, 70), (200, 4096, 4096)])
def test_the_smallest_values(dtype, T, n, k):
    """Values of x below 2^-126 are rounded in bf16 to multiples of 2^-133, a half of that off (with fp16 gradients their common
    scale keeps them); sums are off by a unit of fp32 of the magnitudes, or 2^-149, for each token."""
    t = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, k, device="cuda", generator=g) * torch.exp2(-torch.randint(118, 140, (1, k), device="cuda", generator=g).float())
    c, x64 = zp.Checkpoint(T, k), torch.empty(T, k, device="cuda")
    c.store(x)
    c.load(x64)
    x64 = x64.double()
    dy = torch.randn(T, n, device="cuda", generator=g).to(t)
    w = torch.empty(n, k, device="cuda")
    zp.weight_grad(dy, c, w)
    want, mag, most = dy.double().t() @ x64, dy.double().abs().t() @ x64.abs(), dy.double().abs().sum(0)[:, None]
    low = torch.zeros_like(most) if dtype == "fp16" else most * 2.0 ** -134
    assert bool(((w.double() - want).abs() <= 3 * (T + 2) * (2.0 ** -23 * mag + 2.0 ** -149) + low).all())


def test_more_than_2_31_bytes_of_gradients():
    """Sums of 65536 whole numbers up to 24 are exact in fp32, the library's too."""
    T, n, k = 65536, 20480, 4200
    dy, x, c = whole(T, n, k, torch.bfloat16, 0, 9)
    w, b = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    zp.weight_grad(dy.t, c, w, bias=b)
    wide = dy.t.float()
    assert torch.equal(w, wide.t() @ x) and torch.equal(b, wide.sum(0))
