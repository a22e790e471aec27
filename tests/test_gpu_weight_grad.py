"""The weight gradient from an 8-bit checkpoint on the GPU: whole numbers exactly, others against 64 bits."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES, Guarded, Kept, activations, half_unit, held
from oracle import activations as A

pytestmark = pytest.mark.gpu

# tokens, outputs n, inputs k: one to a few, the ends of a step, of a tile and of a wave's part, many tokens for few outputs
SHAPES = [(1, 1, 1), (2, 3, 5), (31, 8, 8), (33, 16, 32), (63, 127, 31), (64, 128, 256), (65, 129, 257), (100, 255, 33), (128, 256, 96),
          (129, 257, 300), (500, 600, 40), (700, 40, 600), (3000, 17, 65), (5000, 130, 1), (4096, 1, 130), (1024, 520, 264)]


def whole_numbers(rng, T, n, k, dtype):
    """Small whole numbers, so that every sum is exact: dy in -3 .. 3, x in -8 .. 8 times a power of two for each block."""
    dy = rng.integers(-3, 4, (T, n)).astype(np.float32)
    x = rng.integers(-8, 9, (T, k)).astype(np.float32)
    b = A.blocks(k)
    power = 2.0 ** rng.integers(-2, 3, (T, b))
    x = (x * np.repeat(power, 32, 1)[:, :k]).astype(np.float32)
    code, scale = A.store(x)
    assert np.array_equal(A.load(code, scale, k), x)
    return held(dy, dtype), x, code, scale


def run(T, n, k, dtype, out, transposed=False, bias=True, accumulate=False, seed=0, off=0, pad=0, values=whole_numbers):
    rng = np.random.default_rng(seed + 31 * T + 7 * n + k)
    dy, x, code, scale = values(rng, T, n, k, dtype)
    g = Guarded(T, n, dtype, off, pad, dy)
    kept = Kept(T, k, off).fill(code, scale)
    old, old_b = held(rng.integers(-9, 10, (n, k)), out), held(rng.integers(-9, 10, (1, n)), out)
    w = Guarded(k, n, out, off, pad, old.T) if transposed else Guarded(n, k, out, off, pad, old)
    b = Guarded(1, n, out, off + 1, 0, old_b)
    zp.weight_grad(g.t, kept.c, w.t.t() if transposed else w.t, bias=b.t[0] if bias else None, accumulate=accumulate)
    assert w.untouched() and b.untouched() and g.untouched() and kept.untouched()
    (dw, db), (mag, mag_b) = A.weight_grad(dy, A.load(code, scale, k))
    if accumulate:
        dw, db, mag, mag_b = dw + old, db + old_b[0], mag + np.abs(old), mag_b + np.abs(old_b[0])
    got = w.wide().T if transposed else w.wide()
    if not bias:
        assert np.array_equal(b.wide(), old_b)
        db = mag_b = None
    return got, dw, mag, (b.wide()[0] if bias else None), db, mag_b


def rounded(x, dtype):
    return torch.from_numpy(x).to(torch.float32).to(dtype).to(torch.float64).numpy()    # x is a whole number of quarters below 2^22


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", SHAPES)
def test_whole_numbers(dtype, T, n, k):
    t = DTYPES[dtype]
    for i, (out, transposed, bias, accumulate, off, pad) in enumerate((
            (torch.float32, False, True, False, 0, 0), (t, False, True, True, 1, 3), (torch.float32, True, False, True, 3, 0),
            (t, True, True, False, 0, 8), (torch.float32, False, False, False, 8, 8))):
        got, dw, _, got_b, db, _ = run(T, n, k, t, out, transposed, bias, accumulate, i, off, pad)
        assert np.array_equal(got, rounded(dw, out)), (out, transposed, accumulate, off)
        if bias:
            assert np.array_equal(got_b, rounded(db, out))


def test_every_pair_of_types():
    for dtype in DTYPES.values():
        for out in DTYPES.values():
            got, dw, _, got_b, db, _ = run(300, 70, 50, dtype, out)
            assert np.array_equal(got, rounded(dw, out)) and np.array_equal(got_b, rounded(db, out))


def layer_values(rng, T, n, k, dtype):
    code, scale = A.store(activations(rng, T, k))
    return held(rng.standard_normal((T, n)).astype(np.float32) * 2.0 ** rng.uniform(-6, 0, (T, 1)), dtype), None, code, scale


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", [(65, 129, 257), (700, 300, 65), (3000, 17, 65)])
def test_against_64_bits(dtype, T, n, k):
    """Products are exact; each of T sums (in any order, and as many parts as dy has) is off by a unit of fp32 of the
    running sum, at most the sum of magnitudes, and then there is the rounding to the type."""
    t = DTYPES[dtype]
    for out in (torch.float32, t):
        got, dw, mag, got_b, db, mag_b = run(T, n, k, t, out, accumulate=True, values=layer_values)
        assert (np.abs(got - dw) <= 3 * (T + 2) * 2.0 ** -23 * mag + half_unit(dw, out) * (1 + 2.0 ** -10)).all()
        assert (np.abs(got_b - db) <= 3 * (T + 2) * 2.0 ** -23 * mag_b + half_unit(db, out) * (1 + 2.0 ** -10)).all()
        # typical rounding is far below that bound: half units at random, sqrt(T) of them, six deviations
        near = 6 * np.sqrt(3 * T) * 2.0 ** -23 * mag + half_unit(dw, out) * (1 + 2.0 ** -10)
        assert (np.abs(got - dw) <= near).mean() > 0.999


def test_parts_of_dy_are_kept():
    """Values whose lowest bits count: 2^10 + 1 in fp16, 2^23 + 1 in fp32, times a power of two."""
    for dtype, big in ((torch.float16, 2.0 ** 10), (torch.float32, 2.0 ** 23)):
        dy = torch.tensor([[big + 1, 1.0], [-big, 2.0 ** -14]], device="cuda").to(dtype)
        c, dw, db = zp.Checkpoint(2, 1), torch.empty(2, 1, device="cuda"), torch.empty(2, device="cuda")
        c.store(torch.full((2, 1), 0.5, device="cuda"))
        zp.weight_grad(dy, c, dw, bias=db)
        assert dw.view(-1).tolist() == [0.5, 0.5 + 2.0 ** -15] and db.tolist() == [1.0, 1 + 2.0 ** -14]


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_tokens_no_inputs_no_outputs(dtype):
    t = DTYPES[dtype]
    for accumulate in (False, True):
        dw, db = torch.ones(5, 7, device="cuda"), torch.ones(5, device="cuda")
        zp.weight_grad(torch.empty(0, 5, dtype=t, device="cuda"), zp.Checkpoint(0, 7), dw, bias=db, accumulate=accumulate)
        assert bool((dw == (1 if accumulate else 0)).all()) and bool((db == (1 if accumulate else 0)).all())
    dy = torch.ones(9, 5, dtype=t, device="cuda")
    zp.weight_grad(dy, zp.Checkpoint(9, 0), torch.empty(5, 0, device="cuda"), bias=db)          # inputs of none: the bias all the same
    assert db.tolist() == [9.0] * 5
    c = zp.Checkpoint(9, 7)
    c.store(torch.ones(9, 7, device="cuda"))
    zp.weight_grad(dy[:, :0], c, torch.empty(0, 7, device="cuda"))


def test_broadcast_gradient():
    """The gradient of a sum arrives as one value, or one row, for all tokens."""
    x = torch.randint(-4, 5, (300, 40), device="cuda").float()
    c, dw = zp.Checkpoint(300, 40), torch.empty(70, 40, device="cuda")
    c.store(x)
    row = torch.randint(-2, 3, (1, 70), device="cuda").bfloat16()
    zp.weight_grad(row.expand(300, 70), c, dw)
    assert torch.equal(dw, row.float().t() * x.sum(0)[None])
    with pytest.raises(ValueError, match="neighbours"):
        zp.weight_grad(torch.ones(1, 1, device="cuda").expand(300, 70), c, dw)


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan_stay_in_their_columns(dtype):
    t = DTYPES[dtype]
    x = torch.randint(-4, 5, (200, 300), device="cuda").float()
    dy = torch.randint(-2, 3, (200, 150), device="cuda").to(t)
    c, dw, db, clean, clean_b = zp.Checkpoint(200, 300), *(torch.empty(s, device="cuda") for s in ((150, 300), (150,)) * 2)
    c.store(x)
    zp.weight_grad(dy, c, clean, bias=clean_b)
    dy[7, 20], dy[199, 149] = float("inf"), float("nan")
    zp.weight_grad(dy, c, dw, bias=db)
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[[20, 149]] = True
    assert torch.equal(dw[~bad], clean[~bad]) and torch.equal(db[~bad], clean_b[~bad])
    assert not bool(dw[149].isfinite().any()) and not bool(db[bad].isfinite().any())
    assert not bool(dw[20][x[7] != 0].isfinite().any())


def test_equal_inputs_give_equal_bits_at_any_alignment():
    g = torch.Generator(device="cuda").manual_seed(0)
    for T, n, k in ((3000, 136, 72), (500, 300, 260)):
        for t in DTYPES.values():
            dy = torch.randn(T, n, device="cuda", generator=g).to(t)
            c = zp.Checkpoint(T, k)
            c.store(torch.randn(T, k, device="cuda", generator=g))
            want, want_b = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
            zp.weight_grad(dy, c, want, bias=want_b)
            for off, pad in ((1, 0), (0, 1), (8, 8), (3, 5)):
                other, w, b = Guarded(T, n, t, off, pad, dy), Guarded(k, n, torch.float32, off, pad), torch.empty(n, device="cuda")
                zp.weight_grad(other.t, c, w.t.t(), bias=b)
                assert torch.equal(w.t.t(), want) and torch.equal(b, want_b)


def test_refusals_of_the_binding():
    c, dy = zp.Checkpoint(10, 8), torch.zeros(10, 6, device="cuda")
    for kw in (dict(dw=torch.zeros(6, 9, device="cuda")), dict(dw=torch.zeros(8, 6, device="cuda")), dict(dw=torch.zeros(48, device="cuda")),
               dict(dw=torch.zeros(6, 16, device="cuda")[:, ::2]), dict(dw=torch.zeros(6, 8)), dict(bias=torch.zeros(5, device="cuda")),
               dict(bias=torch.zeros(6, device="cuda").half()), dict(bias=torch.zeros(12, device="cuda")[::2])):
        with pytest.raises(ValueError):
            zp.weight_grad(dy, c, **{"dw": torch.zeros(6, 8, device="cuda"), **kw})
    with pytest.raises(zp.ZeroError, match="INVALID_ARG"):
        zp.weight_grad(dy[:9], c, torch.zeros(6, 8, device="cuda"))
