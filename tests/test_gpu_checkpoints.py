"""Activation checkpoints on the GPU: codes and scales bit for bit, activations and their gradients against 64 bits."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES, Guarded, Kept, activations, half_unit, held
from oracle import activations as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 31), (4, 32), (3, 33), (70, 100), (9, 257), (1, 5000), (600, 64), (33, 2047)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store_and_load(dtype, rows, cols):
    rng = np.random.default_rng(rows * 10007 + cols)
    kind = DTYPES[dtype]
    for off, pad in ((0, 0), (1, 3), (5, 0), (0, 8)):
        x = held(activations(rng, rows, cols), kind)
        src, kept = Guarded(rows, cols, kind, off, pad, x), Kept(rows, cols, scale_off=off)
        kept.c.store(src.t)
        code, scale = A.store(x)
        got = kept.host()
        assert np.array_equal(got[1], scale) and np.array_equal(got[0], code)
        assert kept.untouched()
        for other in DTYPES.values():
            out = Guarded(rows, cols, other, pad, off)
            kept.c.load(out.t)
            want = torch.from_numpy(A.load(code, scale, cols)).to(torch.float32).to(other)      # exact in fp32
            assert torch.equal(out.t.cpu(), want) and out.untouched()


@pytest.mark.parametrize("dtype", DTYPES)
def test_numbers_at_the_ends_of_the_range(dtype):
    """Infinities and NaN, the largest and least numbers, subnormals, halves between codes."""
    kind = DTYPES[dtype]
    f = torch.finfo(kind)
    x = np.zeros((12, 70), np.float32)
    x[0, 3], x[1, 40], x[2, 69], x[3, 0], x[3, 69] = np.inf, -np.inf, np.nan, np.nan, np.inf
    x[4], x[5, :33] = f.max, -f.max
    x[6], x[7, 1] = f.smallest_normal * f.eps, -f.smallest_normal * f.eps
    x[8] = f.smallest_normal
    x[9] = np.arange(70) / 16.0 + 1                      # on the ties of e4m3 and between
    x[10, :64] = np.ldexp(448.0, -6)
    x[10, 5] = np.ldexp(450.0, -6)
    x[11] = -0.0
    x = held(x, kind)
    kept = Kept(12, 70)
    kept.c.store(torch.from_numpy(x).to(kind).cuda())
    code, scale = A.store(x)
    got = kept.host()
    assert np.array_equal(got[1], scale) and np.array_equal(got[0], code)
    want = A.load(code, scale, 70)
    for other in DTYPES.values():
        out = torch.empty(12, 70, dtype=other, device="cuda")
        kept.c.load(out)
        back = torch.from_numpy(want).to(torch.float32).to(other)
        assert torch.equal(out.isnan().cpu(), back.isnan())
        assert torch.equal(out.nan_to_num(0, 1, 2).cpu(), back.nan_to_num(0, 1, 2))
    # a NaN reaches what is made from it
    dy, dx, dw = torch.ones(12, 70, device="cuda"), torch.empty(12, 70, device="cuda"), torch.empty(70, 70, device="cuda")
    for k in A.KINDS:
        zp.activation_grad(k, dy, kept.c, dx)
        assert torch.equal(dx.isnan().cpu(), torch.from_numpy(np.isnan(want)))
    zp.weight_grad(dy, kept.c, dw)
    assert torch.equal(dw.isnan().cpu(), torch.from_numpy(np.isnan(want).any(0))[None].expand(70, 70))


def test_broadcast_rows_and_more_dimensions():
    x = torch.randn(1, 100, device="cuda").expand(50, 100)
    c, d = zp.Checkpoint(50, 100), zp.Checkpoint(50, 100)
    c.store(x)
    d.store(x.contiguous())
    assert torch.equal(c.code, d.code) and torch.equal(c.scale, d.scale)
    y = torch.randn(5, 10, 100, device="cuda")
    c.store(y)
    d.store(y.view(50, 100))
    assert torch.equal(c.code, d.code)
    out = torch.empty(5, 10, 100, device="cuda")
    c.load(out)
    assert torch.equal(zp_load(d), out.view(50, 100))
    part = zp.Checkpoint(code=c.code[20:30], scale=c.scale[20:30], cols=100)      # rows of a checkpoint
    assert torch.equal(zp_load(part), out.view(50, 100)[20:30])
    for bad in (torch.randn(50, 200, device="cuda")[:, ::2], torch.randn(100, 50, device="cuda").t(), y.transpose(0, 1),
                torch.randn(50, 101, device="cuda"), torch.randn(50, 100, device="cuda", dtype=torch.float64)):
        with pytest.raises((ValueError, zp.ZeroError)):
            c.store(bad)


def zp_load(c):
    out = torch.empty(c.rows, c.cols, device="cuda")
    c.load(out)
    return out


def test_empty_matrices():
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        x, c = torch.empty(rows, cols, device="cuda"), zp.Checkpoint(rows, cols)
        c.store(x)
        c.load(x)
        zp.activation("gelu", x, torch.empty_like(x), c)
        zp.activation_grad("gelu", x, c, torch.empty_like(x))


def value_bound(kind, z, h, dtype):
    """What rounding may do to act(z) = h: the argument of the exponential (or z^2 / 2 for the normal distribution) is
    off by 4 half-units of its own, which the exponential turns into as much of its value; 8 more roundings of the value
    (products, sum, reciprocal and exponential, an ulp each); what underflows; one rounding to the type."""
    with np.errstate(invalid="ignore"):
        off = np.abs(h) * U * (16 + 4 * np.minimum(np.abs(A.angle(kind, z)), 100)) + np.abs(z) * 2.0 ** -125
        return half_unit(h, dtype) * (1 + 2.0 ** -10) + off


@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_activation(kind, dtype, gated):
    rng = np.random.default_rng(len(kind) + 7 * gated)
    t = DTYPES[dtype]
    for rows, cols, off, pad in ((1, 1, 0, 0), (5, 64, 0, 0), (37, 101, 1, 4), (3, 1500, 3, 0), (200, 40, 0, 1)):
        z = held(activations(rng, rows, cols), t)
        z[0, 0] = -25.0
        up = held(activations(rng, rows, cols), t) if gated else None
        x, out = Guarded(rows, cols, t, off, pad, z), Guarded(rows, cols, t, pad, off)
        u = Guarded(rows, cols, t, off + 1, pad, up) if gated else None
        cx, cu, ch = Kept(rows, cols, 1), Kept(rows, cols, 2), Kept(rows, cols, 3)
        zp.activation(kind, x.t, out.t, cx.c, up=u.t if gated else None, up_checkpoint=cu.c if gated else None, out_checkpoint=ch.c)
        h = A.act(kind, z.astype(np.float64))[0]
        bound = value_bound(kind, z.astype(np.float64), h, t)
        if gated:
            h, bound = h * up, bound * np.abs(up) + half_unit(h * up, t) * (1 + 2.0 ** -10) + np.abs(h * up) * U
        with np.errstate(over="ignore"):
            clear = np.abs(h) < torch.finfo(t).max * 0.99
        assert (np.abs(out.wide() - h) <= bound)[clear].all(), (kind, rows, cols)
        assert out.untouched() and x.untouched()
        for kept, values in ((cx, z), (cu, up), (ch, out.t.to(torch.float32).cpu().numpy())):
            if values is None:
                continue
            code, scale = A.store(values)
            got = kept.host()
            assert np.array_equal(got[0], code) and np.array_equal(got[1], scale) and kept.untouched()
        # in place, with nothing kept: the same bits
        first = out.t.clone()
        zp.activation(kind, x.t, x.t, up=u.t if gated else None)
        assert torch.equal(x.t, first) and x.untouched()
        if gated:
            x2 = Guarded(rows, cols, t, off, pad, z)
            zp.activation(kind, x2.t, u.t, up=u.t)
            assert torch.equal(u.t, first) and u.untouched()


@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_activation_grad(kind, dtype, gated):
    rng = np.random.default_rng(100 + len(kind) + 7 * gated)
    t = DTYPES[dtype]
    for rows, cols, off, pad in ((1, 1, 0, 0), (5, 64, 0, 0), (37, 101, 1, 4), (3, 1500, 3, 0), (200, 40, 0, 1)):
        cx, cu = Kept(rows, cols, 1).fill(*A.store(activations(rng, rows, cols))), Kept(rows, cols, 2).fill(*A.store(activations(rng, rows, cols)))
        z, up = A.load(*cx.host(), cols), A.load(*cu.host(), cols) if gated else 1.0
        g = held(rng.standard_normal((rows, cols)).astype(np.float32), t)
        dy, dx, du = Guarded(rows, cols, t, off, pad, g), Guarded(rows, cols, t, pad, off), Guarded(rows, cols, t, 1, 1)
        kw = dict(up_checkpoint=cu.c, dup=du.t) if gated else {}
        zp.activation_grad(kind, dy.t, cx.c, dx.t, **kw)
        a, d, mag = A.act(kind, z)
        # as for the value, of the derivative's two terms; the slope in the second has 4 roundings of its own
        arg = np.minimum(np.abs(A.angle(kind, z)), 100)
        off_d = np.abs(g * up) * (mag * U * (24 + 8 * arg) + (1 + np.abs(z)) * 2.0 ** -118)
        want = g * up * d
        assert (np.abs(dx.wide() - want) <= half_unit(want, t) * (1 + 2.0 ** -10) + off_d).all(), (kind, rows, cols)
        assert dx.untouched() and dy.untouched()
        if gated:
            want = g * a
            bound = np.abs(g) * value_bound(kind, z, a, torch.float32) + half_unit(want, t) * (1 + 2.0 ** -10)
            assert (np.abs(du.wide() - want) <= bound).all() and du.untouched()
        # in place: dx, or dup, where dy is
        first, second = dx.t.clone(), du.t.clone()
        other = Guarded(rows, cols, t, off, pad, g)
        zp.activation_grad(kind, dy.t, cx.c, dy.t, **kw)
        assert torch.equal(dy.t, first) and dy.untouched()
        if gated:
            zp.activation_grad(kind, other.t, cx.c, dx.t, up_checkpoint=cu.c, dup=other.t)
            assert torch.equal(other.t, second) and other.untouched()


@pytest.mark.parametrize("kind", A.KINDS)
def test_values_far_out(kind):
    """Arguments whose exponential, or whose square, leaves fp32's range."""
    z = np.array([[3e38, -3e38, 1e20, -1e20, 500.0, -500.0, 89.0, -89.0, 20.0, -20.0, 13.5, -13.5, 1e-30, -1e-30, 1e-38, 0.0]], np.float32)
    z = np.repeat(z.T, 32, 1)                     # a block each: every value is its block's largest
    x, out, c = torch.from_numpy(z).cuda(), torch.empty(16, 32, device="cuda"), zp.Checkpoint(16, 32)
    zp.activation(kind, x, out, c)
    h = A.act(kind, z.astype(np.float64))[0]
    h = np.where(np.isnan(h), 0.0, h)             # inf * 0 in 64 bits too: z^3 there
    assert (np.abs(out.cpu().numpy() - h) <= value_bound(kind, z.astype(np.float64), h, torch.float32) + np.abs(h) * 2.0 ** -16).all()
    zr = zp_load(c).cpu().numpy().astype(np.float64)
    dx = torch.empty(16, 32, device="cuda")
    zp.activation_grad(kind, torch.ones(16, 32, device="cuda"), c, dx)
    got = dx.cpu().numpy()
    assert np.isfinite(got).all()
    assert (got[zr > 20] == 1).all() and (np.abs(got[zr < -20]) <= 1e-6).all()
    assert np.abs(got[-4:-1] - A.act(kind, zr[-4:-1])[1]).max() <= 4 * U


def test_halves_of_one_buffer():
    rows, cols = 50, 96
    both = torch.randn(rows, 2 * cols, device="cuda").half()
    g, u = both[:, :cols], both[:, cols:]
    cg, cu, out = zp.Checkpoint(rows, cols), zp.Checkpoint(rows, cols), torch.empty(rows, cols, device="cuda").half()
    zp.activation("silu", g, out, cg, up=u, up_checkpoint=cu)
    want = torch.empty_like(out)
    zp.activation("silu", g.contiguous(), want, up=u.contiguous())
    assert torch.equal(out, want)
    dy = torch.randn(rows, cols, device="cuda").half()
    grads = torch.empty(rows, 2 * cols, device="cuda").half()
    zp.activation_grad("silu", dy, cg, grads[:, :cols], up_checkpoint=cu, dup=grads[:, cols:])
    a, b = torch.empty_like(dy), torch.empty_like(dy)
    zp.activation_grad("silu", dy, cg, a, up_checkpoint=cu, dup=b)
    assert torch.equal(grads, torch.cat([a, b], 1))
    zp.activation("silu", g, g, up=u)
    assert torch.equal(g, want)
    with pytest.raises(zp.ZeroError, match="overlaps"):
        zp.activation("silu", g, both[:, 1:cols + 1], up=u)


def test_more_than_2_31_elements():
    rows, cols = 65543, 32771                    # 2.148e9 values, rows that end inside a block and off their lines
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    c = zp.Checkpoint(rows, cols)
    c.store(x)
    part, wide = zp.Checkpoint(64, cols), torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    c.load(wide)
    for r in (0, 30000, 65535 - 60, rows - 64):
        part.store(x[r:r + 64].clone())
        assert torch.equal(part.code, c.code[r:r + 64]) and torch.equal(part.scale, c.scale[r:r + 64])
    for r in range(0, rows, 8192):               # half a step of an e4m3: 2^-4 of the value, or 2^-10 of a scale whose block's largest is above 224
        a, b = x[r:r + 8192].float(), wide[r:r + 8192].float()
        top = torch.nn.functional.pad(a, (0, 29)).abs().view(a.shape[0], -1, 32).amax(2).repeat_interleave(32, 1)[:, :cols]
        assert bool(((a - b).abs() <= torch.maximum(a.abs() / 16, top * 2.0 ** -10 / 224)).all())
