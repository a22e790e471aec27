"""CPU checks of the calls on activation checkpoints and embeddings: the numpy oracle against torch and against
differences, and every refusal that is decided before a device is touched."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import activations as A


@pytest.fixture(scope="module")
def zp():
    from sharded_zero_partition_amd import build as zbuild
    if not os.path.exists(zbuild.LIB):
        zbuild.build()
    import sharded_zero_partition_amd as z
    return z


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

TORCH = {"relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


@pytest.mark.parametrize("kind", A.KINDS)
def test_activations_match_torch_and_differences(kind):
    z = np.concatenate([np.linspace(-9, 9, 1801), [1e-30, -1e-30, 30.0, -30.0]])
    t = torch.from_numpy(z).requires_grad_()
    y = TORCH[kind](t)
    y.sum().backward()
    a, d, mag = A.act(kind, z)
    # both in 64 bits: some roundings, and what the exponential's argument makes of its own
    off = (mag + np.abs(a)) * 2.0 ** -53 * (16 + 8 * np.abs(A.angle(kind, z)))
    # torch's own value forms 1 + erf or 1 + tanh: near -1 that is off by 2^-53, erf's or tanh's own unit 2^-53 more, times z / 2
    assert (np.abs(a - y.detach().numpy()) <= off + np.abs(z) * 2.0 ** -52).all()
    # ... and its derivative of gelu_tanh 1 - tanh^2, which is off by 2^-52 of its own accord, times z / 2 times the slope
    assert (np.abs(d - t.grad.numpy()) <= off + 2.0 ** -52 * (1 + np.abs(z) * (1 + 3 * 0.044715 * z * z))).all()
    smooth = np.abs(z) > 1e-3 if kind == "relu" else np.abs(z) < 9
    h = 1e-5
    diff = (A.act(kind, z + h)[0] - A.act(kind, z - h)[0]) / (2 * h)
    # the third derivative is below 3 for each of them: h^2 / 6 of it, and 2^-53 z / h
    assert (np.abs(diff - d) <= h * h / 2 + 2.0 ** -52 * (1 + np.abs(z)) / h)[smooth].all()


def test_store_matches_torch_and_reads_back():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 101)) * 10.0 ** rng.uniform(-6, 6, (40, 1))).astype(np.float32)
    x[3] = 0
    code, scale = A.store(x)
    assert code.shape == (40, 128) and scale.shape == (40, 4) and (code[:, 101:] == 0).all()
    power = np.repeat(2.0 ** (127.0 - scale), 32, axis=1)[:, :101]
    want = torch.from_numpy((x * power).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(code[:, :101], want)
    top = np.abs(np.pad(x, ((0, 0), (0, 27))).reshape(40, 4, 32)).max(2)
    assert (top * 2.0 ** (127.0 - scale) <= 448).all() and ((scale == 1) | (top * 2.0 ** (128.0 - scale) > 448)).all()
    back = A.load(code, scale, 101)
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 / power)).all()
    again = A.store(back.astype(np.float32))
    assert np.array_equal(A.load(*again, 101), back)       # the values (a largest one that went down to 224 takes a lower scale)


def test_a_block_that_is_not_finite_is_nan():
    x = np.ones((2, 70), np.float32)
    x[0, 5], x[1, 69] = np.inf, np.nan
    code, scale = A.store(x)
    assert (scale == [[255, 119, 119], [119, 119, 255]]).all()
    back = A.load(code, scale, 70)
    assert np.isnan(back[0, :32]).all() and np.isnan(back[1, 64:]).all() and (code[:, 70:] == 0).all()
    assert (back[0, 32:] == 1).all() and (back[1, :64] == 1).all()


def test_embedding_gradient_is_the_lookup_s():
    rng = np.random.default_rng(1)
    table = torch.from_numpy(rng.standard_normal((7, 5))).requires_grad_()
    tokens = np.array([3, 9, 3, 12, 3, -1, 4])
    dy = rng.standard_normal((7, 5))
    y = A.lookup(table.detach().numpy(), tokens, 3, 2.0)
    t = torch.from_numpy(tokens) - 3
    ok = (t >= 0) & (t < 7)
    out = torch.where(ok[:, None], table[t.clamp(0, 6)] * 2.0, 0.0)
    (out * torch.from_numpy(dy)).sum().backward()
    assert np.array_equal(y, out.detach().numpy())
    got, mag, count = A.embedding_grad(dy, tokens, 7, 3, 2.0)
    assert np.allclose(got, table.grad.numpy(), rtol=1e-14, atol=0) and list(count) == [3, 1, 0, 0, 0, 0, 1]
    assert (mag >= np.abs(got) - 1e-15).all()


# ---------------------------------------------------------------------------
# refusals, before any device is touched
# ---------------------------------------------------------------------------

BASE = 1 << 40      # addresses that are only compared
GAP = 1 << 30
INV, ALI, OVF, HIP = -1, -2, -4, -5
FP16, BF16, FP32 = 1, 2, 3


class Call:
    """Sound arguments of a call, of which a test changes some."""

    def __init__(self, zp):
        self.zp, self.B = zp, zp.binding

    def matrix(self, at, rows=8, cols=64, stride=None, type=BF16, data=None):
        return self.B.MatrixC(BASE + at * GAP if data is None else data, rows, cols, cols if stride is None else stride, type, 0)

    def kept(self, at, rows=8, cols=64, code=None, scale=None):
        return self.B.CheckpointC(BASE + at * GAP if code is None else code, BASE + at * GAP + GAP // 2 if scale is None else scale, rows, cols)

    def ref(self, x):
        return None if x is None else ctypes.byref(x)

    def store(self, x=None, c=None):
        return self.zp.lib.zero_checkpoint_store(self.ref(x or self.matrix(0)), self.ref(c or self.kept(1)), None)

    def load(self, c=None, out=None):
        return self.zp.lib.zero_checkpoint_load(self.ref(c or self.kept(1)), self.ref(out or self.matrix(0)), None)

    def activation(self, kind=1, x=None, up=None, out=None, cx=None, cup=None, cout=None):
        return self.zp.lib.zero_activation(kind, self.ref(x or self.matrix(0)), self.ref(up), self.ref(out or self.matrix(2)),
                                           self.ref(cx), self.ref(cup), self.ref(cout), None)

    def grad(self, kind=1, dy=None, cx=None, cup=None, dx=None, dup=None):
        return self.zp.lib.zero_activation_grad(kind, self.ref(dy or self.matrix(0)), self.ref(cx or self.kept(1)), self.ref(cup),
                                                self.ref(dx or self.matrix(2)), self.ref(dup), None)

    def weight(self, dy=None, x=None, dw=None, transposed=0, bias=None, accumulate=0, work=None):
        return self.zp.lib.zero_weight_grad(self.ref(dy or self.matrix(0, 8, 64)), self.ref(x or self.kept(1, 8, 96)),
                                            self.ref(dw or self.matrix(2, 64, 96, type=FP32)), transposed, bias, accumulate, work, None)

    def lookup(self, table=None, tokens=BASE + 5 * GAP, size=8, first=0, scale=1.0, out=None):
        return self.zp.lib.zero_embedding_lookup(self.ref(table or self.matrix(0, 100, 64)), tokens, size, first, scale,
                                                 self.ref(out or self.matrix(2)), None)

    def egrad(self, dy=None, tokens=BASE + 5 * GAP, size=8, first=0, scale=1.0, dt=None, accumulate=0, work=BASE + 6 * GAP):
        return self.zp.lib.zero_embedding_grad(self.ref(dy or self.matrix(0)), tokens, size, first, scale,
                                               self.ref(dt or self.matrix(2, 100, 64)), accumulate, work, None)


@pytest.fixture
def call(zp):
    return Call(zp)


def sound(rc):
    """Passed every check that needs no device."""
    assert rc == (0 if torch.cuda.is_available() else HIP)


@pytest.fixture
def cpu_only():
    if torch.cuda.is_available():
        pytest.skip("addresses that only a CPU run may pass")


def test_matrices_are_checked(call):
    m, lib = call.matrix, call.zp.lib
    assert lib.zero_checkpoint_store(None, call.ref(call.kept(1)), None) == INV
    for bad, rc in ((m(0, type=0), INV), (m(0, type=4), INV), (m(0, rows=-1), INV), (m(0, cols=-1), INV), (m(0, data=0), INV),
                    (m(0, stride=-1), INV), (m(0, data=BASE + 1), ALI), (m(0, data=BASE + 2, type=FP32), ALI),
                    (m(0, cols=1 << 31), OVF), (m(0, rows=1 << 40, stride=1 << 40), OVF), (m(0, data=(1 << 64) - 64), OVF)):
        assert call.store(x=bad) == rc
        assert call.activation(x=bad) == rc
        assert call.activation(up=bad) == rc
        assert call.activation(out=bad) == rc
        assert call.grad(dy=bad) == rc and call.grad(dx=bad) == rc
        assert call.weight(dy=bad) == rc and call.weight(dw=bad) == rc
        assert call.lookup(table=bad) == rc and call.lookup(out=bad) == rc
        assert call.egrad(dy=bad) == rc and call.egrad(dt=bad) == rc
        assert call.load(out=bad) == rc
    assert call.load(out=m(0, stride=63)) == INV           # rows that are written may not meet
    assert call.activation(out=m(2, stride=0)) == INV
    assert call.weight(dw=m(2, 64, 96, stride=95)) == INV


def test_checkpoints_are_checked(call):
    k, lib = call.kept, call.zp.lib
    assert lib.zero_checkpoint_store(call.ref(call.matrix(0)), None, None) == INV
    for bad, rc in ((k(1, rows=-1), INV), (k(1, cols=-1), INV), (k(1, code=0), INV), (k(1, scale=0), INV), (k(1, code=BASE + 8), ALI),
                    (k(1, cols=1 << 31), OVF), (k(1, rows=1 << 47), OVF), (k(1, code=(1 << 64) - 256), OVF)):
        assert call.store(c=bad) == rc
        assert call.load(c=bad) == rc
        assert call.activation(cx=bad) == rc and call.activation(cout=bad) == rc
        assert call.grad(cx=bad) == rc
        assert call.weight(x=bad) == rc
    for bad in (k(1, rows=7), k(1, cols=65)):
        assert call.store(c=bad) == INV and call.load(c=bad) == INV and call.activation(cx=bad) == INV and call.grad(cx=bad) == INV
    n = (ctypes.c_int64 * 2)()
    assert lib.zero_checkpoint_bytes(7, 65, ctypes.addressof(n), ctypes.addressof(n) + 8) == 0 and list(n) == [7 * 96, 21]
    assert lib.zero_checkpoint_bytes(7, 0, ctypes.addressof(n), None) == 0 and n[0] == 0
    assert lib.zero_checkpoint_bytes(-1, 5, None, None) == INV and lib.zero_checkpoint_bytes(1 << 45, 512, None, None) == OVF


def test_activation_refusals(call):
    m, k = call.matrix, call.kept
    for kind in (-1, 4):
        assert call.activation(kind=kind) == INV and call.grad(kind=kind) == INV
    assert call.activation(cup=k(3)) == INV                                  # without up
    assert call.activation(up=m(4), cx=k(1)) == INV                          # gated keeps both
    assert call.activation(up=m(4), cup=k(1)) == INV
    for bad in (m(4, rows=7), m(4, cols=63), m(4, type=FP16)):
        assert call.activation(up=bad) == INV and call.activation(out=bad) == INV and call.grad(dx=bad) == INV
        assert call.grad(cup=k(3), dup=bad) == INV
    assert call.grad(cup=k(3)) == INV and call.grad(dup=m(4)) == INV
    # overlaps: shifted by an element, another stride, a checkpoint in a matrix, a checkpoint twice
    x = m(0)
    assert call.activation(out=m(0, data=BASE + 2)) == INV
    assert call.activation(out=m(0, stride=65)) == INV
    assert call.activation(x=m(0, stride=128), out=m(0, data=BASE + 64, stride=128)) == INV
    assert call.activation(cx=k(0)) == INV and call.activation(cx=k(1, scale=BASE)) == INV
    assert call.activation(cx=k(1), cout=k(1)) == INV
    assert call.activation(up=m(4), cx=k(1), cup=k(1)) == INV
    assert call.activation(cx=k(1, scale=BASE + GAP + 8 * 64 - 1)) == INV
    assert call.store(x=m(1)) == INV and call.load(out=m(1)) == INV
    assert call.grad(dx=m(1)) == INV and call.grad(dx=m(0, data=BASE + 2)) == INV
    assert call.grad(cup=k(3), dup=m(2)) == INV and call.grad(cup=k(3), dup=m(3)) == INV


def test_sound_activations_pass(call, cpu_only):
    m, k = call.matrix, call.kept
    sound(call.store())
    sound(call.load())
    sound(call.store(x=m(0, stride=0)))
    sound(call.store(c=k(1, scale=BASE + GAP + 8 * 64)))
    sound(call.activation())
    sound(call.activation(out=m(0)))                                          # in place
    sound(call.activation(up=m(4), out=m(4), cx=k(1), cup=k(3), cout=k(5)))
    # halves of one buffer
    left, right = m(0, stride=128), m(0, data=BASE + 128, stride=128)
    sound(call.activation(x=left, up=right, cx=k(1), cup=k(3)))
    sound(call.activation(x=left, up=right, out=left))
    sound(call.activation(x=right, up=left, out=right))
    sound(call.grad(dx=m(0)))
    sound(call.grad(dx=left, dup=right, dy=m(2), cup=k(3)))
    sound(call.grad(dx=m(2), dup=m(0), cup=k(3)))
    sound(call.grad(dy=m(0, rows=0, data=0), cx=k(1, rows=0, code=0), dx=m(2, rows=0, data=0)))


def test_weight_grad_refusals(call):
    m, k, lib = call.matrix, call.kept, call.zp.lib
    for kw in (dict(transposed=2), dict(accumulate=-1), dict(x=k(1, 7, 96)), dict(dw=m(2, 96, 64, type=FP32)), dict(dw=m(2, 64, 97)),
               dict(dw=m(2, 64, 96), transposed=1)):
        assert call.weight(**kw) == INV, kw
    assert call.weight(bias=BASE + 3 * GAP + 2) == ALI                          # dw is fp32
    assert call.weight(bias=(1 << 64) - 4) == OVF
    for at in (BASE, BASE + GAP, BASE + GAP + GAP // 2, BASE + 2 * GAP):       # bias in dy, codes, scales, dw
        assert call.weight(bias=at) == INV
    assert call.weight(dw=m(0, 64, 96, type=FP32)) == INV and call.weight(dw=m(1, 64, 96, type=FP32)) == INV
    # a workspace where the tokens are split
    T = 4096
    big = dict(dy=m(0, T, 64), x=k(1, T, 96))
    need = lib.zero_weight_grad_work_bytes(T, 64, 96, BF16)
    assert need > 0
    assert call.weight(**big) == INV
    assert call.weight(**big, work=BASE + 6 * GAP + 8) == ALI
    assert call.weight(**big, work=BASE + 2 * GAP + 64) == INV and call.weight(**big, work=BASE + T * 128 - 16) == INV
    assert call.weight(**big, work=(1 << 64) - 64) == OVF
    for bad in ((-1, 64, 96, BF16), (T, 0, 96, BF16), (T, 64, -1, BF16), (T, 64, 96, 4), (T, 1 << 31, 96, BF16)):
        assert lib.zero_weight_grad_work_bytes(*bad) == 0


def test_sound_weight_grads_pass(call, cpu_only):
    m, k, lib = call.matrix, call.kept, call.zp.lib
    sound(call.weight())
    sound(call.weight(dw=m(2, 96, 64), transposed=1, bias=BASE + 3 * GAP + 2, accumulate=1))
    sound(call.weight(dy=m(0, 0, 64, data=0), x=k(1, 0, 96, code=0)))
    sound(call.weight(x=k(1, 8, 0, code=0), dw=m(2, 64, 0, data=0)))
    sound(call.weight(dy=m(0, stride=0)))
    T = 4096
    sound(call.weight(dy=m(0, T, 64), x=k(1, T, 96), work=BASE + 6 * GAP))


def test_embedding_refusals(call):
    m, lib = call.matrix, call.zp.lib
    nan, inf = float("nan"), float("inf")
    for f in (call.lookup, call.egrad):
        assert f(tokens=None) == INV and f(size=2) == INV and f(tokens=BASE + 5 * GAP + 4) == ALI
        assert f(scale=nan) == INV and f(scale=inf) == INV
        assert f(tokens=(1 << 64) - 8) == OVF
    assert call.lookup(out=m(2, cols=63)) == INV and call.egrad(dt=m(2, 100, 63)) == INV
    assert call.lookup(out=m(0)) == INV and call.lookup(tokens=BASE + 2 * GAP) == INV
    assert call.egrad(accumulate=2) == INV and call.egrad(work=None) == INV and call.egrad(work=BASE + 6 * GAP + 4) == ALI
    assert call.egrad(dt=m(0, 100, 64)) == INV and call.egrad(tokens=BASE + 2 * GAP) == INV
    assert call.egrad(work=BASE) == INV and call.egrad(work=BASE + 2 * GAP) == INV and call.egrad(work=BASE + 5 * GAP) == INV
    assert call.egrad(dy=m(0, rows=(1 << 30) + 1)) == OVF and call.egrad(dt=m(2, (1 << 30) + 1, 64)) == OVF
    for bad in ((0, 10, 10), (10, 0, 10), (10, 10, 0), ((1 << 30) + 1, 10, 10), (10, (1 << 30) + 1, 10), (10, 10, 1 << 31), (-5, 1, 1)):
        assert lib.zero_embedding_grad_work_bytes(*bad) == 0
    assert lib.zero_embedding_grad_work_bytes(100, 10, 10) % 16 == 0


def test_sound_embeddings_pass(call, cpu_only):
    m = call.matrix
    sound(call.lookup())
    sound(call.lookup(size=4, first=-(1 << 62), scale=0.0, tokens=BASE + 5 * GAP + 4))
    sound(call.lookup(table=m(0, 0, 64, data=0)))
    sound(call.lookup(out=m(2, rows=0, data=0), tokens=None))
    sound(call.egrad())
    sound(call.egrad(dy=m(0, rows=0, data=0), tokens=None, work=None))
    sound(call.egrad(dt=m(2, 0, 64, data=0), work=None))


def test_binding_refuses_what_does_not_fit(zp):
    """Tensors that live elsewhere, or of a shape or type that no call takes; nothing here reaches the library."""
    t = torch.zeros(4, 32)
    bad = (ValueError, RuntimeError, AssertionError)
    for kw in (dict(), dict(rows=4), dict(rows=4, cols=-1), dict(code=t, cols=32), dict(rows=4, cols=32, code=t.byte(), scale=t[:, :1].byte()),
               dict(code=t.byte(), scale=t[:, :1].byte(), cols=32)):
        with pytest.raises(bad):
            zp.Checkpoint(**kw)
    for f in (lambda: zp.activation("silu", t, t), lambda: zp.activation("tanh", t, t), lambda: zp.embedding_lookup(t, t, t),
              lambda: zp.embedding_grad(t, t, t), lambda: zp.weight_grad(t, None, t), lambda: zp.activation_grad("relu", t, None, t)):
        with pytest.raises(bad + (AttributeError,)):
            f()
