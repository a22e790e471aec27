"""CPU checks of the tensor sets: the numpy oracle against torch.optim.AdamW, torch's float8 casts and its own 64-bit
form; and every refusal of the C ABI that is decided before a device is touched."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import tensor_set as T


@pytest.fixture(scope="module")
def zp():
    import os
    from sharded_zero_partition_amd import build as zbuild
    if not os.path.exists(zbuild.LIB):
        zbuild.build()
    import sharded_zero_partition_amd as z
    return z


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(T.E4M3, want, equal_nan=True)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 2.0 ** rng.uniform(-12, 7, 20000),
                        (T.E4M3[:126] + T.E4M3[1:127]) / 2, [0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -11]])
    y = np.clip(y, -448, 448).astype(np.float32)
    assert np.array_equal(T.e4m3_nearest(y), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_is_the_least_that_fits():
    rng = np.random.default_rng(1)
    top = np.concatenate([2.0 ** rng.uniform(-149, 127.9, 5000), 448 * 2.0 ** np.arange(-120, 110),
                          np.nextafter((448 * 2.0 ** np.arange(-110.0, 110)).astype(np.float32), np.float32(np.inf))]).astype(np.float32)
    s = T.scale_bytes(top)
    assert (top.astype(np.float64) * 2.0 ** (127.0 - s) <= 448).all()
    assert ((s == 1) | (top.astype(np.float64) * 2.0 ** (128.0 - s) > 448)).all()
    assert (s >= 1).all() and (s <= 247).all() and T.scale_bytes(np.zeros(1))[0] == 1


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1000])
def test_nearest_encoding_error_and_round_trip(n):
    rng = np.random.default_rng(n)
    x = (rng.standard_normal(n) * 10.0 ** rng.uniform(-6, 3, n)).astype(np.float32)
    code, s = T.encode(x, False)
    y = T.decode(code, s)
    scale = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32)[:n]
    # half a step: 2^-4 relative, or half of 2^-9 of the scale
    assert (np.abs(y.astype(np.float64) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)).all()
    again = T.decode(*T.encode(y, False))
    assert np.array_equal(again, y)
    v = np.square(x)
    vc, vs = T.encode(v, True)
    assert ((T.decode(vc, vs) > 0) == (v > 0)).all()


def test_random_rounding_keeps_the_mean():
    """Each value goes to one of its two neighbours, and the mean over N steps is within 6 standard deviations of it:
    a step's deviation is at most half the gap, so 6 * gap / 2 / sqrt(N); the 16-bit chances add gap * 2^-17."""
    x = np.concatenate([[1.0], np.linspace(1e-6, 1.0, 31)]).astype(np.float32)
    N = 4000
    s = T.encode(x, True)[1]
    assert s.size == 1
    got = np.array([T.decode(*T.encode(x, True, T.chances(32, 7, 3, t))) for t in range(N)], np.float64)
    power = 2.0 ** (float(s[0]) - 127)
    grid = T.E4M3[:127] * power
    hi = np.searchsorted(grid, x.astype(np.float64), side="left")
    lo = np.where(grid[hi] == x, hi, hi - 1)
    lo = np.where(lo == 0, 1, lo)                       # never to zero
    gap = np.maximum(grid[hi] - grid[lo], 0)
    for k in range(32):
        assert set(np.unique(got[:, k])) <= {grid[lo[k]], grid[hi[k]]}
    inside = x >= grid[1]
    off = np.abs(got.mean(0) - x)
    assert (off <= 6 * gap / 2 / np.sqrt(N) + gap * 2.0 ** -17 + 1e-9)[inside].all()


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_oracle_matches_torch_adamw(wd):
    rng = np.random.default_rng(3)
    n, h = 257, T.HParams(lr=1e-2, weight_decay=wd)
    p = rng.standard_normal(n).astype(np.float32)
    tp = torch.nn.Parameter(torch.from_numpy(p.astype(np.float64)))
    opt = torch.optim.AdamW([tp], lr=h.lr, betas=(h.beta1, h.beta2), eps=h.eps, weight_decay=wd and h.weight_decay)
    m, v, c = np.zeros(n, np.float32), np.zeros(n, np.float32), T.Control()
    for _ in range(5):
        g = rng.standard_normal(n).astype(np.float32)
        tp.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        assert c.begin([h], check=False)
        before = p, m, v
        (wide, off) = T.adamw_wide(h, 1.0, c.t, g, 1.0, *before)
        p, m, v = T.adamw(c.consts[0], g, 1.0, *before)
        for a, b, o in zip((p, m, v), wide, off):
            assert (np.abs(a.astype(np.float64) - b) <= o).all()
    # five steps, each off by p_off at most (about 1e-7 of p and of the update), in a form that decays p first:
    # p (1 - lr wd) - update, the same number
    assert np.abs(p - tp.detach().numpy()).max() < 5 * 4 * T.U * (np.abs(p).max() + 5 * h.lr * 20)


def test_begin_matches_the_shard_step_scaler():
    o, c = oracle.LossScaler(1024.0), T.Control(scale=1024.0)
    class Rule:
        backoff, growth, min_scale, growth_interval = 0.5, 2.0, 1.0, 3
    o.growth_interval = 3
    rng = np.random.default_rng(9)
    for _ in range(60):
        bad = rng.random() < 0.3
        c.sumsq = np.inf if bad else 4.0
        assert c.begin([T.HParams()], scaler=Rule) == (not bad)
        o.update(bad)
        assert (c.scale, c.good_steps) == (o.scale, o.good_steps)
    assert c.t + c.skipped == 60


# ---------------------------------------------------------------------------
# refusals, before any device is touched
# ---------------------------------------------------------------------------

BASE = 1 << 40      # addresses that are only compared


def _tensor(zp, i=0, numel=64, **kw):
    B = zp.binding
    f = dict(numel=numel, p=BASE + (i << 20), grad=BASE + (i << 20) + (1 << 16), m=BASE + (i << 20) + (2 << 16),
             v=BASE + (i << 20) + (3 << 16), out=BASE + (i << 20) + (4 << 16), group=0)
    f.update(kw)
    return B.TensorC(**f)


def _create(zp, tensors, grad=1, state=3, out=1, n=None, null_out=False):
    arr = (zp.binding.TensorC * max(1, len(tensors)))(*tensors)
    h = ctypes.c_void_p()
    return zp.lib.zero_tensor_set_create(arr, len(tensors) if n is None else n, grad, state, out, 0, None,
                                         None if null_out else ctypes.byref(h))


def test_create_refusals(zp):
    INV, ALI, OVF, OOM = -1, -2, -4, -6
    ok = _tensor(zp)
    assert _create(zp, [ok], null_out=True) == INV
    assert _create(zp, [ok], n=-1) == INV
    assert zp.lib.zero_tensor_set_create(None, 1, 1, 3, 1, 0, None, ctypes.byref(ctypes.c_void_p())) == INV
    for kw in (dict(grad=4), dict(grad=-1), dict(state=1), dict(state=5), dict(out=3), dict(out=4)):
        assert _create(zp, [ok], **kw) == INV, kw
    for t in (dict(numel=-1), dict(group=-1), dict(group=16), dict(m=None), dict(v=None), dict(out=None),
              dict(m_scale=BASE), dict(p=None)):
        assert _create(zp, [_tensor(zp, **t)]) == INV, t
    assert _create(zp, [ok], out=0) == INV                                   # out without out_type
    assert _create(zp, [ok], grad=0) == INV                                  # gradient without grad_type
    assert _create(zp, [ok], state=0) == INV                                 # states without state_type
    assert _create(zp, [ok], state=4) == INV                                 # 8 bits without scales
    assert _create(zp, [ok, _tensor(zp, 1, grad=None)]) == INV               # some with, some without
    assert _create(zp, [ok, _tensor(zp, 1, p=None)]) == INV
    for t in (dict(p=BASE + 2), dict(m=BASE + (2 << 16) + 1), dict(v=BASE + (3 << 16) + 2), dict(out=BASE + (4 << 16) + 1),
              dict(grad=BASE + (1 << 16) + 1)):
        assert _create(zp, [_tensor(zp, **t)]) == ALI, t
    assert _create(zp, [_tensor(zp, grad=BASE + (1 << 16) + 2)], grad=3) == ALI
    # overlaps: the same tensor twice, states in p, an out's end in the next p, a gradient in m
    assert _create(zp, [ok, ok]) == INV
    assert _create(zp, [_tensor(zp, m=BASE + 252)]) == INV
    assert _create(zp, [ok, _tensor(zp, 1, out=BASE + 254)]) == INV
    assert _create(zp, [_tensor(zp, grad=BASE + (2 << 16) + 254)]) == INV
    # too large for the tables, past the address space
    assert _create(zp, [_tensor(zp, numel=(1 << 35) + 1)]) == OOM
    top = (1 << 64) - 4096
    assert _create(zp, [_tensor(zp, numel=2048, p=top)]) == OVF
    assert _create(zp, [_tensor(zp, numel=4096, grad=top)]) == OVF
    assert zp.lib.zero_tensor_set_destroy(None) == 0


def test_accepted_arguments_reach_the_device_check(zp):
    """The same tensors, sound: adjacent arrays do not overlap, empty tensors' pointers are ignored.  Where there is no
    device the next check fails as a HIP error."""
    if torch.cuda.is_available():
        pytest.skip("addresses that only a CPU run may pass")
    sound = [
        ([_tensor(zp)], {}),
        ([_tensor(zp, m=BASE + 256)], {}),
        ([_tensor(zp), _tensor(zp, 1, numel=0, p=None, grad=None, m=3, v=None, out=None)], {}),
        ([_tensor(zp, grad=None)], {}),
        ([_tensor(zp, p=None, out=None)], dict(out=0)),
        ([_tensor(zp, p=None, out=None, m=None, v=None)], dict(out=0, state=0)),
        ([_tensor(zp, m=BASE + 257, v=BASE + 321, m_scale=BASE + 385, v_scale=BASE + 387)], dict(state=4)),
    ]
    for tensors, kw in sound:
        assert _create(zp, tensors, **kw) == -5, kw
    # scales that reach one byte into the next array
    t = _tensor(zp, numel=65, m=BASE + 300, v=BASE + 400, m_scale=BASE + 500, v_scale=BASE + 502)
    assert _create(zp, [t], state=4) == -1


def _begin(zp, ctl=BASE, groups=None, n=1, max_norm=0.0, check=1, scaler=None):
    arr = (zp.AdamHParams * 16)(*(groups or [zp.AdamHParams(1e-3, 0.9, 0.999, 1e-8, 0.1)] * 16))
    return zp.lib.zero_step_begin(ctl, arr, n, max_norm, check, None if scaler is None else ctypes.byref(scaler), None)


def test_begin_refusals(zp):
    inf, nan = float("inf"), float("nan")
    assert _begin(zp, ctl=None) == -1
    assert zp.lib.zero_step_begin(BASE, None, 1, 0.0, 1, None, None) == -1
    assert _begin(zp, ctl=BASE + 4) == -2
    for kw in (dict(n=0), dict(n=17), dict(check=2), dict(max_norm=-1.0), dict(max_norm=inf), dict(max_norm=nan),
               dict(max_norm=1.0, check=0)):
        assert _begin(zp, **kw) == -1, kw
    H = zp.AdamHParams
    for h in (H(inf, .9, .99, 1e-8, 0), H(1, 1.0, .99, 1e-8, 0), H(1, -.1, .99, 1e-8, 0), H(1, .9, 1.0, 1e-8, 0),
              H(1, .9, nan, 1e-8, 0), H(1, .9, .99, 0, 0), H(1, .9, .99, inf, 0), H(1, .9, .99, 1e-8, nan)):
        assert _begin(zp, groups=[h] * 16) == -1
    good = H(1e-3, .9, .999, 1e-8, 0)
    assert _begin(zp, groups=[good, H(nan, .9, .999, 1e-8, 0)] + [good] * 14, n=2) == -1
    L = zp.LossScaler.make
    for s in (L(min_scale=0.0), L(min_scale=inf), L(backoff=0.0), L(backoff=nan), L(growth=0.0), L(growth=inf),
              L(growth_interval=-1)):
        assert _begin(zp, scaler=s) == -1
    if not torch.cuda.is_available():
        assert _begin(zp) == -5 and _begin(zp, scaler=L(scale=0.0, good_steps=-3)) == -5


def test_null_sets_are_refused(zp):
    lib = zp.lib
    assert lib.zero_grad_sumsq(None, BASE, 0, None, None) == -1
    assert lib.zero_adamw_step(None, BASE, 1, None) == -1
    assert lib.zero_states_convert(None, None, None) == -1
    assert lib.zero_tensor_set_bind_grads(None, None, None) == -1
    assert lib.zero_grad_sumsq_work_bytes(None) == 0


def test_binding_refuses_lists_that_do_not_fit(zp):
    z = torch.zeros(4)
    for kw in (dict(), dict(m=[z]), dict(m=[z], v=[z.to(torch.uint8)]), dict(m=[z], v=[z], m_scale=[z]),
               dict(grads=[z.double()]), dict(grads=[z, z.half()]), dict(p=[z.half()]), dict(grads=[z])):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            zp.TensorSet(**kw)
    for kw in (dict(scale=0.0), dict(scale=float("inf")), dict(t=-1), dict(device="cpu")):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            zp.StepControl(**kw)
