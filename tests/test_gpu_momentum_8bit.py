"""The rounding of an 8-bit momentum on the GPU: bit for bit against the oracle at every beta1, and over many steps
against the formula."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from oracle import tensor_set as T
from set_harness import SIZES, Twin, same_control
from test_gpu_tensor_set import follow, hparams

pytestmark = pytest.mark.gpu


class RoundedTwin(Twin):
    """A set with MXFP8 states whose host side rounds m as the group's beta1, or the set, says."""

    def __init__(self, sizes, *args, always=False, **kw):
        super().__init__(sizes, *args, state="mx", **kw)
        self.always = always
        self.set = zp.TensorSet(p=self.view["p"], grads=self.view["g"], m=self.view["m"], v=self.view["v"],
                                m_scale=self.view["ms"], v_scale=self.view["vs"], out=self.view.get("out"),
                                groups=self.groups, seed=self.seed, m_rounding="random" if always else "auto")

    def expect(self, c):
        if c.skip:
            return
        h = self.host
        for i, n in enumerate(self.sizes):
            m, v = T.decode(h["m"][i], h["ms"][i]), T.decode(h["v"][i], h["vs"][i])
            k, seed = c.consts[self.groups[i]], self.seed & 0xFFFFFFFF
            w, off = T.adamw_wide(c.groups[self.groups[i]], float(np.float32(c.lr_mult)), c.t, h["g"][i], c.grad_mult, h["p"][i], m, v, fast=True)
            self.bound[i] = w[0], off[0]
            h["p"][i], m, v = T.adamw(k, h["g"][i], c.grad_mult, h["p"][i], m, v)
            h["m"][i], h["ms"][i] = T.encode_m(m, k["beta1"], seed, i, c.t, self.always)
            h["v"][i], h["vs"][i] = T.encode(v, True, T.chances(n, seed, i, c.t))
            if "out" in h:
                h["out"][i] = h["p"][i]


def step(t, control, c, groups, max_norm, what):
    t.new_grads()
    t.set.grad_sumsq(control.sumsq)
    c.sumsq = t.sumsq()
    control.begin(hparams(groups), max_norm=max_norm)
    c.begin(groups, max_norm)
    t.set.adamw_step(control)
    torch.cuda.synchronize()
    follow(c, same_control(control, c, rel=2.0 ** -23))
    t.expect(c)
    t.compare(what)


def group(beta1, beta2=0.999):
    return T.HParams(1e-3, beta1, beta2, 1e-8, 0.1)


@pytest.mark.parametrize("always", [False, True])
@pytest.mark.parametrize("gaps", [None, "lines", "halves"])
@pytest.mark.parametrize("grad,out", [("fp16", "fp16"), ("bf16", "none"), ("fp32", "bf16")])
def test_codes_match_the_oracle_on_both_sides_of_the_limit(grad, out, gaps, always):
    """Groups on both sides in one set; starts anywhere, and on lines or half lines in every kind."""
    apart = {None: None, "lines": [(-n) % 128 for n in [0] + SIZES[:-1]], "halves": [32 + (-n) % 128 for n in [0] + SIZES[:-1]]}[gaps]
    below, above = float(np.float32(0.9444)), float(np.nextafter(np.float32(0.9444), np.float32(1)))
    groups = [group(0.9), group(below), group(above), group(0.99, 0.95), group(0.0)]
    t = RoundedTwin(SIZES, grad, out, seed=60, gaps=apart, always=always, groups=[i % 5 for i in range(len(SIZES))])
    control, c = zp.StepControl(scale=1024.0, t=7), T.Control(t=7, scale=1024.0)
    for k in range(3):
        step(t, control, c, groups, 0.05 if k else 0.0, f"{grad} {out} {gaps} step {k}")


@pytest.mark.parametrize("seed", range(8))
def test_random_sets_with_high_beta1(seed):
    rng = np.random.default_rng([11, seed])
    sizes = [int(2 ** rng.uniform(0, 13)) for _ in range(int(rng.integers(1, 20)))]
    gaps = None if seed % 2 else [int(x) for x in rng.integers(0, 130, len(sizes))]
    groups = [group(float(rng.uniform(0.9, 0.9999)), float(rng.uniform(0.5, 0.9999))) for _ in range(3)]
    print(f"[high beta1] seed {seed}", flush=True)
    t = RoundedTwin(sizes, ("fp16", "bf16", "fp32")[seed % 3], ("fp16", "none")[seed % 2], seed=3000 + seed, gaps=gaps,
                    groups=[int(rng.integers(3)) for _ in sizes], always=seed % 4 == 3)
    control, c = zp.StepControl(scale=1024.0, t=10 ** (seed % 5)), T.Control(t=10 ** (seed % 5), scale=1024.0)
    for k in range(3):
        step(t, control, c, groups, 0.05, f"step {k}")


def states(n):
    z = {k: [torch.zeros(n, dtype=torch.uint8, device="cuda")] for k in "mv"}
    z.update({k: [torch.zeros(-(-n // 32), dtype=torch.uint8, device="cuda")] for k in ("m_scale", "v_scale")})
    return z


@pytest.mark.parametrize("beta1,mode", [(0.9, "random"), (0.95, "auto"), (0.99, "auto")])
def test_m_and_p_follow_a_gradient_that_rises_falls_and_turns(beta1, mode):
    """One gradient for N elements: 1, then 0.1, then -1.  To nearest m would stop on the way (at 0.69, 0.5 and 0.22 of
    the first, and never turn for beta1 = 0.99).  |m| stays at 1 or below (the gradient's most; 1 is a code), where codes
    are 1/16 apart at most, so a rounding's error has mean zero (to 2^-17 of the gap) and deviation 1/32 at most,
    independent over elements and steps.  An error of step s reaches m of step t times beta1^(t - s), and with beta2 = 0,
    where the update is lr m / (|g| + eps), reaches p times lr times the sum of beta1^(t - s) / |g_t| over the later t.
    Six deviations of the mean over N, and what the chances' and fp32's roundings may add."""
    N, T1, T2, lr = 16384, 400, 300, 1e-3
    h = T.HParams(lr=lr, beta1=beta1, beta2=0.0)
    g = torch.empty(N, device="cuda")
    p = torch.zeros(N, device="cuda")
    z = states(N)
    s = zp.TensorSet(p=[p], grads=[g], seed=4, m_rounding=mode, **z)
    wide = [torch.empty(N, device="cuda") for _ in range(2)]
    read = zp.TensorSet(m=wide[:1], v=wide[1:])
    control, m, q, gs = zp.StepControl(t=10 ** 6), 0.0, 0.0, []
    for value in (1.0, 0.1, -1.0):
        value = float(np.float32(value))
        g.fill_(value)
        for _ in range(T1 if not gs else T2):
            control.begin(hparams([h]), check=False)
            s.adamw_step(control)
            m = h.beta1 * m + (1 - h.beta1) * value
            q -= h.lr * m / (abs(value) + h.eps)
            gs.append(abs(value))
        read.states_from(s)
        ways = np.zeros(len(gs))                        # of an error of step s into p, over lr
        for k in range(len(gs) - 2, -1, -1):
            ways[k] = h.beta1 * (1 / gs[k + 1] + ways[k + 1])
        off_m = 6 / 32 / np.sqrt(1 - h.beta1 ** 2) / np.sqrt(N) + 2.0 ** -17 / 16 / (1 - h.beta1) + 1e-5
        off_p = h.lr * (6 / 32 * np.sqrt((ways ** 2).sum()) / np.sqrt(N) + (2.0 ** -17 / 16 + 1e-6) * ways.sum()) + len(gs) * 2.0 ** -22
        got_m, got_p = wide[0].double().mean().item(), p.double().mean().item()
        assert abs(got_m - m) <= off_m, (value, got_m, m, off_m)
        assert abs(got_p - q) <= off_p, (value, got_p, q, off_p)


@pytest.mark.parametrize("beta1,beta2,mode", [(0.9, 0.95, "auto"), (0.9, 0.95, "random"), (0.95, 0.95, "auto"), (0.95, 0.999, "auto"), (0.99, 0.999, "auto")])
def test_rows_whose_gradients_end_stop_moving(beta1, beta2, mode):
    """As on the host (test_momentum_8bit_host.py, where the bound is derived), rows of a table that no batch names any
    more among them beside one that every batch does."""
    n, lr = 4096, 1e-4
    gen = torch.Generator(device="cuda").manual_seed(1)
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    s = zp.TensorSet(p=[p], grads=[g], seed=6, m_rounding=mode, **states(n))
    control, h = zp.StepControl(), T.HParams(lr=lr, beta1=beta1, beta2=beta2)
    at = None
    for k in range(3000):
        if k < 200:
            g.copy_(torch.randn(n, generator=gen, device="cuda") * 1e-3)
        elif k == 200:
            g.zero_()
        if k == 1400:
            at = p.clone()
        s.grad_sumsq(control.sumsq)
        control.begin(hparams([h]), max_norm=1.0)
        s.adamw_step(control)
    assert control.t.item() == 3000 and torch.isfinite(p).all()
    assert (p - at).abs().max().item() <= 10 * lr


@pytest.mark.parametrize("mode", ["auto", "random"])
def test_training_in_8_bits_follows_the_oracle(mode):
    """A linear model trained through autograd with states in 8 bits: on the gradients that came, every step's codes equal
    the oracle's, p is within a step's bound of the 64-bit form, and the copies are p rounded."""
    torch.manual_seed(0)
    n_in, n_out, batch = 96, 41, 64
    x = torch.randn(batch, n_in, device="cuda")
    y = x @ torch.randn(n_in, n_out, device="cuda") * 0.1
    t = RoundedTwin([n_in * n_out, n_out], "fp16", "fp16", seed=61, always=mode == "random", groups=[0, 1])
    groups = [group(0.9), group(0.95, 0.99)]
    control, c = zp.StepControl(scale=64.0), T.Control(scale=64.0)
    for k in range(20):
        w, b = (q.half().requires_grad_() for q in t.view["p"])
        loss = ((x.half() @ w.view(n_in, n_out) + b).float() - y).square().mean()
        (loss * 64.0).backward()
        for i, q in enumerate((w, b)):
            t.view["g"][i].copy_(q.grad)
            t.host["g"][i] = q.grad.float().cpu().numpy()
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(groups), max_norm=0.5)
        t.set.adamw_step(control)
        torch.cuda.synchronize()
        c.sumsq = t.sumsq()
        c.begin(groups, 0.5)
        follow(c, same_control(control, c, rel=2.0 ** -23))
        t.expect(c)
        t.compare(f"step {k}")
    assert c.t == 20


def test_a_captured_step_with_random_m_replays_as_new_steps():
    t = RoundedTwin(SIZES, "bf16", "fp16", seed=62, groups=[0] * len(SIZES))
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    groups = [group(0.97)]
    step(t, control, c, groups, 0.05, "eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(groups), max_norm=0.05)
        t.set.adamw_step(control)
    for k in range(4):
        t.new_grads()
        torch.randn(1 << 20, device="cuda").sum()
        c.sumsq = t.sumsq()
        graph.replay()
        torch.cuda.synchronize()
        c.begin(groups, 0.05)
        follow(c, same_control(control, c, rel=2.0 ** -23))
        t.expect(c)
        t.compare(f"replay {k}")


def test_m_rounding_is_refused_for_other_states():
    z = [torch.zeros(8, device="cuda") for _ in range(4)]
    with pytest.raises(ValueError, match="m_rounding"):
        zp.TensorSet(m=z[:1], v=z[1:2], m_rounding="random")
    f = zp.TensorSet(m=z[:1], v=z[1:2])
    assert zp.lib.zero_tensor_set_m_rounding(f._h, 1) == -7
    e = zp.TensorSet(p=z[2:3], **states(8))
    assert zp.lib.zero_tensor_set_m_rounding(e._h, 2) == -1
    assert zp.lib.zero_tensor_set_m_rounding(e._h, 1) == 0
