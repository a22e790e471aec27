"""Embedding, gated feed-forward layer, their gradients and the optimizer's step together, as a training step runs them:
each result against 64 bits, eager against captured, on streams and threads."""

import os
import threading

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES, half_unit
from oracle import activations as A

pytestmark = pytest.mark.gpu

HP = [zp.AdamHParams(1e-3, 0.9, 0.95, 1e-8, 0.1)]
U = 2.0 ** -24


class Model:
    """Rows of a table, then down(silu(gate x) * up x), all weights in `dtype` with fp32 masters; products of activations with
    weights are the library's."""

    def __init__(self, vocab, width, hidden, tokens, dtype, kind="silu", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.n = kind, tokens
        shapes = dict(table=(vocab, width), gate=(hidden, width), up=(hidden, width), down=(width, hidden), bias=(width,))
        self.master = {k: torch.randn(s, device="cuda", generator=g) * 0.1 for k, s in shapes.items()}
        self.w = {k: x.to(dtype) for k, x in self.master.items()}
        self.grad = {k: torch.zeros(s, device="cuda") for k, s in shapes.items()}
        e = lambda c: torch.empty(tokens, c, dtype=dtype, device="cuda")   # noqa: E731
        self.x, self.g, self.u, self.h, self.dh, self.dg, self.du, self.dx, self.dy = (
            e(c) for c in (width, hidden, hidden, hidden, hidden, hidden, hidden, width, width))
        self.kept = {k: zp.Checkpoint(tokens, c) for k, c in dict(x=width, g=hidden, u=hidden, h=hidden).items()}
        self.tokens = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        flat = lambda d: [d[k].view(-1) for k in shapes]   # noqa: E731
        state = [[torch.zeros(x.numel(), device="cuda") for x in self.master.values()] for _ in "mv"]
        self.state = state
        self.set = zp.TensorSet(p=flat(self.master), grads=flat(self.grad), m=state[0], v=state[1],
                                out=None if dtype == torch.float32 else flat(self.w))   # fp32: the masters themselves
        self.control = zp.StepControl()

    def batch(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens.copy_(torch.randint(-1, self.w["table"].shape[0], (self.n,), device="cuda", generator=g) // 3 * 2)
        self.dy.copy_(torch.randn(self.dy.shape, device="cuda", generator=g) * 0.1)

    def look_up(self, **kw):
        zp.embedding_lookup(self.w["table"], self.tokens, self.x, scale=3.0, **kw)
        self.kept["x"].store(self.x, **kw)

    def into(self):
        self.g.copy_(self.x @ self.w["gate"].t())
        self.u.copy_(self.x @ self.w["up"].t())

    def act(self, **kw):
        zp.activation(self.kind, self.g, self.h, self.kept["g"], up=self.u, up_checkpoint=self.kept["u"],
                      out_checkpoint=self.kept["h"], **kw)

    def down_grad(self, **kw):
        zp.weight_grad(self.dy, self.kept["h"], self.grad["down"], bias=self.grad["bias"], **kw)

    def through(self):
        self.dh.copy_(self.dy @ self.w["down"])

    def act_grad(self, **kw):
        zp.activation_grad(self.kind, self.dh, self.kept["g"], self.dg, up_checkpoint=self.kept["u"], dup=self.du, **kw)
        zp.weight_grad(self.dg, self.kept["x"], self.grad["gate"], **kw)
        zp.weight_grad(self.du, self.kept["x"], self.grad["up"], **kw)

    def back(self):
        self.dx.copy_(self.dg @ self.w["gate"] + self.du @ self.w["up"])

    def table_grad(self, **kw):
        zp.embedding_grad(self.dx, self.tokens, self.grad["table"], scale=3.0, **kw)

    def update(self, **kw):
        self.set.grad_sumsq(self.control.sumsq, **kw)
        self.control.begin(HP, max_norm=1.0, **kw)
        self.set.adamw_step(self.control, **kw)

    def own(self, **kw):
        """The calls of this library alone, one after the other."""
        for f in (self.look_up, self.act, self.down_grad, self.act_grad, self.table_grad, self.update):
            f(**kw)

    def whole(self):
        for f in (self.look_up, self.into, self.act, self.down_grad, self.through, self.act_grad, self.back, self.table_grad):
            f()

    def everything(self):
        kept = {f"{k} {n}": t for k, c in self.kept.items() for n, t in (("code", c.code), ("scale", c.scale))}
        return {**{k: getattr(self, k) for k in ("x", "h", "dg", "du")}, **kept, **{f"grad {k}": v for k, v in self.grad.items()},
                **{f"weight {k}": v for k, v in self.w.items()}, **{f"master {k}": v for k, v in self.master.items()},
                **{f"state {i} {j}": v for i, s in enumerate(self.state) for j, v in enumerate(s)}}


def same(a, b, what=""):
    b = b.everything()
    for k, v in a.everything().items():
        assert torch.equal(v, b[k]), f"{what}: {k}"


def wide(t):
    return t.detach().double().cpu().numpy()


def held_in(c):
    return A.load(c.code.cpu().numpy(), c.scale.cpu().numpy(), c.cols)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_step_against_64_bits(dtype):
    """Each call's result from what it read, and the gradients from those of the formula with what the checkpoints lost."""
    t = DTYPES[dtype]
    m = Model(500, 72, 200, 333, t)
    m.batch(1)
    m.whole()
    tokens = m.tokens.cpu().numpy()
    table, gate, up, down, dy = (wide(x) for x in (m.w["table"], m.w["gate"], m.w["up"], m.w["down"], m.dy))
    x = A.lookup(table, tokens, 0, 3.0)
    assert (np.abs(wide(m.x) - x) <= half_unit(x, t) * (1 + 2.0 ** -10)).all()
    g, u, xk = wide(m.g), wide(m.u), held_in(m.kept["x"])
    for k, want in (("x", m.x), ("g", m.g), ("u", m.u)):
        code, scale = A.store(want.float().cpu().numpy())
        assert np.array_equal(m.kept[k].code.cpu().numpy(), code) and np.array_equal(m.kept[k].scale.cpu().numpy(), scale)
    a = A.act("silu", g)[0]
    # as test_activation has it: 16 + 4 |z| half-units of the activation, one of the product, and the type's rounding
    off = np.abs(a * u) * U * (20 + 4 * np.abs(g)) + np.abs(g * u) * 2.0 ** -125
    assert (np.abs(wide(m.h) - a * u) <= off + half_unit(a * u, t) * (1 + 2.0 ** -9)).all()

    def product(got, left, right, bias=None):
        (dw, db), (mag, mag_b) = A.weight_grad(left, right)
        assert (np.abs(wide(got) - dw) <= 3 * (m.n + 2) * 2.0 ** -23 * mag).all()
        if bias is not None:
            assert (np.abs(wide(bias) - db) <= 3 * (m.n + 2) * 2.0 ** -23 * mag_b).all()

    product(m.grad["down"], dy, held_in(m.kept["h"]), m.grad["bias"])
    dg, du = wide(m.dg), wide(m.du)
    product(m.grad["gate"], dg, xk)
    product(m.grad["up"], du, xk)
    gk, uk, dh = held_in(m.kept["g"]), held_in(m.kept["u"]), wide(m.dh)
    ak, dak, terms = A.act("silu", gk)
    assert (np.abs(du - dh * ak) <= np.abs(dh) * (np.abs(ak) * U * (20 + 4 * np.abs(gk)) + np.abs(gk) * 2.0 ** -125)
            + half_unit(dh * ak, t) * (1 + 2.0 ** -9)).all()
    # as test_activation_grad has it, of the derivative's two terms
    size = terms * U * (24 + 8 * np.abs(gk)) + (1 + np.abs(gk)) * 2.0 ** -118
    assert (np.abs(dg - dh * uk * dak) <= np.abs(dh * uk) * size + half_unit(dh * uk * dak, t) * (1 + 2.0 ** -9)).all()
    dtable, mag, count = A.embedding_grad(wide(m.dx), tokens, 500, 0, 3.0)
    assert (np.abs(wide(m.grad["table"]) - dtable) <= (count[:, None] + 3) * U * mag + np.abs(dtable) * U).all()


@pytest.mark.parametrize("kind", A.KINDS)
def test_gradients_against_differences(kind):
    """d act / dz against central differences of the activation itself, both of this library and in fp32.  With a step of
    h = 2^-6 the differences are off by h^2 / 6 times the third derivative, below 2 for all of these, and by the
    values' own roundings (U (17 + 4 * 17 + 1) |act|, act below 6, on both sides) over h."""
    z = torch.linspace(-5.9, 5.9, 4096, device="cuda").view(64, 64)
    c = zp.Checkpoint(64, 64)
    c.store(z)
    c.load(z)
    h = 2.0 ** -6
    values = [torch.empty_like(z), torch.empty_like(z)]
    for out, step in zip(values, (h, -h)):
        zp.activation(kind, z + step, out)                    # z is a multiple of 2^-15, so its sum is exact
    slope = (values[0].double() - values[1].double()) / (2 * h)
    got = torch.empty_like(z)
    zp.activation_grad(kind, torch.ones_like(z), c, got)
    bound = h * h / 6 * 2 + U * 86 * 6 / h
    away = z.abs() > h if kind == "relu" else torch.ones_like(z, dtype=torch.bool)
    assert bool(((got.double() - slope).abs() <= bound)[away].all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_captured_steps_replay_like_eager_ones(dtype):
    """Two models' steps in two graphs, replayed in turn with the program's own work between, each against its eager twin
    bit for bit.  The table is large enough for the sorted way and the products for parts by tokens."""
    t = DTYPES[dtype]
    sizes = [(9000, 64, 136, 9001), (300, 136, 520, 700)]
    pairs = [(Model(*s, t, seed=i), Model(*s, t, seed=i)) for i, s in enumerate(sizes)]

    def fresh(step):
        for i, pair in enumerate(pairs):
            for m in pair:
                m.batch(10 * step + i)
                g = torch.Generator(device="cuda").manual_seed(100 + 10 * step + i)
                for x in (m.g, m.u, m.dh, m.dx):
                    x.copy_(torch.randn(x.shape, device="cuda", generator=g))

    fresh(0)
    for pair in pairs:
        for m in pair:
            m.own()
    graphs = []
    for _, m in pairs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            m.own()
    torch.cuda.synchronize()
    for step in range(1, 5):
        fresh(step)
        for (eager, _) in pairs:
            eager.own()
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        for g in graphs if step % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for i, (eager, captured) in enumerate(pairs):
            same(eager, captured, f"model {i}, replay {step}")


def test_another_stream_and_memory_that_goes():
    """Calls on a stream that is named, behind work that holds it up, while the current stream takes all memory that the
    calls have given back."""
    a, b = (Model(9000, 64, 136, 9001, torch.bfloat16, seed=3) for _ in range(2))
    for m in (a, b):
        m.batch(4)
        m.g.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
        m.u.copy_(m.g).mul_(0.5)
        m.dh.copy_(m.g).mul_(0.1)
        m.dx.fill_(0.25)
    a.own()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(4):
            busy = busy @ busy * 1e-3
    for f in (b.look_up, b.act, b.down_grad, b.act_grad, b.table_grad, b.update):
        f(stream=s)
        for n in (1 << 16, 1 << 20, 1 << 22):
            torch.full((n,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    same(a, b)


def test_two_threads_at_once():
    models = [[Model(9000, 64, 136, 9001, torch.float16, seed=i) for _ in range(2)] for i in range(2)]
    for i, pair in enumerate(models):
        for m in pair:
            m.batch(i)
            for x in (m.g, m.u, m.dh, m.dx):
                x.fill_(0.5 + i)
    for first, _ in models:
        for _ in range(5):
            first.own()
    torch.cuda.synchronize()
    went = []

    def work(m):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                m.own()
        s.synchronize()
        went.append(m)

    threads = [threading.Thread(target=work, args=(m,)) for _, m in models]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert len(went) == 2
    for i, (first, second) in enumerate(models):
        same(first, second, f"thread {i}")


def test_version_counters_and_times():
    m = Model(100, 40, 64, 50, torch.bfloat16)
    m.batch(0)
    m.whole()
    calls = {m.look_up: [m.x, m.kept["x"].code, m.kept["x"].scale], m.act: [m.h] + [t for k in "guh" for t in (m.kept[k].code, m.kept[k].scale)],
             m.down_grad: [m.grad["down"], m.grad["bias"]], m.act_grad: [m.dg, m.du, m.grad["gate"], m.grad["up"]], m.table_grad: [m.grad["table"]]}
    zp.set_kernel_timing(True)
    try:
        for call, written in calls.items():
            before = [t._version for t in written]
            call()
            assert all(t._version > v for t, v in zip(written, before)), call
            assert zp.last_kernel_ms() > 0
        assert len(zp.kernel_times()) == 8 and min(zp.kernel_times()) > 0
    finally:
        zp.set_kernel_timing(False)
    out = torch.empty(50, 40, device="cuda")
    m.kept["x"].load(out)
    assert out._version == 1
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    y = x * 2                                                 # its gradient needs nothing of y
    z = y.exp()                                               # this one needs z
    zp.activation("relu", z.detach(), z.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()


def test_the_readme_s_layer():
    """The README's code runs as it stands, and its gradients are those of its formulas on what it kept."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = next(b for b in text.split("```python\n")[1:] if b.startswith("tokens = ids.numel()")).split("```")[0]
    g = torch.Generator(device="cuda").manual_seed(7)
    vocab, width, hidden, n = 300, 64, 96, 130
    make = lambda *s: (torch.randn(*s, device="cuda", generator=g) * 0.2).bfloat16()   # noqa: E731
    v = dict(torch=torch, zp=zp, width=width, hidden=hidden, ids=torch.randint(0, vocab, (n,), device="cuda", generator=g),
             table=make(vocab, width), w_gate=make(hidden, width), w_up=make(hidden, width), w_down=make(width, hidden), dy=make(n, width),
             x=make(n, width), **{k: make(n, hidden) for k in ("g", "u", "h", "dh", "dg", "du")},
             **{f"grad_{k}": torch.empty(s, device="cuda") for k, s in dict(gate=(hidden, width), up=(hidden, width), down=(width, hidden),
                                                                         bias=(width,), table=(vocab, width)).items()})
    exec(code, v)
    kept = {k: held_in(c) for k, c in v["kept"].items()}
    for dw, left, right in (("grad_down", "dy", "h"), ("grad_gate", "dg", "x"), ("grad_up", "du", "x")):
        (want, want_b), (mag, mag_b) = A.weight_grad(wide(v[left]), kept[right])
        assert (np.abs(wide(v[dw]) - want) <= (n + 2) * 2.0 ** -23 * mag).all()
        if dw == "grad_down":
            assert (np.abs(wide(v["grad_bias"]) - want_b) <= (n + 2) * 2.0 ** -23 * mag_b).all()
    dx = wide(v["dg"] @ v["w_gate"] + v["du"] @ v["w_up"])
    want, mag, count = A.embedding_grad(dx, v["ids"].cpu().numpy(), vocab, 0, 1.0)
    assert (np.abs(wide(v["grad_table"]) - want) <= (count[:, None] + 3) * U * mag).all()
