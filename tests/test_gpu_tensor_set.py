"""The tensor sets on the GPU against the numpy oracle: bit for bit against its fp32 form, within derived bounds against
its 64-bit form."""

import threading

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from oracle import tensor_set as T
from set_harness import GRAD, SIZES, Twin, bits, read, same_control

pytestmark = pytest.mark.gpu

HP = [T.HParams(1e-3, 0.9, 0.999, 1e-8, 0.1), T.HParams(2e-3, 0.8, 0.95, 1e-6, 0.0)]


def hparams(hs):
    return [zp.AdamHParams(h.lr, h.beta1, h.beta2, h.eps, h.weight_decay) for h in hs]


def follow(c, d):
    """The oracle's control takes the device's factor and constants (their last bits come from a pow and a sum)."""
    c.grad_mult = d.grad_mult
    if not c.skip:
        names = ("beta1", "omb1", "beta2", "omb2", "decay", "step", "rbc2", "eps")
        for k, want in enumerate(c.consts):
            got = dict(zip(names, d.group[k]))
            for n in names:
                assert abs(got[n] - want[n]) <= 2.0 ** -23 * abs(want[n]), n
            c.consts[k] = got


def take_step(twins, control, c, groups=HP, max_norm=0.0, check=True, scaler=None, what=""):
    if check:
        for k, t in enumerate(twins):
            t.set.grad_sumsq(control.sumsq, accumulate=k > 0)
        c.sumsq = sum(t.sumsq() for t in twins)
    control.begin(hparams(groups), max_norm=max_norm, check=check, scaler=scaler)
    c.begin(groups, max_norm, check, scaler)
    for t in twins:
        t.set.adamw_step(control)
    torch.cuda.synchronize()
    follow(c, same_control(control, c, rel=2.0 ** -23))
    for t in twins:
        t.expect(c)
        t.compare(what)


@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_sumsq_against_64_bits(grad):
    for sizes, gaps in (([1], None), ([0], None), ([], None), ([1024], None), ([3, 0, 1025], None), (SIZES, None), ([40000] * 30 + [5], None),
                        ([2048, 1000, 4096], [64, 0, 24]), ([300000], [17]), ([1024, 1023, 961, 960], [63, 0, 0, 0])):
        t = Twin(sizes or [0], grad=grad, out="none", seed=len(sizes), gaps=gaps)
        out = torch.full((), -1.0, dtype=torch.float64, device="cuda")
        t.set.grad_sumsq(out)
        first = out.item()
        n = sum(sizes)
        # n exact squares (fp32's are rounded once), summed in some order: n 2^-53 relative at most
        assert abs(first - t.sumsq()) <= (n + 1) * 2.0 ** -53 * t.sumsq(), (grad, sizes)
        t.set.grad_sumsq(out)
        assert out.item() == first
        t.set.grad_sumsq(out, accumulate=True)
        assert out.item() == 2 * first


@pytest.mark.parametrize("value,want", [(np.inf, np.inf), (-np.inf, np.inf), (np.nan, np.nan), (65504.0, 65504.0 ** 2)])
@pytest.mark.parametrize("where", [0, 1000, 1500, 5999])
def test_sumsq_of_special_values(value, want, where):
    g = torch.zeros(6000, dtype=torch.float16, device="cuda")
    g[where] = value
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    zp.TensorSet(grads=[g]).grad_sumsq(out)
    assert out.item() == want or (np.isnan(want) and np.isnan(out.item()))


def test_a_norm_past_fp32_range_is_clipped_or_skipped():
    g = torch.full((5000,), 1e30, device="cuda")
    p, m, v = torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda")
    s, control = zp.TensorSet(p=[p], grads=[g], m=[m], v=[v]), zp.StepControl()
    s.grad_sumsq(control.sumsq)
    want = 5000 * float(np.float32(1e30)) ** 2
    assert abs(control.sumsq.item() - want) <= 5001 * 2.0 ** -53 * want
    control.begin(hparams(HP[:1]))
    s.adamw_step(control)
    assert control.skip.item() == 1 and int(torch.count_nonzero(p)) == 0
    control.begin(hparams(HP[:1]), max_norm=1.0)
    s.adamw_step(control)
    # every value clipped to 1 / sqrt(5000), times 1 - beta1 with beta1 as fp32 has it (a difference that is exact):
    # the factor's rounding and the two products', 3 * 2^-24
    want = (1 - HP[0].beta1) / np.sqrt(5000)
    assert control.skip.item() == 0 and (m.double() / want - 1).abs().max().item() <= 3.01 * 2.0 ** -24
    assert torch.isfinite(p).all() and torch.isfinite(v).all()
    for bad in (1e-50, -1.0, float("nan"), float("inf")):
        with pytest.raises((ValueError, zp.ZeroError)):
            control.begin(hparams(HP[:1]), max_norm=bad)


def test_bit_patterns_in_int16_are_fp16():
    """fp16 data as int16 patterns, as the rest of the library passes it."""
    a, b = Twin(SIZES, "fp16", "fp16", "fp32", seed=50), Twin(SIZES, "fp16", "fp16", "fp32", seed=50)
    s = zp.TensorSet(p=b.view["p"], grads=[x.view(torch.int16) for x in b.view["g"]], m=b.view["m"], v=b.view["v"],
                     out=[x.view(torch.int16) for x in b.view["out"]], groups=b.groups)
    for t, tensors in ((a, a.set), (b, s)):
        control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
        tensors.grad_sumsq(control.sumsq)
        control.begin(hparams(HP), max_norm=0.05)
        tensors.adamw_step(control)
        c.sumsq = t.sumsq()
        c.begin(HP, 0.05)
        follow(c, same_control(control, c, rel=2.0 ** -23))
        t.expect(c)
        t.compare()


def test_replays_read_gradients_that_are_bound_later():
    t = Twin(SIZES, "bf16", "none", "mx", seed=51)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    take_step([t], control, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(HP))
        t.set.adamw_step(control)
    del t.kinds["g"]                                          # the old buffer is not compared
    for shift in (0, 1, 3):                                   # other places, at other alignments
        t.new_grads()
        moved = [torch.cat([x.new_zeros(shift), x])[shift:] for x in t.view["g"]]
        for x in t.view["g"]:
            x.fill_(float("nan"))
        t.set.bind_grads(moved)
        c.sumsq = t.sumsq()
        graph.replay()
        torch.cuda.synchronize()
        c.begin(HP)
        follow(c, same_control(control, c, rel=2.0 ** -23))
        t.expect(c)
        t.compare(f"moved by {shift}")


@pytest.mark.parametrize("state", ["fp32", "mx"])
@pytest.mark.parametrize("out", ["fp16", "bf16", "none"])
@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_steps_match_the_oracle(grad, out, state):
    print(f"[adamw] {grad} {out} {state}", flush=True)
    t = Twin(SIZES, grad, out, state, seed=11)
    control, c = zp.StepControl(scale=1024.0, t=3), T.Control(t=3, scale=1024.0)
    for step in range(4):
        t.new_grads()
        take_step([t], control, c, max_norm=0.05 if step % 2 else 0.0, check=step != 2, what=f"step {step}")


@pytest.mark.parametrize("state", ["fp32", "mx"])
@pytest.mark.parametrize("first", [0, 1, 16, 31, 32, 33, 63, 64, 96, 100])
def test_starts_that_all_kinds_share(first, state):
    """Tensors whose starts stand in the same place in every buffer: on lines, on half lines, beside them.  Sizes around
    those at which a shifted tile needs one tile more."""
    sizes = [5000, 1024 - first % 64, 1025 - first % 64, 64 * 33, 32, 992, 1, 4096 - 32, 960, 961, 31]
    gaps = [first] + [0, 64, 32, 128, 1, 0, 33, 64, 31, 2][: len(sizes) - 1]
    t = Twin(sizes, "bf16", "fp16", state, seed=first, gaps=gaps)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    for step in range(2):
        t.new_grads()
        take_step([t], control, c, max_norm=0.05, what=f"step {step}")
    if state == "mx":
        wide = [[torch.empty(n + 3, device="cuda")[first % 4: first % 4 + n] if n < 64 else torch.empty(n, device="cuda") for n in sizes] for _ in range(2)]
        f = zp.TensorSet(m=wide[0], v=wide[1])
        f.states_from(t.set)
        for i in range(len(sizes)):
            for k, s, w in (("m", "ms", wide[0]), ("v", "vs", wide[1])):
                assert np.array_equal(bits(w[i]), T.decode(t.host[k][i], t.host[s][i]).view(np.int32)), (i, k)
        for k in ("m", "v", "ms", "vs"):
            for x in t.view[k]:
                x.zero_()
        t.set.states_from(f)
        for i in range(len(sizes)):
            for k, s in (("m", "ms"), ("v", "vs")):
                t.host[k][i], t.host[s][i] = T.encode(T.decode(t.host[k][i], t.host[s][i]), k == "v")
        t.compare("read back")


@pytest.mark.parametrize("state", ["fp32", "mx"])
def test_a_step_against_64_bits(state):
    """From values that the states hold exactly, p (and fp32 states) within the bound that the roundings add up to."""
    t = Twin([50001, 257, 33], "fp32", "none", state, seed=5)
    control = zp.StepControl(scale=256.0, t=41)
    before = [{k: a[i].copy() for k, a in t.host.items()} for i in range(3)]
    t.set.grad_sumsq(control.sumsq)
    control.begin(hparams(HP), max_norm=0.05)
    t.set.adamw_step(control)
    norm = np.sqrt(t.sumsq()) / 256.0
    assert norm > 0.05
    for i, b in enumerate(before):
        m = T.decode(b["m"], b["ms"]) if state == "mx" else b["m"]
        v = T.decode(b["v"], b["vs"]) if state == "mx" else b["v"]
        want, off = T.adamw_wide(HP[i % 2], 1.0, 42, b["g"], 0.05 / norm / 256.0, b["p"], m, v,
                                 fast=state == "mx")
        names = "p" if state == "mx" else "pmv"
        for k, w, o in zip(names, want, off):
            d = np.abs(t.view[k][i].cpu().numpy().astype(np.float64) - w)
            assert (d <= o).all(), (k, float((d / o).max()))
        if state == "mx":
            for k, w, s, half in (("m", want[1], "ms", 2.0 ** -4), ("v", want[2], "vs", 2.0 ** -3)):
                got = T.decode(t.view[k][i].cpu().numpy(), t.view[s][i].cpu().numpy()).astype(np.float64)
                power = np.repeat(2.0 ** (t.view[s][i].cpu().numpy().astype(np.float64) - 127), 32)[:got.size]
                # m: half a step, v: one; steps are 2^-3 of the power of two below, at least 2^-9 of the scale
                # (v above zero is at least one); 2^-20 covers the fp32 roundings before
                lim = np.maximum(np.abs(w) * half, power * 2.0 ** -9 * (0.5 if k == "m" else 1)) * (1 + 2.0 ** -20)
                assert (np.abs(got - w) <= lim).all(), k


@pytest.mark.parametrize("state", ["fp32", "mx"])
@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_a_skipped_step_changes_nothing(state, bad):
    t = Twin(SIZES, "fp16", "bf16", state, seed=2)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    rule = zp.LossScaler.make(min_scale=300.0, growth_interval=2)
    for step in range(7):
        t.new_grads()
        if step in (1, 2, 5):
            i = len(SIZES) - 1 if step == 1 else step
            t.view["g"][i][-1] = bad
            t.host["g"][i][-1] = bad
        take_step([t], control, c, max_norm=1.0, scaler=rule, what=f"step {step}")
    # 1024, two skips: 512 and the floor 300, two taken steps: 600, a skip: 300
    assert (c.skipped, c.t, c.scale) == (3, 4, 300.0)


def test_device_side_values_that_skip():
    """A scale or factor on lr that the caller left unusable, and a norm whose squares would leave fp32."""
    t = Twin([100], "fp32", "none", "fp32", seed=1)
    for name, value, std in (("scale", 0.0, 1), ("scale", float("inf"), 1), ("scale", float("nan"), 1),
                             ("lr_mult", float("inf"), 1), ("lr_mult", float("nan"), 1), ("t", -1, 1), ("t", (1 << 63) - 1, 1),
                             (None, 0, 2.0 ** 63)):
        t.new_grads([np.full(100, std, np.float32)])
        control = zp.StepControl()
        if name:
            getattr(control, name).fill_(value)
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(HP[:1]))
        t.set.adamw_step(control)
        assert (control.skip.item(), control.t.item(), control.skipped.item()) == (1, value if name == "t" else 0, 1), name
        t.compare(str(name))
    for scale in (float("nan"), float("inf"), 2.0 ** 127, 1.0):       # a dynamic scale comes back from any of them
        control = zp.StepControl()
        control.scale.fill_(scale)
        control.sumsq.fill_(float("inf") if scale == 1.0 else 1.0)
        control.begin(hparams(HP[:1]), scaler=zp.LossScaler.make(min_scale=0.75))
        assert (control.skip.item(), control.scale.item()) == (1, 2.0 ** 126 if scale == 2.0 ** 127 else 0.75), scale
    control = zp.StepControl()                        # clipped, the same gradients are fine
    t.set.grad_sumsq(control.sumsq)
    control.begin(hparams(HP[:1]), max_norm=1.0)
    t.set.adamw_step(control)
    assert control.skip.item() == 0 and torch.isfinite(t.view["p"][0]).all()


def test_two_sets_under_one_norm():
    """Large tensors in 8 bits, small ones in 32, one clip over both, and a schedule on the device."""
    a = Twin([4099, 50001], "fp16", "fp16", "mx", seed=7)
    b = Twin([1, 33, 700], "fp16", "fp16", "fp32", seed=8)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    for step in range(3):
        for t in (a, b):
            t.new_grads()
        control.lr_mult.fill_(0.5 ** step)
        c.lr_mult = 0.5 ** step
        take_step([a, b], control, c, max_norm=0.1, what=f"step {step}")


def test_gradients_bound_later_and_replaced():
    t = Twin(SIZES, "bf16", "none", "fp32", seed=4)
    p = [x.clone() for x in t.view["p"]]
    state = dict(m=[x.clone() for x in t.view["m"]], v=[x.clone() for x in t.view["v"]])
    control = zp.StepControl()
    control.begin(hparams(HP), check=False)
    never = zp.TensorSet(p=p, **state)
    late = zp.TensorSet(p=p, grad_dtype=torch.bfloat16, **state)
    for s in (never, late):
        with pytest.raises(zp.ZeroError, match="STATE"):
            s.adamw_step(control)
        with pytest.raises(zp.ZeroError, match="STATE"):
            s.grad_sumsq(control.sumsq)
    with pytest.raises((ValueError, zp.ZeroError)):
        never.bind_grads(t.view["g"])
    late.bind_grads([torch.ones_like(x) for x in t.view["g"]])
    late.grad_sumsq(control.sumsq)
    assert control.sumsq.item() == sum(SIZES)
    with pytest.raises(ValueError):
        t.set.bind_grads([x.float() for x in t.view["g"]])
    with pytest.raises(zp.ZeroError, match="INVALID_ARG"):
        t.set.bind_grads([v.view(torch.bfloat16)[: v.numel()] for v in t.view["p"]])   # in the master values
    moved = [torch.cat([x.new_zeros(1), x])[1:] for x in t.view["g"]]                  # 2-byte aligned copies
    for x in t.view["g"]:
        x.fill_(float("nan"))                                                          # the old ones are not read again
    t.set.bind_grads(moved)
    del t.kinds["g"]                                                                   # the old buffer is not compared
    c = T.Control(scale=1024.0)
    take_step([t], zp.StepControl(scale=1024.0), c, max_norm=0.05)


def test_bind_grads_refusal_keeps_the_old_addresses():
    t = Twin([100, 200], "fp16", "none", "fp32", seed=6)
    with pytest.raises(zp.ZeroError):
        t.set.bind_grads([t.view["g"][0], t.view["m"][1].view(torch.float16)[:200]])
    c = T.Control(scale=1024.0)
    take_step([t], zp.StepControl(scale=1024.0), c)


def test_refusals_on_the_device():
    t = Twin([100, 40], "fp16", "fp16", "mx", seed=3)
    control = zp.StepControl()
    with pytest.raises(ValueError, match="begun"):
        t.set.adamw_step(control)
    with pytest.raises(zp.ZeroError, match="INVALID_ARG"):
        control.begin([])
    control.begin(hparams(HP[:1]), check=False)
    with pytest.raises(zp.ZeroError, match="group"):
        t.set.adamw_step(control)                           # tensor 1 is of group 1
    grads_only = zp.TensorSet(grads=t.view["g"])
    states_only = zp.TensorSet(m=t.view["m"], v=t.view["v"], m_scale=t.view["ms"], v_scale=t.view["vs"])
    control.begin(hparams(HP), check=False)
    for s in (grads_only, states_only):
        with pytest.raises(zp.ZeroError, match="STATE"):
            s.adamw_step(control)
    with pytest.raises(zp.ZeroError, match="STATE"):
        states_only.grad_sumsq(control.sumsq)
    with pytest.raises(zp.ZeroError, match="STATE"):
        states_only.states_from(grads_only)
    with pytest.raises(zp.ZeroError, match="same type"):
        states_only.states_from(t.set)
    f = [torch.zeros(n, device="cuda") for n in (100, 41)]
    with pytest.raises(zp.ZeroError, match="sizes"):
        zp.TensorSet(m=f, v=[x.clone() for x in f]).states_from(t.set)
    mem = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    inside = zp.TensorSet(m=[mem[:400].view(torch.float32)], v=[mem[400:800].view(torch.float32)])
    codes = zp.TensorSet(m=[mem[700:800]], v=[mem[1000:1100]], m_scale=[mem[1200:1204]], v_scale=[mem[1204:1208]])
    with pytest.raises(zp.ZeroError, match="overlap"):
        inside.states_from(codes)
    with pytest.raises(ValueError):
        t.set.grad_sumsq(torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        zp.TensorSet(grads=[torch.zeros(8, 8, device="cuda").half()[:, ::2]])
    t.compare()                                              # nothing was written


@pytest.mark.parametrize("sizes", [SIZES, [0], [1], [200003]])
def test_states_convert_both_ways(sizes):
    t = Twin(sizes, "fp16", "none", "mx", seed=9)
    wide = [[torch.full((n,), float("nan"), device="cuda") for n in sizes] for _ in range(2)]
    f = zp.TensorSet(m=wide[0], v=wide[1])
    f.states_from(t.set)
    for i in range(len(sizes)):
        for k, s, w in (("m", "ms", wide[0]), ("v", "vs", wide[1])):
            assert np.array_equal(bits(w[i]), T.decode(t.host[k][i], t.host[s][i]).view(np.int32)), (i, k)
    # fp32 states of every magnitude to 8 bits
    rng = np.random.default_rng(1)
    for i, n in enumerate(sizes):
        m = (rng.standard_normal(n) * 10.0 ** rng.uniform(-44, 30, 1)).astype(np.float32)
        v = np.square(rng.standard_normal(n) * 10.0 ** rng.uniform(-22, 15, 1)).astype(np.float32)
        m[::7], v[::5] = 0, 0
        wide[0][i].copy_(torch.from_numpy(m))
        wide[1][i].copy_(torch.from_numpy(v))
        t.host["m"][i], t.host["ms"][i] = T.encode(m, False)
        t.host["v"][i], t.host["vs"][i] = T.encode(v, True)
    t.set.states_from(f)
    torch.cuda.synchronize()
    t.compare()


def test_scale_byte_ends():
    """Scales 0 (2^-127) to 254 decode to their products; encoding reaches its own ends, 1 and 247."""
    s = torch.arange(255, dtype=torch.int32).to(torch.uint8)
    code = torch.randint(0, 0x7F, (255 * 32,), dtype=torch.uint8)
    code |= torch.randint(0, 2, code.shape, dtype=torch.uint8) * 0x80
    dev = [x.cuda() for x in (code, code & 0x7F, s, s.clone())]
    wide = [torch.zeros(code.numel(), device="cuda") for _ in range(2)]
    f, e = zp.TensorSet(m=wide[:1], v=wide[1:]), zp.TensorSet(m=dev[:1], v=dev[1:2], m_scale=[dev[2].view(torch.float8_e8m0fnu)], v_scale=dev[3:])
    f.states_from(e)
    with np.errstate(over="ignore"):
        want = T.decode(code.numpy(), s.numpy())
    got = wide[0].cpu().numpy()
    assert np.array_equal(got, want)
    big = torch.tensor([np.finfo(np.float32).max, 0.0, 1e-45] + [1.0] * 29, device="cuda")
    tiny = torch.tensor([1e-45, 0.0] + [0.0] * 30, device="cuda")
    x = torch.cat([big, tiny, torch.zeros(32, device="cuda")])
    f, out = zp.TensorSet(m=[x], v=[x.clone()]), [torch.zeros(96, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(3, dtype=torch.uint8, device="cuda") for _ in range(2)]
    zp.TensorSet(m=out[:1], v=out[1:], m_scale=sc[:1], v_scale=sc[1:]).states_from(f)
    for k, positive in ((0, False), (1, True)):
        c, b = T.encode(x.cpu().numpy(), positive)
        assert np.array_equal(out[k].cpu().numpy(), c) and np.array_equal(sc[k].cpu().numpy(), b)
        assert list(b) == [247, 1, 1]


@pytest.mark.parametrize("state", ["fp32", "mx"])
def test_captured_steps_replay_like_eager_ones(state):
    """One captured step, replayed with new gradients, another learning rate and an overflow between eager work, against
    the oracle; the step count advances on the device, so each replay is a new step."""
    t = Twin(SIZES + [300000], "fp16", "fp16", state, seed=12)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    rule = zp.LossScaler.make(growth_interval=3)
    take_step([t], control, c, max_norm=0.05, scaler=rule, what="eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(HP), max_norm=0.05, scaler=rule)
        t.set.adamw_step(control)
    torch.cuda.synchronize()
    t.compare("capturing runs nothing")
    for step in range(6):
        t.new_grads()
        if step == 2:
            t.view["g"][6][0] = float("inf")
            t.host["g"][6][0] = np.inf
        control.lr_mult.fill_(1.0 / (1 + step))
        c.lr_mult = float(np.float32(1.0 / (1 + step)))
        torch.randn(1 << 20, device="cuda").sum()             # the program's own work between replays
        c.sumsq = t.sumsq()
        graph.replay()
        torch.cuda.synchronize()
        c.begin(HP, 0.05, True, rule)
        follow(c, same_control(control, c, rel=2.0 ** -23))
        t.expect(c)
        t.compare(f"replay {step}")
        if step == 3:                                         # an eager step in between, with memory of its own
            take_step([t], control, c, max_norm=0.05, scaler=rule, what="eager between")


def test_a_set_that_goes_during_a_capture():
    t = Twin([5000, 70], "fp16", "none", "fp32", seed=52)
    other = zp.TensorSet(grads=[torch.ones(100, device="cuda")])
    out = torch.zeros((), dtype=torch.float64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.set.grad_sumsq(out)
        del other                                             # collected here
        t.set.grad_sumsq(out, accumulate=True)
    assert len(zp.TensorSet._late) == 1
    for _ in range(3):
        graph.replay()
        assert abs(out.item() - 2 * t.sumsq()) <= 6000 * 2.0 ** -53 * 2 * t.sumsq()
    zp.TensorSet(grads=[torch.ones(3, device="cuda")]).close()
    assert not zp.TensorSet._late


def test_two_graphs_of_one_set_on_two_streams():
    """Sums of one set captured twice and replayed at the same time do not share a workspace."""
    g = torch.randn(3_000_000, device="cuda")
    s = zp.TensorSet(grads=[g])
    outs = [torch.zeros(1, dtype=torch.float64, device="cuda") for _ in range(2)]
    s.grad_sumsq(outs[0])
    want = outs[0].item()
    graphs = []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                s.grad_sumsq(o)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert [o.item() for o in outs] == [want, want]


def test_another_stream():
    t = Twin(SIZES, "bf16", "bf16", "mx", seed=13)
    control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    t.set.grad_sumsq(control.sumsq, stream=st)
    control.begin(hparams(HP), max_norm=0.05, stream=st)
    t.set.adamw_step(control, stream=st)
    st.synchronize()
    c.sumsq = t.sumsq()
    c.begin(HP, 0.05)
    follow(c, same_control(control, c, rel=2.0 ** -23))
    t.expect(c)
    t.compare()


def test_two_threads_with_their_own_sets():
    twins = [Twin(SIZES, "fp16", "fp16", s, seed=20 + k) for k, s in enumerate(("fp32", "mx"))]
    errors = []

    def work(t):
        try:
            st = torch.cuda.Stream()
            control, c = zp.StepControl(scale=1024.0), T.Control(scale=1024.0)
            st.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(st):
                for _ in range(5):
                    t.set.grad_sumsq(control.sumsq)
                    control.begin(hparams(HP), max_norm=0.05)
                    t.set.adamw_step(control)
                    st.synchronize()
                    c.sumsq = t.sumsq()
                    c.begin(HP, 0.05)
                    follow(c, same_control(control, c, rel=2.0 ** -23))
                    t.expect(c)
                    t.compare()
        except Exception as e:                                # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(t,)) for t in twins]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    for t in twins:
        t.compare()


def test_equal_runs_give_equal_bits_and_another_seed_does_not():
    def run(seed):
        t = Twin([50001], "fp16", "none", "mx", seed=30)
        s = zp.TensorSet(p=t.view["p"], grads=t.view["g"], m=t.view["m"], v=t.view["v"], m_scale=t.view["ms"],
                         v_scale=t.view["vs"], seed=seed)
        control = zp.StepControl(scale=1024.0)
        for _ in range(5):
            s.grad_sumsq(control.sumsq)
            control.begin(hparams(HP))
            s.adamw_step(control)
        return bits(t.view["p"][0]), bits(t.view["v"][0])
    a, b, c = run(1), run(1), run(2)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert not np.array_equal(a[1], c[1])


@pytest.mark.parametrize("seed", range(24))
def test_random_sets(seed):
    """Seeded sets of any sizes, starts, types, groups and hyper-parameters, three steps each with clip, skip and
    schedule drawn, then the states converted to the other type and back."""
    rng = np.random.default_rng([7, seed])
    pick = lambda *x: x[int(rng.integers(len(x)))]            # noqa: E731
    sizes = [int(2 ** rng.uniform(0, pick(5, 9, 12, 16))) + int(rng.integers(0, 2)) * int(rng.integers(-1, 2)) for _ in range(int(rng.integers(1, 30)))]
    grad, out, state = pick("fp16", "bf16", "fp32"), pick("fp16", "bf16", "none"), pick("fp32", "mx")
    gaps = pick(None, [int(x) for x in rng.integers(0, 130, len(sizes))], [int(x) * 32 for x in rng.integers(0, 5, len(sizes))])
    print(f"[random] seed {seed}: {grad} {out} {state} {len(sizes)} tensors, gaps {gaps is not None}", flush=True)
    groups = [T.HParams(float(10 ** rng.uniform(-5, -2)), float(rng.uniform(0, 0.99)), float(rng.uniform(0.5, 0.9999)),
                        float(10 ** rng.uniform(-10, -4)), pick(0.0, 0.1)) for _ in range(int(rng.integers(1, 17)))]
    t = Twin(sizes, grad, out, state, seed=1000 + seed, gaps=gaps, groups=[int(rng.integers(len(groups))) for _ in sizes])
    t0 = int(pick(0, 1, 10 ** int(rng.integers(1, 7))))
    control, c = zp.StepControl(scale=1024.0, t=t0), T.Control(t=t0, scale=1024.0)
    rule = zp.LossScaler.make(growth_interval=2)
    for step in range(3):
        t.new_grads()
        if rng.random() < 0.2 and sum(sizes):
            i = int(rng.choice([k for k, n in enumerate(sizes) if n]))
            at = int(rng.integers(sizes[i]))
            t.view["g"][i][at] = float("inf")
            t.host["g"][i][at] = np.inf
        c.lr_mult = float(np.float32(rng.uniform(0, 2)))
        control.lr_mult.fill_(c.lr_mult)
        check = rng.random() < 0.8 or np.isinf(t.sumsq())
        take_step([t], control, c, groups=groups, max_norm=float(np.float32(pick(0.0, 0.01, 1.0))) if check else 0.0, check=check,
                  scaler=pick(None, rule), what=f"step {step}")
    if state == "mx":
        wide = [[torch.empty(n + 1, device="cuda")[1:] for n in sizes] for _ in range(2)]
        f = zp.TensorSet(m=wide[0], v=wide[1])
        f.states_from(t.set)
        for i in range(len(sizes)):
            for k, s, w in (("m", "ms", wide[0]), ("v", "vs", wide[1])):
                assert np.array_equal(bits(w[i]), T.decode(t.host[k][i], t.host[s][i]).view(np.int32)), (i, k)
    else:
        mx = Twin(sizes, grad, "none", "mx", seed=2000 + seed, gaps=gaps)
        mx.set.states_from(t.set)
        for i in range(len(sizes)):
            for k, s in (("m", "ms"), ("v", "vs")):
                mx.host[k][i], mx.host[s][i] = T.encode(t.host[k][i], k == "v")
        mx.compare("to 8 bits")
        t.compare("from 32 bits")


def test_empty_sets_and_many_tiny_tensors():
    z = [torch.zeros(0, device="cuda")]
    control = zp.StepControl()
    s = zp.TensorSet(p=z, grads=z, m=z, v=z)
    control.sumsq.fill_(7.0)
    s.grad_sumsq(control.sumsq)
    assert control.sumsq.item() == 0.0
    control.begin(hparams(HP[:1]))
    s.adamw_step(control)
    assert control.t.item() == 1
    rng = np.random.default_rng(2)
    t = Twin([int(x) for x in rng.integers(1, 40, 3000)], "fp16", "bf16", "mx", seed=14)
    take_step([t], zp.StepControl(scale=1024.0), T.Control(scale=1024.0), max_norm=0.05)


def test_a_tensor_past_2_31_elements():
    """Element numbers past 2^31 and byte offsets past 2^32: the last tiles against the oracle, and the sum."""
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-4099:] = 1.0
    g[: 1 << 20] = 2.0
    p = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    s = zp.TensorSet(p=[p], grads=[g], m=[m], v=[v], m_scale=[ms], v_scale=[vs], seed=5)
    control, c = zp.StepControl(), T.Control()
    s.grad_sumsq(control.sumsq)
    assert control.sumsq.item() == 4099 + 4 * (1 << 20)
    control.begin(hparams(HP[:1]), check=False)
    s.adamw_step(control)
    torch.cuda.synchronize()
    c.begin(HP[:1], check=False)
    follow(c, read(control))
    k = 4099 + 1024
    lo = n - n % 1024 - 4096 - 1024
    k = n - lo
    hg = g[lo:].float().cpu().numpy()
    zero = [np.zeros(k, np.float32) for _ in range(3)]
    _, hm, hv = T.adamw(c.consts[0], hg, c.grad_mult, *zero)
    wide, off = T.adamw_wide(HP[0], 1.0, 1, hg, 1.0, *zero, fast=True)
    assert (np.abs(p[lo:].cpu().numpy().astype(np.float64) - wide[0]) <= off[0]).all()
    for x, sc, want, w in ((m, ms, hm, None), (v, vs, hv, T.chances(k, 5, 0, 1, lo))):
        code, scale = T.encode(want, w is not None, w)
        assert np.array_equal(x[lo:].cpu().numpy(), code) and np.array_equal(sc[lo // 32:].cpu().numpy(), scale)
    middle = slice(1 << 20, lo)                    # no gradient, no state, no decay of zeros
    assert int(torch.count_nonzero(p[middle])) == 0 and int(torch.count_nonzero(m[middle])) == 0


def test_a_variance_in_8_bits_follows_a_falling_gradient():
    """v moves by 1% a step here, under half of an e4m3 step: rounded to nearest it would stay where it is.  Rounded at
    random its mean over N elements follows the formula.  A rounding's error has mean zero and, the neighbours being v / 8
    apart at most, variance (v / 16)^2 at most; an error of step s is multiplied by beta2^(T - s) until the end, and
    v_s beta2^(T - s) <= v_T, so T steps add up to at most T (v_T / 16)^2, independent over the elements: 6 deviations of the
    mean are 6 sqrt(T) / 16 / sqrt(N) of v_T."""
    N, T1, T2 = 16384, 50, 250
    h = T.HParams(lr=0.0, beta1=0.0, beta2=0.99)
    g = torch.ones(N, device="cuda")
    z = {k: [torch.zeros(N, dtype=torch.uint8, device="cuda")] for k in "mv"}
    z.update({k: [torch.zeros(N // 32, dtype=torch.uint8, device="cuda")] for k in ("m_scale", "v_scale")})
    s = zp.TensorSet(p=[torch.zeros(N, device="cuda")], grads=[g], seed=9, **z)
    control, v = zp.StepControl(), 0.0
    for step in range(T1 + T2):
        if step == T1:
            g.fill_(0.05)
        control.begin(hparams([h]), check=False)
        s.adamw_step(control)
        v = h.beta2 * v + (1 - h.beta2) * (1.0 if step < T1 else float(np.float32(0.05)) ** 2)
    wide = [torch.empty(N, device="cuda") for _ in range(2)]
    zp.TensorSet(m=wide[:1], v=wide[1:]).states_from(s)
    mean = wide[1].double().mean().item()
    assert v < 0.05 and abs(mean - v) <= 6 * np.sqrt(T1 + T2) / 16 / np.sqrt(N) * v, (mean, v)


def test_uploads_are_refused_while_the_stream_is_captured():
    t = Twin([100, 200], "fp16", "none", "fp32", seed=41)
    g = torch.ones(64, device="cuda")
    out = torch.zeros((), dtype=torch.float64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(zp.ZeroError, match="captured"):
            t.set.bind_grads(t.view["g"])
        with pytest.raises(zp.ZeroError, match="captured"):
            zp.TensorSet(grads=[g])
        t.set.grad_sumsq(out)                                 # the capture goes on
    for _ in range(3):
        out.fill_(-1.0)
        graph.replay()
        assert abs(out.item() - t.sumsq()) <= 301 * 2.0 ** -53 * t.sumsq()


@pytest.mark.parametrize("n_ranks,align", [(1, 1), (3, 1), (4, 32), (7, 64)])
def test_partitioned_steps_equal_the_whole_model_s(n_ranks, align):
    """A ZeRO-2 step from end to end, rank after rank on one device: gradients reduced to their owner, each rank's set
    made of the tensor pieces of its shard, one norm over all ranks, the update, and the fp16 copies in the rank's slot of
    the gather buffer.  Each element's result hangs on no other's, so it equals the step of one set of whole tensors."""
    rng = np.random.default_rng(n_ranks)
    numels = [1600, 7, 50257, 1, 3000, 129, 64, 9000]
    lists = [[torch.from_numpy((rng.standard_normal(n) * 0.5).astype(np.float16)).cuda() for n in numels] for _ in range(2)]
    lay = zp.partition_layout(numels, n_ranks, stage=2, align=align, bucket=8192)
    lay.bind_contributions([[x.view(torch.int16) for x in lst] for lst in lists])
    S, psi = lay.info.shard_elems, sum(numels)
    p0 = torch.zeros(n_ranks * S, device="cuda")
    p0[:psi] = torch.randn(psi, device="cuda") * 0.02
    gather = torch.zeros(n_ranks * S, dtype=torch.float16, device="cuda")
    flat = {k: torch.zeros(n_ranks * S, device="cuda") for k in "mv"}
    flat.update(p=p0.clone(), g=torch.zeros(n_ranks * S, dtype=torch.float16, device="cuda"), out=gather)
    groups = [0 if n > 200 else 1 for n in numels]
    sets = []
    for r in range(n_ranks):
        shard = {k: x[r * S:(r + 1) * S] for k, x in flat.items()}
        pieces = lay.rank_segments(r)
        cut = {}
        for sg in pieces:                                     # a tensor's pieces of one shard, joined over bucket fills
            lo, hi = cut.get(sg.tensor, (sg.shard_off, sg.shard_off))
            assert hi == sg.shard_off
            cut[sg.tensor] = (lo, hi + sg.len)
        view = {k: [x[lo:hi] for lo, hi in cut.values()] for k, x in shard.items()}
        sets.append(zp.TensorSet(p=view["p"], grads=view["g"], m=view["m"], v=view["v"], out=view["out"],
                                 groups=[groups[i] for i in cut]))
    whole = {k: [torch.zeros(n, device="cuda") for n in numels] for k in "mv"}
    off = np.concatenate([[0], np.cumsum(numels)])
    wp = [p0[a:b].clone() for a, b in zip(off, off[1:])]
    total = [(a.float() + b.float()).half() for a, b in zip(*lists)]
    ref = zp.TensorSet(p=wp, grads=total, m=whole["m"], v=whole["v"], groups=groups)
    control, other = zp.StepControl(), zp.StepControl()
    for _ in range(3):
        for r, s in enumerate(sets):
            for fill in range(lay.info.n_fills):
                lay.reduce_to_owner(fill, r, flat["g"][r * S:(r + 1) * S].view(torch.int16))
            s.grad_sumsq(control.sumsq, accumulate=r > 0)     # the all-reduce over ranks
        ref.grad_sumsq(other.sumsq)
        a, b = control.sumsq.item(), other.sumsq.item()
        assert abs(a - b) <= (psi + n_ranks) * 2.0 ** -53 * b
        other.sumsq.copy_(control.sumsq)
        for c in (control, other):
            c.begin(hparams(HP), max_norm=1.0)
        for s in sets:
            s.adamw_step(control)
        ref.adamw_step(other)
    torch.cuda.synchronize()
    assert control.grad_mult.item() < 1.0
    for k, want in (("p", wp), ("m", whole["m"]), ("v", whole["v"])):
        assert torch.equal(flat[k][:psi].view(torch.int32), torch.cat(want).view(torch.int32)), k
    assert torch.equal(gather[:psi], torch.cat(wp).half())
    for x in (gather, flat["p"], flat["m"], flat["v"]):       # padding stays as it was
        assert int(torch.count_nonzero(x[psi:])) == 0


@pytest.mark.parametrize("state", ["fp32", "mx"])
def test_training_together(state):
    """The operators as a program uses them: a linear model's gradients through autograd, norm, clip, step and the fp16
    copies feeding the next pass; p follows a 64-bit AdamW on the same gradients."""
    torch.manual_seed(0)
    n_in, n_out, batch = 96, 41, 64
    x = torch.randn(batch, n_in, device="cuda")
    y = x @ torch.randn(n_in, n_out, device="cuda") * 0.1
    p = [torch.randn(n_in, n_out, device="cuda") * 0.02, torch.zeros(n_out, device="cuda")]
    low = [q.half().requires_grad_() for q in p]
    for q in low:
        q.grad = torch.zeros_like(q)
    st = dict(m=[torch.zeros_like(q) for q in p], v=[torch.zeros_like(q) for q in p])
    if state == "mx":
        st = {k: [torch.zeros(q.shape, dtype=torch.float8_e4m3fn, device="cuda") for q in p] for k in "mv"}
        st.update({k: [torch.zeros(-(-q.numel() // 32), dtype=torch.uint8, device="cuda") for q in p] for k in ("m_scale", "v_scale")})
    s = zp.TensorSet(p=p, grads=[q.grad for q in low], out=[q.data for q in low], groups=[0, 1], **st)
    control = zp.StepControl(scale=64.0)
    ref = [q.double().cpu().numpy().ravel() for q in p]
    rm, rv = [np.zeros_like(q) for q in ref], [np.zeros_like(q) for q in ref]
    first = None
    for step in range(1, 21):
        for q in low:
            q.grad.zero_()
        loss = ((x.half() @ low[0] + low[1]).float() - y).square().mean()
        (loss * 64.0).backward()
        first = loss.item() if first is None else first
        g = [q.grad.double().cpu().numpy().ravel() for q in low]
        s.grad_sumsq(control.sumsq)
        control.begin(hparams(HP), max_norm=0.5)
        s.adamw_step(control)
        norm = np.sqrt(sum((k ** 2).sum() for k in g)) / 64.0
        assert abs(control.norm.item() - norm) <= 2.0 ** -22 * norm
        mult = min(1.0, 0.5 / norm) / 64.0
        for i in range(2):
            h = HP[i]
            rm[i] = h.beta1 * rm[i] + (1 - h.beta1) * g[i] * mult
            rv[i] = h.beta2 * rv[i] + (1 - h.beta2) * (g[i] * mult) ** 2
            ref[i] = ref[i] - (h.lr * h.weight_decay * ref[i] + h.lr / (1 - h.beta1 ** step) * rm[i] /
                               (np.sqrt(rv[i]) / np.sqrt(1 - h.beta2 ** step) + h.eps))
        assert torch.equal(low[0].detach(), p[0].half()) and torch.equal(low[1].detach(), p[1].half())
    assert control.t.item() == 20 and np.isfinite(loss.item())
    if state == "fp32":
        # a step is off by at most p_off, about 16 U of |update| <= 8 lr here and U |p|; the updates' own errors add up
        for q, r in zip(p, ref):
            assert np.abs(q.cpu().numpy().ravel() - r).max() <= 20 * (T.U * np.abs(r).max() + 16 * T.U * 8 * 2e-3) * 2


def test_kernel_timing_covers_the_set_calls():
    t = Twin([50001], "fp16", "fp16", "fp32", seed=40)
    control = zp.StepControl(scale=1024.0)
    zp.set_kernel_timing(True)
    try:
        t.set.grad_sumsq(control.sumsq)
        control.begin(hparams(HP))
        t.set.adamw_step(control)
        assert len(zp.kernel_times()) == 2 and all(0 < x < 100 for x in zp.kernel_times())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t.set.adamw_step(control)                         # captured: not timed
        assert len(zp.kernel_times()) == 2
        t.set.adamw_step(control)
        assert len(zp.kernel_times()) == 3
    finally:
        zp.set_kernel_timing(False)
