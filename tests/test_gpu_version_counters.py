"""Steps and conversions are in-place writes that autograd knows of."""

import pytest
import torch

import sharded_zero_partition_amd as zp

pytestmark = pytest.mark.gpu

HP = [zp.AdamHParams(1e-2, 0.9, 0.999, 1e-8, 0.0)]


def made(p, out=None, **kw):
    z = lambda: [torch.zeros(x.numel(), device="cuda") for x in p]   # noqa: E731
    return zp.TensorSet(p=p, grads=[torch.ones(x.numel(), device="cuda") for x in p], m=z(), v=z(), out=out, **kw)


def step(s):
    control = zp.StepControl()
    control.begin(HP, check=False)
    s.adamw_step(control)


@pytest.mark.parametrize("which", ["p", "out", "view"])
def test_a_backward_pass_through_overwritten_weights_is_an_error(which):
    """A product saves its weight for the other operand's gradient; a step between it and the backward pass changes that
    weight."""
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    flat = torch.randn(100, device="cuda")
    p = torch.randn(64, device="cuda") if which != "view" else flat[3:67]
    if which == "out":
        w = torch.randn(64, device="cuda").half()
        s = made([p], out=[w])
        y = (x.half() @ w.view(8, 8)).float().sum()
    else:
        w = (flat if which == "view" else p).requires_grad_(which == "view")
        s = made([p.detach()])
        y = (x @ (w[3:67] if which == "view" else w).view(8, 8)).sum()
    step(s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_counters_of_tensors_and_views():
    flat, own = torch.randn(300, device="cuda"), torch.randn(40, device="cuda")
    other = torch.randn(40, device="cuda")
    s = made([flat[:100], flat[100:300], own])
    before = flat._version, own._version, other._version
    step(s)
    assert flat._version > before[0] and own._version > before[1] and other._version == before[2]
    assert len(s._counted["p", "out"]) == 2                   # one for the flat buffer's two views


def test_a_conversion_raises_the_states_counters():
    f = [torch.rand(64, device="cuda") for _ in range(2)]
    c = [torch.zeros(64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    wide, small = zp.TensorSet(m=f[:1], v=f[1:]), zp.TensorSet(m=c[:1], v=c[1:], m_scale=sc[:1], v_scale=sc[1:])
    at = [x._version for x in f + c]
    small.states_from(wide)
    assert [x._version > v for x, v in zip(f + c, at)] == [False, False, True, True]


def test_leaves_tensors_of_inference_mode_and_empty_sets_pass():
    with torch.inference_mode():
        p = [torch.randn(10, device="cuda"), torch.randn(5, device="cuda")]
    step(made(p))
    leaf = torch.randn(10, device="cuda", requires_grad=True)
    with torch.no_grad():
        step(made([leaf]))
    step(made([leaf.detach()]))
    assert leaf._version == 2
    step(made([torch.zeros(0, device="cuda")]))
