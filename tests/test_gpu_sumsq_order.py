"""The gradient norm's sum has one order, whatever addresses the tensors have."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from set_harness import GRAD, bits
from test_gpu_tensor_set import HP, hparams

pytestmark = pytest.mark.gpu


def moved(tensors, shift, rng):
    """Copies at odd starts of one buffer, `shift` elements in and up to 70 apart."""
    gaps = [shift] + [int(x) for x in rng.integers(0, 71, len(tensors) - 1)]
    buf = torch.zeros(sum(gaps) + sum(t.numel() for t in tensors), dtype=tensors[0].dtype, device="cuda")
    out, at = [], 0
    for t, gap in zip(tensors, gaps):
        at += gap
        out.append(buf[at: at + t.numel()])
        out[-1].copy_(t)
        at += t.numel()
    return out


@pytest.mark.parametrize("sizes", [[20000], [1024, 1, 1023, 1025], [5, 63, 64, 65, 500], [300, 70000, 2048, 17, 4096, 123457]])
@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_equal_values_at_any_address_give_equal_bits(grad, sizes):
    """Values of many magnitudes, so that a sum in another order is another number."""
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    g = [(torch.randn(n, generator=gen, device="cuda") * 10.0 ** (torch.rand(n, generator=gen, device="cuda") * 4 - 3)).to(GRAD[grad]) for n in sizes]
    rng = np.random.default_rng(3)
    want = None
    bound = zp.TensorSet(grads=moved(g, 0, rng))
    for shift in (0, 1, 2, 3, 7, 16, 17, 31, 32, 33, 48, 63, 64):
        here = moved(g, shift, rng)
        p, m, v = (moved([torch.zeros(n, device="cuda") for n in sizes], int(rng.integers(0, 70)), rng) for _ in range(3))
        bound.bind_grads(here)
        for s in (zp.TensorSet(grads=here), zp.TensorSet(p=p, grads=here, m=m, v=v), bound):
            out = torch.zeros((), dtype=torch.float64, device="cuda")
            s.grad_sumsq(out)
            got = out.view(torch.int64).item()
            want = got if want is None else want
            assert got == want, (shift, out.item())


@pytest.mark.parametrize("state", ["fp32", "mx"])
def test_clipped_runs_give_equal_bits_at_other_addresses(state):
    sizes = [50001, 300, 1024, 7, 20000]
    gen = torch.Generator(device="cuda").manual_seed(8)
    g0 = [torch.randn(n, generator=gen, device="cuda") * 10.0 ** (torch.rand(n, generator=gen, device="cuda") * 3 - 2) for n in sizes]
    p0 = [torch.randn(n, generator=gen, device="cuda") * 0.02 for n in sizes]

    def run(shift):
        rng = np.random.default_rng(shift)
        grads, p = moved(g0, shift, rng), moved(p0, shift // 2, rng)
        kinds = dict(m=torch.float32, v=torch.float32)
        if state == "mx":
            kinds = dict(m=torch.uint8, v=torch.uint8, m_scale=torch.uint8, v_scale=torch.uint8)
        st = {k: moved([torch.zeros(-(-n // 32) if "scale" in k else n, dtype=d, device="cuda") for n in sizes], shift // 3, rng)
              for k, d in kinds.items()}
        s, control = zp.TensorSet(p=p, grads=grads, groups=[0, 1, 0, 1, 0], seed=2, **st), zp.StepControl(scale=8.0)
        for k in range(4):
            s.grad_sumsq(control.sumsq)
            control.begin(hparams(HP), max_norm=0.5)
            s.adamw_step(control)
            s.bind_grads(moved(g0[:], shift + k, rng))
        return [bits(x) for x in (control.norm, control.grad_mult, *p, *[x for lst in st.values() for x in lst])]
    want = run(0)
    for shift in (1, 17, 32, 65):
        for a, b in zip(want, run(shift)):
            assert np.array_equal(a, b), shift
