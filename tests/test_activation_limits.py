"""CPU checks of sizes that no launch takes: empty or broadcast matrices whose row numbers alone are huge."""

import pytest

from test_activations_host import BASE, BF16, FP32, GAP, OVF, call, cpu_only, sound, zp   # noqa: F401


@pytest.mark.parametrize("T", [(1 << 40) + 1, (1 << 56) + 1, (1 << 63) - 1])
def test_tokens_of_a_broadcast_gradient(call, T):   # noqa: F811
    """One row of dy for all tokens, of inputs of width 0: nothing bounds T but the limit itself, behind which the size of
    the workspace is given as 0."""
    m, k = call.matrix, call.kept
    args = dict(dy=m(0, T, 64, stride=0), x=k(1, T, 0, code=0), dw=m(2, 64, 0, data=0, type=FP32))
    assert call.zp.lib.zero_weight_grad_work_bytes(T, 64, 0, BF16) == 0
    for work in (None, BASE + 6 * GAP):
        assert call.weight(**args, bias=BASE + 3 * GAP, work=work) == OVF
    assert call.weight(**args) == OVF


def test_the_most_tokens_pass(call, cpu_only):   # noqa: F811
    m, k, T = call.matrix, call.kept, 1 << 40
    assert call.zp.lib.zero_weight_grad_work_bytes(T, 64, 0, BF16) > 0
    sound(call.weight(dy=m(0, T, 64, stride=0), x=k(1, T, 0, code=0), dw=m(2, 64, 0, data=0, type=FP32), bias=BASE + 3 * GAP, work=BASE + 6 * GAP))
    sound(call.lookup(table=m(0, 100, 0), out=m(2, T, 0)))


@pytest.mark.parametrize("n", [(1 << 40) + 1, (1 << 61) + 1, (1 << 63) - 1])
def test_tokens_of_rows_of_width_0(call, n):   # noqa: F811
    m = call.matrix
    assert call.lookup(table=m(0, 100, 0), out=m(2, n, 0)) == OVF
    assert call.egrad(dy=m(0, n, 0), dt=m(2, 100, 0)) == OVF
