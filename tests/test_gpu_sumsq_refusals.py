"""What the sum of squares refuses to be written over, before anything is launched."""

import pytest
import torch

import sharded_zero_partition_amd as zp

pytestmark = pytest.mark.gpu
INVALID = -1


def test_sum_and_workspace_in_the_set_s_own_arrays():
    n = 300_000
    g = torch.ones(n, device="cuda")
    mem = torch.zeros(n + 64, device="cuda")
    p, m, v = mem[:n], torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    s = zp.TensorSet(p=[p], grads=[g], m=[m], v=[v])
    bytes_ = zp.lib.zero_grad_sumsq_work_bytes(s._h)
    assert bytes_ > 0 and bytes_ % 8 == 0
    work = torch.zeros(bytes_ // 8 + 2, dtype=torch.float64, device="cuda")
    out = torch.zeros(2, dtype=torch.float64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(sumsq, w):
        return zp.lib.zero_grad_sumsq(s._h, sumsq, 0, w, stream)
    w, o = work.data_ptr(), out.data_ptr()
    for x in (p, m, v):
        for at in (x.data_ptr(), x.data_ptr() + 4 * n - 8):
            assert call(at, w) == INVALID
            assert call(o, at) == INVALID
    assert call(w, w) == INVALID and call(w + bytes_ - 8, w) == INVALID      # the sum inside the workspace
    torch.cuda.synchronize()
    for x in (mem, m, v, work, out):
        assert int(torch.count_nonzero(x)) == 0
    # beside them is fine: the workspace's end, and the eight bytes behind p
    for at in (w + bytes_, mem.data_ptr() + 4 * n):
        assert call(at, w) == 0
    torch.cuda.synchronize()
    assert work[bytes_ // 8].item() == n and mem[n:n + 2].view(torch.float64).item() == n
    assert int(torch.count_nonzero(p)) == 0


def test_a_sum_by_one_block_needs_no_workspace():
    g, p = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    s = zp.TensorSet(p=[p], grads=[g], m=[torch.zeros(64, device="cuda")], v=[torch.zeros(64, device="cuda")])
    assert zp.lib.zero_grad_sumsq_work_bytes(s._h) == 0
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for work in (None, out.data_ptr(), p.data_ptr()):                       # not used
        assert zp.lib.zero_grad_sumsq(s._h, out.data_ptr(), 0, work, stream) == 0
    assert zp.lib.zero_grad_sumsq(s._h, p.data_ptr(), 0, None, stream) == INVALID
    assert out.item() == 64.0
