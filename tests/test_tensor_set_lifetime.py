"""When tensor sets are freed: a refused free is tried again, and captures of this thread or another go on."""

import os
import threading

import pytest
import torch

from sharded_zero_partition_amd import build as zbuild

if not os.path.exists(zbuild.LIB):
    zbuild.build()
import sharded_zero_partition_amd as zp  # noqa: E402


def handle(monkeypatch, answers):
    """A set without a device, whose frees answer as told."""
    freed = []

    def destroy(h):
        rc = answers.pop(0) if answers else 0
        if rc == 0:
            freed.append(h)
        return rc
    monkeypatch.setattr(zp.binding.lib, "zero_tensor_set_destroy", destroy)
    monkeypatch.setattr(zp.TensorSet, "_late", [])
    s = zp.TensorSet.__new__(zp.TensorSet)
    s._h = 7
    return s, freed


def test_a_refused_free_is_tried_again(monkeypatch):
    s, freed = handle(monkeypatch, [-5, -5, 0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    s.close()
    assert freed == [] and zp.TensorSet._late == [7]
    s.close()
    assert freed == [] and zp.TensorSet._late == [7]
    zp.TensorSet._free_late()                                 # as the next set does
    assert freed == [7] and zp.TensorSet._late == []
    s.close()
    assert freed == [7]


def test_a_free_in_this_thread_s_capture_waits(monkeypatch):
    s, freed = handle(monkeypatch, [])
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    s.close()
    assert freed == []
    capturing[0] = False
    zp.TensorSet._free_late()
    assert freed == [7]


@pytest.mark.gpu
@pytest.mark.parametrize("default_stream", [False, True])
def test_sets_come_and_go_in_one_thread_while_another_captures(default_stream):
    """In torch's default mode, in which a plain free or a wait of any thread is refused while a stream is captured."""
    g = torch.randn(200_000, device="cuda")
    other = [torch.ones(5000, device="cuda") for _ in range(3)]
    s, out = zp.TensorSet(grads=[g]), torch.zeros((), dtype=torch.float64, device="cuda")
    s.grad_sumsq(out)
    want, errors, sums = out.item(), [], torch.zeros(8, dtype=torch.float64, device="cuda")
    begun, done = threading.Event(), threading.Event()
    st = torch.cuda.default_stream() if default_stream else torch.cuda.Stream()

    def work():
        try:
            assert begun.wait(60)
            with torch.cuda.stream(st):
                for k in range(4):
                    t = zp.TensorSet(grads=other[:1])
                    t.grad_sumsq(sums[2 * k])
                    t.bind_grads(other[1:2])
                    t.grad_sumsq(sums[2 * k + 1])
                    t.close()
                    assert not zp.TensorSet._late
        except BaseException as e:                            # noqa: BLE001
            errors.append(e)
        finally:
            done.set()

    th = threading.Thread(target=work)
    th.start()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.grad_sumsq(out)
        begun.set()
        assert done.wait(60)
        s.grad_sumsq(out, accumulate=True)
    th.join()
    assert not errors, errors
    st.synchronize()
    assert sums.tolist() == [5000.0] * 8
    for _ in range(3):
        out.fill_(-1.0)
        graph.replay()
        assert out.item() == 2 * want


@pytest.mark.gpu
def test_a_set_deferred_in_a_capture_goes_with_the_next_one_made():
    g = torch.ones(100, device="cuda")
    s, gone = zp.TensorSet(grads=[g]), zp.TensorSet(grads=[g])
    out = torch.zeros((), dtype=torch.float64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.grad_sumsq(out)
        gone.close()
    assert len(zp.TensorSet._late) == 1
    made = zp.TensorSet(grads=[g])
    assert not zp.TensorSet._late and made._h
    for _ in range(3):
        graph.replay()
        assert out.item() == 100.0


@pytest.mark.gpu
def test_the_abi_frees_a_set_while_its_own_thread_captures():
    """As a C program may; the binding waits for the capture's end."""
    g = torch.ones(100, device="cuda")
    s, gone = zp.TensorSet(grads=[g]), zp.TensorSet(grads=[g])
    h, gone._h = gone._h, None
    out = torch.zeros((), dtype=torch.float64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.grad_sumsq(out)
        assert zp.lib.zero_tensor_set_destroy(h) == 0
        s.grad_sumsq(out, accumulate=True)
    for _ in range(3):
        graph.replay()
        assert out.item() == 200.0
