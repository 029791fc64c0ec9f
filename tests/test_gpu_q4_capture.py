"""A mixed batch over a 4-bit cache captured on one stream while another runs
eagerly: both put their decode kernels on a side stream."""

import threading

import pytest
import torch

from test_gpu_q4 import Case, ok

pytestmark = pytest.mark.gpu


def test_an_eager_call_while_another_stream_captures():
    a = Case([(1, 900), (40, 77), (3, 333)], 8, 2, 128, seed=51)
    b = Case([(1, 70), (33, 33), (2, 400)], 16, 2, 64, seed=52)
    want_a, want_b = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        b.out.record_stream(other)
        with torch.cuda.stream(other):
            b.run()
        a.run()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want_b)
    for _ in range(3):
        a.out.fill_(5.0)
        g.replay()
        ok()
        assert torch.equal(a.out, want_a)


def test_one_thread_captures_while_another_runs():
    # many times over: neither's kernels end up in the other's graph or stream
    a = Case([(1, 900), (40, 77), (3, 333)], 8, 2, 128, seed=53)
    b = Case([(1, 70), (33, 33), (2, 400)], 16, 2, 64, seed=54)
    want_a, want_b = a.run().clone(), b.run().clone()
    outs = [torch.zeros_like(a.out) for _ in range(200)]
    torch.cuda.synchronize()
    failed = []

    def eager():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for o in outs:
                    a.run(out=o)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=eager)
    t.start()
    graphs = []
    for _ in range(20):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            b.run()
        graphs.append(g)
    t.join()
    assert not failed, failed
    for o in outs:
        assert torch.equal(o, want_a)
    for g in graphs:
        b.out.fill_(5.0)
        g.replay()
        ok()
        assert torch.equal(b.out, want_b)
