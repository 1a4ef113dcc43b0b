"""Workspaces and CUDA graphs: captured and eager calls share a buffer that is
zeroed once, outside the graphs; it lives as long as a graph that uses it, and
no longer; status bits stay until they are read."""
import ctypes
import gc
import time

import pytest
import torch

from compressed_sparse_attention_15_b200 import _lib, ops
from compressed_sparse_attention_15_b200.build import build

gpu = pytest.mark.gpu
N, K = 700, 16


def _inputs(dev, Q=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(Q, N, generator=g).to(dev), torch.full((Q,), N, dtype=torch.int32, device=dev)


def _capture(f, pool=None):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, pool=pool):
        out = f()
    return graph, out


@gpu
def test_the_calls_of_a_capture_share_one_buffer_that_the_graph_does_not_fill(cuda_device):
    class Recorded(ops.Workspace):
        def get(self, nbytes):
            w = super().get(nbytes)
            given.append(w.data_ptr())
            return w

    given, ws = [], Recorded(cuda_device)
    scores, n = _inputs(cuda_device)
    want = ops.topk(scores, n, K)
    ops.topk(scores, n, K, ws=ops.Workspace(cuda_device))  # (kernel attributes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws.get(1 << 20)
        outs = [ops.topk(scores, n, K, ws=ws) for _ in range(3)]
    assert len(given) == 4 and len(set(given)) == 1
    assert torch.all(ws.buf == 0), "zeroed before any replay"
    ws.buf[-256:] = 7
    graph.replay()
    graph.replay()
    assert torch.all(ws.buf[-256:] == 7), "the replays fill nothing"
    eager = ops.topk(scores, n, K, ws=ws)
    assert len(set(given)) == 1, "an eager call takes the same buffer"
    assert all(torch.equal(o, want) for o in (*outs, eager)) and ws.status() == 0


@gpu
def test_status_before_the_first_replay_is_clean(cuda_device):
    scores, n = _inputs(cuda_device)
    ops.topk(scores, n, K)
    # a graph whose memory pool holds only ones
    first, ones = _capture(lambda: [torch.full((1 << 18,), 255, dtype=torch.uint8, device=cuda_device) for _ in range(8)])
    first.replay()
    torch.cuda.synchronize()
    pool = first.pool()
    del ones
    ws = ops.Workspace(cuda_device)
    graph, out = _capture(lambda: ops.topk(scores, n, K, ws=ws), pool)
    assert ws.status() == 0
    graph.replay()
    assert ws.status() == 0 and torch.equal(out, ops.topk(scores, n, K))


@gpu
@pytest.mark.parametrize("warm", [False, True])
def test_a_fault_of_an_earlier_replay_is_reported(cuda_device, warm):
    scores, n = _inputs(cuda_device)
    ws = ops.Workspace(cuda_device)
    ops.topk(scores, n, K, ws=ws if warm else None)
    graph, _ = _capture(lambda: ops.topk(scores, n, K, ws=ws))
    for bad in (True, False, False):
        n.fill_(N + 1 if bad else N)
        graph.replay()
    assert ws.status() == 1, "the first replay's count was outside the list"
    graph.replay()
    assert ws.status() == 0


@gpu
@pytest.mark.parametrize("warm", [False, True])
def test_a_graph_keeps_the_buffer_of_a_workspace_that_is_gone(cuda_device, warm):
    dev = cuda_device
    scores, n = _inputs(dev, Q=160)  # (lists in segments through the workspace)
    want = ops.topk(scores, n, K)
    ws = ops.Workspace(dev)
    size = 1 << 22
    if warm:
        ws.get(size)
        ops.topk(scores, n, K, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws.get(size)
        out = ops.topk(scores, n, K, ws=ws)
    buffer = ws.buf.data_ptr()
    del ws
    gc.collect()
    others = [torch.full((size,), 255, dtype=torch.uint8, device=dev) for _ in range(16)]
    assert buffer not in [o.data_ptr() for o in others]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.all(o == 255) for o in others)


@gpu
def test_buffers_go_when_their_graphs_are_gone(cuda_device):
    scores, n = _inputs(cuda_device)
    ops.topk(scores, n, K)
    ws = ops.Workspace(cuda_device)
    gc.collect()

    def held():
        return sum(ws.status() == 0 and b.numel() for b in (ws.buf, *ws._older))

    def sizes(graphs):
        for i in range(4):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ws.get((i + 1) << 20)
                ops.topk(scores, n, K, ws=ws)
                ops.topk(scores, n, K, ws=ws)
            graphs.append(graph)

    graphs = []
    sizes(graphs)
    assert held() == 10 << 20, "every graph's buffer is there"
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    del g
    graphs[1:3] = []
    gc.collect()
    for _ in range(200):  # (the driver tells of a graph's end from a thread of its own)
        if held() == 5 << 20:
            break
        time.sleep(0.02)
    assert held() == 5 << 20, "the first graph's buffer and the present one"
    del ws
    graphs.clear()
    gc.collect()
    for _ in range(200):
        ops._drop_ended()
        if not ops._captured:
            break
        time.sleep(0.02)
    assert not ops._captured


@gpu
def test_growth_inside_a_capture_and_a_capture_that_fails(cuda_device):
    scores, n = _inputs(cuda_device, Q=160, seed=4)
    few, m = scores[:2].contiguous(), n[:2].contiguous()
    want = ops.topk(few, m, K), ops.topk(scores, n, K)
    ws = ops.Workspace(cuda_device)
    graph, outs = _capture(lambda: (ops.topk(few, m, K, ws=ws), ops.topk(scores, n, K, ws=ws)))
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    with pytest.raises(RuntimeError, match="on purpose"):
        _capture(lambda: (ws.get(ws.buf.numel() + 1), exec("raise RuntimeError('on purpose')")))
    assert torch.equal(ops.topk(scores, n, K, ws=ws), want[1])
    graph.replay()
    assert ws.status() == 0 and all(torch.equal(o, w) for o, w in zip(outs, want))


@gpu
def test_calls_without_a_workspace_are_captured(cuda_device):
    scores, n = _inputs(cuda_device, Q=160, seed=5)
    want = ops.topk(scores, n, K)
    before = len(ops._captured)
    graph, outs = _capture(lambda: [ops.topk(scores, n, K) for _ in range(3)])
    other = torch.full((1 << 22,), 255, dtype=torch.uint8, device=cuda_device)
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(o, want) for o in outs) and torch.all(other == 255) and len(ops._captured) == before


def test_entry_points_refuse_bad_arguments():
    build()
    L = _lib.lib()
    number, mark = ctypes.c_ulonglong(0), ctypes.c_void_p()
    assert L.csa_graph_mark(None, None, ctypes.byref(mark)) == 1
    assert L.csa_graph_mark(None, ctypes.byref(number), ctypes.byref(mark)) != 0  # no capture (or no device)
    assert not mark.value
    assert L.csa_graph_mark_ended(None) == 0
    for mode in (-1, 3):
        assert L.csa_exchange_capture_mode(ctypes.byref(ctypes.c_int(mode))) == 1
    assert L.csa_exchange_capture_mode(None) == 1
