"""Workspaces and CUDA graphs: captured and eager calls share a buffer that is
zeroed once, outside the graphs; one that is first needed inside a capture lives
as long as its graph; status bits stay until they are read."""
import ctypes
import gc

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
def test_a_graph_keeps_the_buffer_that_was_made_in_its_capture(cuda_device):
    dev = cuda_device
    scores, n = _inputs(dev, Q=160)
    want = ops.topk(scores, n, K)
    ws = ops.Workspace(dev)
    size = 1 << 22
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws.get(size)
        out = ops.topk(scores, n, K, ws=ws)
    del ws
    gc.collect()
    others = [torch.full((size,), 255, dtype=torch.uint8, device=dev) for _ in range(16)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.all(o == 255) for o in others)


@gpu
def test_capturing_again_keeps_no_further_buffers(cuda_device):
    scores, n = _inputs(cuda_device)
    want = ops.topk(scores, n, K)
    for warm in (False, True):
        ws = ops.Workspace(cuda_device)
        if warm:
            ws.get(1 << 20)
        graphs = []
        for _ in range(5):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ws.get(1 << 20)
                out = ops.topk(scores, n, K, ws=ws)
            graphs.append((graph, out))
        assert ws.buf.numel() == 1 << 20 and not ws._older
        address = ws.buf.data_ptr()
        for graph, out in graphs:
            graph.replay()
            assert torch.equal(out, want)
        # growth in small steps, a graph after each: a buffer is at most half as large again as the largest call, and
        # what stays is less than twice that (1 + 1.5 + 2.25 + 3.375 of 5.06 MB here)
        for i in range(40):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                ws.get((1 << 20) + (i << 16))
                out = ops.topk(scores, n, K, ws=ws)
            graphs.append((graph, out))
        assert ws._older[0].data_ptr() == address
        assert ws.buf.numel() <= 1.5 * ((1 << 20) + (39 << 16))
        assert sum(b.numel() for b in ws._older) < 2 * ws.buf.numel()
        n.fill_(N + 1)
        graphs[0][0].replay()
        n.fill_(N)
        for graph, out in graphs:
            graph.replay()
            assert torch.equal(out, want)
        assert ws.status() == 1, "a fault of the graph with the oldest buffer"
        assert ws.status() == 0


@gpu
def test_new_workspaces_in_captures_on_every_stream(cuda_device):
    # torch hands out 32 streams in turn, for captures too
    scores, n = _inputs(cuda_device, Q=2)
    want = ops.topk(scores, n, K)
    kept = []
    for i in range(70):
        ws = ops.Workspace(cuda_device)
        stream = torch.cuda.Stream() if i % 2 else None
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = ops.topk(scores, n, K, ws=ws)
        kept.append((ws, graph, out))
    for ws, graph, out in kept:
        graph.replay()
        assert torch.equal(out, want) and ws.status() == 0


@gpu
def test_nothing_else_writes_to_a_buffer_made_in_a_capture(cuda_device):
    # blocks that the capture has given back before, of every size and of another workspace, are not taken for it
    scores, n = _inputs(cuda_device, Q=160, seed=7)
    want = ops.topk(scores, n, K)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for size in (256, 1 << 12, 1 << 18, 1 << 21, 1 << 23):
            ones = torch.full((size,), 255, dtype=torch.uint8, device=cuda_device)
            del ones
        first = ops.Workspace(cuda_device)
        first.get(1 << 21)
        ops.topk(scores, n, K, ws=first)
        first.get(1 << 21).fill_(255)
        del first
        gc.collect()
        ws = ops.Workspace(cuda_device)
        out = ops.topk(scores, n, K, ws=ws)
        ws.get(1 << 21)[-256:].fill_(3)
    for _ in range(2):
        graph.replay()
        assert torch.equal(out, want) and ws.status() == 0
        assert torch.all(ws.buf[16:256] == 0) and torch.all(ws.buf[-256:] == 3)


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
    graph, outs = _capture(lambda: [ops.topk(scores, n, K) for _ in range(3)])
    other = torch.full((1 << 22,), 255, dtype=torch.uint8, device=cuda_device)
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(o, want) for o in outs) and torch.all(other == 255)


def test_entry_points_refuse_bad_arguments():
    build()
    L = _lib.lib()
    assert L.csa_stream_create(None) == 1
    for mode in (-1, 3):
        assert L.csa_exchange_capture_mode(ctypes.byref(ctypes.c_int(mode))) == 1
    assert L.csa_exchange_capture_mode(None) == 1
