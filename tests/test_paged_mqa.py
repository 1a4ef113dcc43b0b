"""csa_paged_sparse_mqa / csa_paged_hca_mqa vs the formula in 64 bits over the
values that the cache holds (paged_reference.check_attention has the bound)."""
import ctypes
import math
import weakref

import pytest
import torch

import paged_reference as R
from compressed_sparse_attention_15_b200 import _lib, ops
from compressed_sparse_attention_15_b200.build import build

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _inputs(seed, Q, B, H, D, N, page, W, fmt, dtype, qscale=1.0):
    g = torch.Generator().manual_seed(seed)
    pages, scales, table = R.make_cache(seed, B, N, page, D, fmt, dtype)
    T = W + 21
    c = dict(q=(torch.randn(Q, H, D, generator=g) * qscale).to(dtype), pages=pages, scales=scales, table=table,
             sink=torch.randn(H, generator=g), kv_win=None, win_end=None, g=g)
    if W:
        c["kv_win"] = torch.randn(B, T, D, generator=g).to(dtype)
        c["win_end"] = torch.tensor([[T - 1, 0, W // 2, W, 7 % T][i % 5] for i in range(Q)], dtype=torch.int32)
    return c


def _selection(g, Q, N, k):
    """Ragged selections: full, half, empty, one entry; unused slots last."""
    idx = torch.full((Q, k), -1, dtype=torch.int32)
    for i in range(Q):
        m = min([k, k // 2, 0, 1, k][i % 5], N)
        idx[i, :m] = torch.randperm(N, generator=g)[:m].sort().values.to(torch.int32)
    return idx


def _run(dev, c, W, scale, n_cmp=None, idx=None, ws=None, **kw):
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    f, rows = (ops.paged_hca_mqa, n_cmp) if idx is None else (ops.paged_sparse_mqa, idx)
    return f(d(c["q"]), d(c["pages"]), d(c["scales"]), d(c["table"]), d(rows), d(c["kv_win"]), d(c["win_end"]), d(c["sink"]),
             scale, W, ws=ws, **kw)


def _refs(c, W, scale, n_cmp=None, idx=None, q_per_seq=None):
    vals = R.values(c["pages"], c["scales"])
    Q, B = c["q"].shape[0], c["table"].shape[0]
    per = q_per_seq or Q // B
    refs = []
    for i in range(Q):
        b = i // per
        e = torch.arange(int(n_cmp[i])) if idx is None else idx[i][idx[i] >= 0]
        rows = R.entries(vals, c["table"], b, e)
        if W:
            end = int(c["win_end"][i])
            rows = torch.cat([rows, c["kv_win"][b, max(0, end - W + 1):end + 1].double()])
        refs.append(R.attend(c["q"][i], rows, c["sink"], scale))
    return refs


SHAPES = [
    # Q, B, H, D, N, page, W, k
    (5, 5, 64, 512, 700, 64, 128, 512),
    (3, 1, 64, 512, 333, 48, 128, 200),
    (5, 5, 64, 512, 64, 16, 0, 64),
    (4, 2, 128, 512, 300, 64, 130, 300),
    (5, 5, 1, 512, 1000, 17, 1, 100),
    (6, 3, 37, 256, 200, 1, 33, 77),
    (5, 5, 100, 384, 129, 256, 64, 129),
    (10, 5, 16, 128, 90, 64, 2, 65),
    (2, 2, 64, 512, 3000, 128, 128, 1024),
    (5, 1, 3, 64, 70, 7, 5, 31),
    (5, 5, 2, 16, 1500, 64, 9, 40),
    (160, 160, 64, 512, 70, 64, 3, 7),
]


@gpu
@pytest.mark.parametrize("fmt,dtype", [("int4", BF16), ("rows", BF16), ("int4", F32), ("rows", F32)])
@pytest.mark.parametrize("Q,B,H,D,N,page,W,k", SHAPES)
def test_dense(cuda_device, Q, B, H, D, N, page, W, k, fmt, dtype):
    c = _inputs(Q + H + N, Q, B, H, D, N, page, W, fmt, dtype)
    n_cmp = torch.tensor([[N, 0, 1, N // 3, N - 1][i % 5] for i in range(Q)], dtype=torch.int32)
    ws = ops.Workspace(cuda_device)
    out = _run(cuda_device, c, W, D ** -0.5, n_cmp=n_cmp, ws=ws)
    assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, n_cmp=n_cmp), dtype, N + W)


@gpu
@pytest.mark.parametrize("fmt,dtype", [("int4", BF16), ("rows", BF16), ("int4", F32), ("rows", F32)])
@pytest.mark.parametrize("Q,B,H,D,N,page,W,k", SHAPES)
def test_sparse(cuda_device, Q, B, H, D, N, page, W, k, fmt, dtype):
    c = _inputs(Q + H + N + 1, Q, B, H, D, N, page, W, fmt, dtype)
    idx = _selection(c["g"], Q, N, k)
    ws = ops.Workspace(cuda_device)
    out = _run(cuda_device, c, W, D ** -0.5, idx=idx, ws=ws)
    assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, idx=idx), dtype, k + W)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [512, 40])
def test_no_rows_odd_sinks_and_steep_logits(cuda_device, D, dtype):
    fmt = "rows"
    c = _inputs(3, 4, 2, 64, D, 300, 64, 0, fmt, dtype, qscale=30.0)  # logits of several hundreds: the maximum moves
    c["sink"][:3] = torch.tensor([-math.inf, 1e4, -1e4])
    n_cmp = torch.tensor([0, 300, 1, 299], dtype=torch.int32)
    out = _run(cuda_device, c, 0, D ** -0.5, n_cmp=n_cmp)
    assert torch.all(out[0] == 0)
    refs = _refs(c, 0, D ** -0.5, n_cmp=n_cmp)
    R.check_attention(out, refs, dtype, 300)
    idx = torch.full((4, 9), -1, dtype=torch.int32)
    assert torch.all(_run(cuda_device, c, 0, D ** -0.5, idx=idx) == 0)


@gpu
@pytest.mark.parametrize("fmt,dtype", [("int4", BF16), ("rows", BF16), ("rows", F32)])
def test_what_is_not_attended_has_no_effect(cuda_device, fmt, dtype):
    # NaN in every entry past the count or off the list, in rows outside the window, and in a page of no sequence
    Q, B, H, D, N, page, W = 4, 2, 64, 512, 200, 48, 40
    c = _inputs(8, Q, B, H, D, N, page, W, fmt, dtype)
    n_cmp = torch.tensor([150, 0, 77, 64], dtype=torch.int32)
    idx = _selection(c["g"], Q, N, 90)
    keep_dense, keep_sparse = (torch.zeros(B, N, dtype=torch.bool) for _ in range(2))
    for i in range(Q):
        keep_dense[i // 2, :int(n_cmp[i])] = True
        keep_sparse[i // 2, idx[i][idx[i] >= 0].long()] = True
    seen = torch.zeros(B, c["kv_win"].shape[1], dtype=torch.bool)
    for i in range(Q):
        e = int(c["win_end"][i])
        seen[i // 2, max(0, e - W + 1):e + 1] = True
    for keep, kw in ((keep_dense, dict(n_cmp=n_cmp)), (keep_sparse, dict(idx=idx))):
        refs = _refs(c, W, D ** -0.5, **kw)
        live = torch.zeros(c["pages"].shape[:2], dtype=torch.bool)
        for b in range(B):
            e = keep[b].nonzero()[:, 0]
            live[c["table"][b].long()[e // page], e % page] = True
        p = dict(c, pages=c["pages"].clone(), kv_win=c["kv_win"].clone())
        if fmt == "int4":
            s = c["scales"].view(torch.uint8).clone()
            s[~live] = 0x7F
            p["scales"] = s
        else:
            p["pages"][~live] = math.nan
        p["kv_win"][~seen] = math.nan
        R.check_attention(_run(cuda_device, p, W, D ** -0.5, **kw), refs, dtype, N + W)


@gpu
@pytest.mark.parametrize("D,H", [(512, 64), (64, 4)])
def test_bad_device_values_are_skipped_and_reported(cuda_device, D, H):
    Q, B, N, page, W = 4, 2, 128, 64, 16
    c = _inputs(11, Q, B, H, D, N, page, W, "int4", BF16)
    n_cmp = torch.tensor([N + 1, -1, 5, N], dtype=torch.int32)
    ws = ops.Workspace(cuda_device)
    out = _run(cuda_device, c, W, 0.05, n_cmp=n_cmp, ws=ws)
    assert ws.status() == 1
    R.check_attention(out, _refs(c, W, 0.05, n_cmp=n_cmp.clamp(0, N)), BF16, N + W)
    idx = torch.tensor([[0, 5, N, -1], [-2, 3, 4, 5], [1, 1, 2, -1], [-1, -1, -1, 9]], dtype=torch.int32)
    ok = torch.where((idx < 0) | (idx >= N), -1, idx)
    out = _run(cuda_device, c, W, 0.05, idx=idx, ws=ws)
    assert ws.status() == 2
    R.check_attention(out, _refs(c, W, 0.05, idx=ok), BF16, N + W)  # (an entry given twice counts twice)
    bad = dict(c, win_end=torch.tensor([-1, c["kv_win"].shape[1], 3, 4], dtype=torch.int32))
    out = _run(cuda_device, bad, W, 0.05, idx=ok, ws=ws)
    assert ws.status() == 4
    bad["win_end"] = bad["win_end"].clamp(0, c["kv_win"].shape[1] - 1)
    R.check_attention(out, _refs(bad, W, 0.05, idx=ok), BF16, N + W)
    # a page outside the pool: its entries are skipped
    bad = dict(c, table=c["table"].clone())
    bad["table"][1, 0] = -7
    out = _run(cuda_device, bad, W, 0.05, n_cmp=torch.full((Q,), N, dtype=torch.int32), ws=ws)
    assert ws.status() == 16
    rest = torch.full((Q, N), -1, dtype=torch.int32)
    rest[:2] = torch.arange(N)
    rest[2:, :64] = torch.arange(64, N)
    R.check_attention(out, _refs(c, W, 0.05, idx=rest), BF16, N + W)


@gpu
@pytest.mark.parametrize("H,D", [(64, 512), (5, 64)])
def test_capture_side_stream_and_a_shared_workspace(cuda_device, H, D):
    Q, N, W = 2, 400, 30
    c = _inputs(21, Q, Q, H, D, N, 64, W, "int4", BF16)
    dev = cuda_device
    ws = ops.Workspace(dev)
    d = {n: (t.to(dev) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    n_cmp = torch.tensor([N, 9], dtype=torch.int32, device=dev)
    idx = torch.full((Q, 64), -1, dtype=torch.int32, device=dev)
    idx[0, :64] = torch.arange(64) * 5
    args = (d["q"], d["pages"], d["scales"], d["table"])
    tail = (d["kv_win"], d["win_end"], d["sink"], 0.05, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for f, rows in ((ops.paged_hca_mqa, n_cmp), (ops.paged_sparse_mqa, idx)):
            f(*args, rows, *tail, ws=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(f(*args, rows, *tail, ws=ws))
            graphs.append(g)
        q2 = torch.randn(c["q"].shape, generator=c["g"]).to(BF16)
        d["q"].copy_(q2)
        n_cmp.copy_(torch.tensor([17, N], dtype=torch.int32))
        for _ in range(3):
            for g in graphs:
                g.replay()
    side.synchronize()
    assert ws.status() == 0
    c["q"] = q2
    R.check_attention(outs[0], _refs(c, W, 0.05, n_cmp=n_cmp.cpu()), BF16, N + W)
    R.check_attention(outs[1], _refs(c, W, 0.05, idx=idx.cpu()), BF16, N + W)


@gpu
def test_same_results_every_time_and_equal_to_the_unpaged_path(cuda_device):
    # bf16 pages in order hold what hca_mqa takes as one tensor
    Q, N, W, H, D = 4, 512, 128, 64, 512
    c = _inputs(31, Q, Q, H, D, N, 64, W, "rows", BF16)
    n_cmp = torch.tensor([512, 3, 0, 129], dtype=torch.int32)
    out = _run(cuda_device, c, W, D ** -0.5, n_cmp=n_cmp)
    for _ in range(3):
        assert torch.equal(out, _run(cuda_device, c, W, D ** -0.5, n_cmp=n_cmp))
    dev = cuda_device
    kv = torch.stack([R.entries(c["pages"], c["table"], b, torch.arange(N)) for b in range(Q)])
    flat = ops.hca_mqa(c["q"].to(dev), kv.to(dev), n_cmp.to(dev), c["kv_win"].to(dev), c["win_end"].to(dev),
                       c["sink"].to(dev), D ** -0.5, W)
    R.check_attention(flat, _refs(c, W, D ** -0.5, n_cmp=n_cmp), BF16, N + W)


@gpu
@pytest.mark.parametrize("k", [3, 200])
def test_decode_steps_over_a_growing_cache(cuda_device, k):
    # the operators together: norm, append, selection, attention, read-back, four decode steps
    dev, B, H, D, page = cuda_device, 3, 64, 512, 16
    g = torch.Generator().manual_seed(5)
    pages, scales, table = (t.to(dev) for t in R.make_cache(5, B, 64, page, D, "int4", BF16))
    w = torch.ones(D, device=dev)
    sink = torch.randn(H, generator=g)
    ws = ops.Workspace(dev)
    for step in range(4):
        x = torch.randn(B, 5, D, generator=g).to(BF16).to(dev)
        kv, = ops.add_rmsnorm(x, w)
        e0 = torch.full((B,), 5 * step, dtype=torch.int32, device=dev)
        ops.paged_append(kv, pages, scales, table, e0, rope=(64, 160000.0, None, 4), ws=ws)
        n = 5 * step + 5
        q = torch.randn(B, H, D, generator=g).to(BF16)
        scores = torch.randn(B, 64, generator=g).to(dev)
        idx = ops.topk(scores, torch.full((B,), n, dtype=torch.int32, device=dev), k, ws=ws)
        win = torch.randn(B, 12, D, generator=g).to(BF16)
        end = torch.tensor([11, 4, 0], dtype=torch.int32)
        out = ops.paged_sparse_mqa(q.to(dev), pages, scales, table, idx, win.to(dev), end.to(dev), sink.to(dev), D ** -0.5,
                                   8, ws=ws)
        rows = ops.paged_read(pages, scales, table, torch.zeros_like(e0), n, ws=ws)
        assert ws.status() == 0
        c = dict(q=q, pages=pages, scales=scales, table=table.cpu(), kv_win=win, win_end=end, sink=sink)
        R.check_attention(out, _refs(c, 8, D ** -0.5, idx=idx.cpu()), BF16, k + 8)
        # the same attention over the rows read back, unpaged
        flat = ops.sparse_mqa(q.to(dev), rows, idx, win.to(dev), end.to(dev), sink.to(dev), D ** -0.5, 8)
        R.check_attention(flat, _refs(c, 8, D ** -0.5, idx=idx.cpu()), BF16, k + 8)


def test_entry_points_refuse_bad_arguments():
    build()
    L = _lib.lib()
    N, P = ctypes.c_void_p(0), ctypes.c_void_p(4096)  # P is never dereferenced
    odd = ctypes.c_void_p(4097)
    ws = L.csa_paged_mqa_workspace_bytes(2, 4, 64, 1 << 16)

    def call(dense=False, q=P, pages=P, sc=P, table=P, rows=P, win=P, sink=P, out=P, Q=2, B=1, H=4, D=64, np_=9, page=16,
             per=3, k=7, W=5, end=P, T=9, qps=2, dt=1, cd=3, w=P, wb=ws):
        head = (q, pages, sc, table, rows, win, sink, 0.1, out, Q, B, H, D, np_, page, per)
        tail = (W, end, T, qps, dt, cd, w, wb, N)
        return L.csa_paged_hca_mqa(*head, *tail) if dense else L.csa_paged_sparse_mqa(*head, k, *tail)

    bad = [dict(q=N), dict(pages=N), dict(sc=N), dict(table=N), dict(rows=N), dict(win=N), dict(sink=N), dict(out=N),
           dict(end=N), dict(Q=0), dict(B=0), dict(H=0), dict(H=129), dict(D=0), dict(D=1040), dict(D=72), dict(np_=0),
           dict(page=0), dict(per=0), dict(per=1 << 20, page=1 << 12), dict(W=-1), dict(W=70000), dict(T=0), dict(qps=0),
           dict(qps=1), dict(dt=2), dict(cd=1), dict(cd=0, sc=N), dict(q=odd), dict(out=odd), dict(sink=odd),
           dict(rows=odd), dict(table=odd), dict(win=odd), dict(end=odd), dict(pages=ctypes.c_void_p(4100))]
    for kw in bad:
        assert call(**kw) == 1, kw
        assert call(dense=True, **kw) == 1, kw
    assert call(k=0) == 1 and call(k=70000) == 1
    for kw in (dict(w=N), dict(wb=255), dict(w=ctypes.c_void_p(4100))):
        assert call(**kw) == 3 and call(dense=True, **kw) == 3


def test_wrappers_refuse_host_tensors():
    c = _inputs(1, 2, 1, 4, 32, 8, 4, 3, "int4", BF16)
    for kw in (dict(n_cmp=torch.zeros(2, dtype=torch.int32)), dict(idx=torch.zeros(2, 3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            _run("cpu", c, 3, 0.1, **kw)


@gpu
def test_wrappers_refuse_bad_shapes(cuda_device):
    c = {n: (t.to(cuda_device) if isinstance(t, torch.Tensor) else t)
         for n, t in _inputs(1, 2, 2, 4, 32, 8, 4, 3, "int4", BF16).items() if n != "g"}
    idx = torch.zeros(2, 3, dtype=torch.int32, device=cuda_device)
    args = dict(q=c["q"], pages=c["pages"], scales=c["scales"], page_table=c["table"], idx=idx, kv_win=c["kv_win"],
                win_end=c["win_end"], sink=c["sink"], scale=0.1, win_len=3)
    ops.paged_sparse_mqa(**args)
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=cuda_device)  # noqa: E731
    for kw in (dict(q=z(2, 4, 64)), dict(q=z(4, 32)), dict(q=z(2, 4, 32, dtype=torch.float16)), dict(q=z(3, 4, 32)),
               dict(idx=idx[0]), dict(idx=idx.long()), dict(idx=idx[:1]), dict(sink=z(4)), dict(sink=z(5, dtype=F32)),
               dict(kv_win=None), dict(kv_win=z(2, 5, 16)), dict(kv_win=z(1, 5, 32)), dict(win_end=z(3, dtype=torch.int32)),
               dict(win_len=0), dict(scales=None), dict(out=z(2, 4, 31)), dict(out=z(2, 4, 32, dtype=F32)),
               dict(page_table=c["table"][:, :1].t())):
        with pytest.raises((ValueError, TypeError)):
            ops.paged_sparse_mqa(**{**args, **kw})
    with pytest.raises(_lib.CsaError):
        ops.paged_sparse_mqa(**{**args, "idx": idx[:, :0]})


@gpu
@pytest.mark.parametrize("fmt", ["int4", "rows"])
@pytest.mark.parametrize("Q,B,H,D,W", [(450, 450, 64, 512, 0), (400, 2, 64, 512, 70), (170, 1, 100, 256, 3), (310, 31, 5, 128, 64)])
def test_many_queries_of_all_lengths(cuda_device, fmt, Q, B, H, D, W):
    # more queries than SMs, lists from empty to several tiles in any order, used slots behind unused ones
    N, k, page = 200, 200, 16
    c = _inputs(Q + H, Q, B, H, D, N, page, W, fmt, BF16)
    g = c["g"]
    idx = torch.full((Q, k), -1, dtype=torch.int32)
    for i in range(Q):
        m = int(torch.randint(0, k + 1, (1,), generator=g)) * int(i % 3 > 0)
        at = torch.randperm(k, generator=g)[:m]  # anywhere in the list
        idx[i, at] = torch.randperm(N, generator=g)[:m].to(torch.int32)
    ws = ops.Workspace(cuda_device)
    for _ in range(2):
        out = _run(cuda_device, c, W, D ** -0.5, idx=idx, ws=ws)
        assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, idx=idx), BF16, k + W)
    n_cmp = torch.randint(0, N + 1, (Q,), generator=g, dtype=torch.int32)
    n_cmp[::5] = 0
    out = _run(cuda_device, c, W, D ** -0.5, n_cmp=n_cmp, ws=ws)
    assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, n_cmp=n_cmp), BF16, N + W)


@gpu
def test_workspace_on_another_device_is_refused(cuda_device):
    c = _inputs(1, 2, 2, 4, 32, 8, 4, 3, "int4", BF16)
    ws = ops.Workspace("cpu")
    with pytest.raises(ValueError, match="ws is on"):
        _run(cuda_device, c, 3, 0.1, idx=torch.zeros(2, 3, dtype=torch.int32), ws=ws)


@gpu
def test_a_call_s_own_workspace_lives_until_the_launch(cuda_device, monkeypatch):
    made = []

    class Recorded(ops.Workspace):
        def get(self, nbytes):
            w = super().get(nbytes)
            made.append(weakref.ref(w))
            return w

    call, names = ops._call, []

    def checked(name, *args):
        assert made[-1]() is not None, name
        names.append(name)
        call(name, *args)

    monkeypatch.setattr(ops, "Workspace", Recorded)
    monkeypatch.setattr(ops, "_call", checked)
    Q, H, D, N = 2, 4, 128, 40
    c = _inputs(41, Q, Q, H, D, N, 16, 0, "int4", BF16)
    d = {n: (t.to(cuda_device) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    cache, e0 = (d["pages"], d["scales"], d["table"]), torch.zeros(Q, dtype=torch.int32, device=cuda_device)
    ops.paged_append(d["q"], *cache, e0)
    ops.paged_read(*cache, e0, 3)
    ops.paged_hca_mqa(d["q"], *cache, e0, None, None, d["sink"], 0.1, 0)
    ops.paged_sparse_mqa(d["q"], *cache, e0[:, None].contiguous(), None, None, d["sink"], 0.1, 0)
    torch.cuda.synchronize()
    assert len(names) == len(made) == 4


@gpu
def test_graphs_keep_the_workspace_that_they_were_captured_with(cuda_device):
    # Q items above the grid's blocks: the counters in the workspace are used
    Q, H, D, N, W = 170, 64, 128, 70, 0
    c = _inputs(43, Q, 2, H, D, N, 16, W, "int4", BF16)
    dev = cuda_device
    d = {n: (t.to(dev) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    n_cmp = torch.arange(Q, dtype=torch.int32) % (N + 1)
    args = (d["q"], d["pages"], d["scales"], d["table"], n_cmp.to(dev), None, None, d["sink"], 0.1, W)
    want = ops.paged_hca_mqa(*args)
    refs = _refs(c, W, 0.1, n_cmp=n_cmp)
    R.check_attention(want, refs, BF16, N)
    for first in (False, True):  # a workspace that is new to a capture; one that an eager call has used
        ws = ops.Workspace(dev)
        if first:
            ops.paged_hca_mqa(*args, ws=ws)
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(ops.paged_hca_mqa(*args, ws=ws))
            graphs.append(g)
        ws.get(1 << 20)  # a larger call's
        other = torch.full((1 << 18,), 255, dtype=torch.uint8, device=dev)  # (into what was given back, if anything was)
        eager = ops.paged_hca_mqa(*args, ws=ws)
        for g in (graphs[1], graphs[0], graphs[1]):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, want) and all(torch.equal(o, want) for o in outs)
        assert torch.all(other == 255)
        assert ws.status() == 0


@gpu
@pytest.mark.parametrize("fmt,dtype", [("int4", BF16), ("rows", BF16), ("int4", F32)])
@pytest.mark.parametrize("H,D", [(64, 512), (128, 128), (5, 64)])
def test_a_table_far_longer_than_the_visible_list(cuda_device, H, D, fmt, dtype):
    # a server's table: room for 262,144 entries, pages assigned to the first 100; most splits of the list are empty
    N, W, page = 100, 70, 64
    c = _inputs(51 + H, 2, 2, H, D, N, page, W, fmt, dtype)
    table = torch.full((2, 4096), -1, dtype=torch.int32)
    table[:, :c["table"].shape[1]] = c["table"]
    c["table"] = table
    ws = ops.Workspace(cuda_device)
    for n_cmp in ([N, 3], [0, N], [0, 0]):
        n_cmp = torch.tensor(n_cmp, dtype=torch.int32)
        for rows in (dict(c, q=c["q"][:1], table=table[:1], kv_win=c["kv_win"][:1], win_end=c["win_end"][:1]), c):
            Q = rows["q"].shape[0]
            out = _run(cuda_device, rows, W, D ** -0.5, n_cmp=n_cmp[:Q], ws=ws)
            assert ws.status() == 0
            R.check_attention(out, _refs(rows, W, D ** -0.5, n_cmp=n_cmp[:Q]), dtype, N + W)
    out = _run(cuda_device, dict(c, kv_win=None, win_end=None), 0, D ** -0.5, n_cmp=torch.zeros(2, dtype=torch.int32), ws=ws)
    assert torch.all(out == 0) and ws.status() == 0


@gpu
@pytest.mark.parametrize("fmt,which", [(f, w) for f in ("int4", "rows") for w in ("q", "pages", "scales", "kv_win", "out")
                                       if (f, w) != ("rows", "scales")])
def test_a_tensor_off_the_16_byte_grid(cuda_device, fmt, which):
    Q, H, D, N, W = 3, 64, 512, 200, 40
    c = _inputs(61, Q, Q, H, D, N, 16, W, fmt, BF16)
    n_cmp = torch.tensor([N, 0, 77], dtype=torch.int32)
    off = 8 if which == "pages" and fmt == "int4" else 2  # bytes (code pages are 8-byte aligned)

    def moved(t):
        t = t.to(cuda_device)
        buf = torch.zeros(t.numel() * t.element_size() + 64, dtype=torch.uint8, device=cuda_device)
        buf = buf[off:off + t.numel() * t.element_size()]
        view = buf.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype).view(t.shape)
        view.copy_(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t)
        assert view.data_ptr() % 16
        return view

    d = {n: t.to(cuda_device) if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    out = torch.empty_like(d["q"])
    if which == "out":
        out = moved(out)
    else:
        d[which] = moved(c[which])
    ws = ops.Workspace(cuda_device)
    got = ops.paged_hca_mqa(d["q"], d["pages"], d["scales"], d["table"], n_cmp.to(cuda_device), d["kv_win"], d["win_end"], d["sink"],
                            D ** -0.5, W, out=out, ws=ws)
    assert got.data_ptr() == out.data_ptr() and ws.status() == 0
    R.check_attention(got, _refs(c, W, D ** -0.5, n_cmp=n_cmp), BF16, N + W)
