"""Bounded waits of the paged attention: with a limit of a nanosecond (bytes
8..15 of the workspace) some wait of its pipeline runs out, the kernel raises
CSA_STATUS_WAIT_TIMEOUT, ends what it has in flight and returns, its counters at
zero. The context stays usable. The limit is an ordinary argument of the wait: no
GPU fault is caused."""
import pytest
import torch

import paged_reference as R
from compressed_sparse_attention_15_b200 import ops
from test_paged_mqa import _inputs, _refs, _run

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("Q,W", [(2, 130), (300, 0)])
def test_wait_timeout_raises_status_and_returns(cuda_device, Q, W):
    # one used slot in front of 65,535 unused ones: every role waits while the list's end is looked for
    H, D, N, k = 64, 512, 90, 65536
    c = _inputs(Q, Q, Q, H, D, N, 64, W, "int4", BF16)
    idx = torch.full((Q, k), -1, dtype=torch.int32)
    idx[:, 0] = torch.arange(Q) % N
    ws = ops.Workspace(cuda_device)
    ws.get(1 << 26)[8:16].copy_(torch.tensor([1], dtype=torch.int64).view(torch.uint8).to(cuda_device))
    _run(cuda_device, c, W, D ** -0.5, idx=idx, ws=ws)
    torch.cuda.synchronize()  # the call returned: every wait ended
    assert ws.status() & 8
    assert torch.all(ws.buf[16:256] == 0), "the counters are back at zero"
    # the same workspace without the limit: clean and right
    ws.buf[8:16].zero_()
    out = _run(cuda_device, c, W, D ** -0.5, idx=idx, ws=ws)
    assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, idx=idx), BF16, 1 + W)


@pytest.mark.parametrize("D", [128, 512])
@pytest.mark.parametrize("Q", [2, 300])
def test_teardown_with_window_copies_in_flight(cuda_device, Q, D):
    # Four whole window tiles a query: both tile buffers may be filling in bulk when the wait for one of them runs out.
    # The block waits for their bytes, not for the roles that left, so the call returns at once (a copy takes
    # microseconds; waiting for a phase that nobody completes would take the 2 s of the drain's own limit).
    H, N, W = 64, 90, 300
    c = _inputs(Q + D, Q, Q, H, D, N, 64, W, "int4", BF16)
    c["win_end"][:] = c["kv_win"].shape[1] - 1
    n_cmp = torch.arange(Q, dtype=torch.int32) % (N + 1)
    d = {n: (t.to(cuda_device) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    ws = ops.Workspace(cuda_device)

    def call():
        return ops.paged_hca_mqa(d["q"], d["pages"], d["scales"], d["table"], n_cmp.to(cuda_device), d["kv_win"], d["win_end"],
                                 d["sink"], D ** -0.5, W, ws=ws)

    call()
    assert ws.status() == 0
    limit = ws.buf[8:16].view(torch.int64)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for ns in (1, 2000, 1, 4000):
        limit.fill_(ns)
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        assert start.elapsed_time(end) < 1000, "the block waited for a phase that nobody completes"
        assert ws.status() in (0, 8)
        assert torch.all(ws.buf[16:256] == 0), "the counters are back at zero"
    limit.zero_()
    out = call()
    assert ws.status() == 0
    R.check_attention(out, _refs(c, W, D ** -0.5, n_cmp=n_cmp), BF16, N + W)
