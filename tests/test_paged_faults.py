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
