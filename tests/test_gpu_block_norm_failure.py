"""The device-side failure path of the block norm's backward: a bounded wait of its ring that runs
out.

The test hook slm_debug_set(1, ...) makes the first stage of each block's ring (of a cluster, of its
first block's) want a release that no warp gives, so that the copying warp's wait for it runs out,
and in a cluster the other blocks' waits for that block's sums.  The kernel must record SLM_ERR_TIMEOUT, let
its copies land and return, and the next call must be right.  Every wait is bounded; nothing
faults."""

import pytest
import torch

from lm_head_loss_streaming_b200 import _lib, block_norm_bwd, block_norm_fwd
from test_gpu_block_norm import BF, F32, make

pytestmark = pytest.mark.gpu


def status(ws):
    return _lib.slm_device_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)


# More batches for a worker than its ring has stages.  One warp per row, one block per row, clusters of
# 2, 4 and 8 blocks; rows on and off 16-byte boundaries; a gate per token.
@pytest.mark.parametrize("N,d,dtype,gate_rows", [
    (20000, 256, BF, 1), (2000, 4096, BF, 1), (2000, 4097, BF, 0), (2000, 2048, BF, 2000),
    (1200, 8192, BF, 1), (700, 16384, BF, 1), (700, 16377, BF, 1), (400, 16384, F32, 0)])
def test_wait_runs_out_reports_timeout_and_the_next_call_is_right(N, d, dtype, gate_rows):
    t, dr, dh = make(N, d, dtype, gate_rows=gate_rows, seed=d)
    kw = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    f = block_norm_fwd(t["x"], t["y"], **kw)
    ws = torch.empty(_lib.slm_block_norm_workspace_bytes(N, d, gate_rows), dtype=torch.uint8,
                     device="cuda")
    back = lambda: block_norm_bwd(f, t["x"], t["y"], d_residual=dr, d_hidden=dh,  # noqa: E731
                                  workspace=ws, **kw)
    want = back()
    assert status(ws) == 0
    assert _lib.slm_debug_set(1, 100_000_000) == 0   # ~0.05-0.1 s per wait
    try:
        back()
        st = status(ws)
    finally:
        assert _lib.slm_debug_set(0, 0) == 0
    assert st == 7, _lib.status_string(st)           # SLM_ERR_TIMEOUT
    got = back()
    assert status(ws) == 0
    for k, v in want.__dict__.items():
        if isinstance(v, torch.Tensor):
            assert torch.equal(getattr(got, k), v), k


@pytest.mark.parametrize("what", ["norm", "norm clusters", "update", "small update"])
def test_wait_that_ran_out_is_known_without_a_workspace(what):
    """The default calls and autograd drop their workspace; the device remembers."""
    from lm_head_loss_streaming_b200 import block_norm, device_status, orthogonalize
    n, d = (700, 16384) if what == "norm clusters" else (2000, 4096)
    x, y = (torch.randn(n, d, device="cuda").to(BF).requires_grad_() for _ in range(2))
    w = torch.ones(d, device="cuda", dtype=BF)
    side = 200 if what == "small update" else 500
    g = torch.randn(side, side, device="cuda")

    def call():
        if "update" in what:
            orthogonalize(g)
        else:
            block_norm(x, y, w_pre=w)[1].sum().backward()

    device_status()                                  # what earlier tests left
    call()
    assert device_status() == 0
    assert _lib.slm_debug_set(1, 100_000_000) == 0   # ~0.05-0.1 s per wait
    try:
        call()
        torch.cuda.synchronize()
    finally:
        assert _lib.slm_debug_set(0, 0) == 0
    call()                                           # a good call after it clears nothing
    assert device_status() == 7
    assert device_status() == 0
