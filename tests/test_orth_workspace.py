"""The workspace that the orthogonalised update asks for."""

import pytest
import torch

from lm_head_loss_streaming_b200 import orthogonalize, orthogonalize_workspace_bytes


def test_matrices_worked_on_chip_ask_for_no_copies():
    """Up to 256 x 256 nothing but the status word lies in the workspace, however many there are."""
    for batch, m, n in ((1, 256, 256), (100, 256, 256), (65535, 1, 9), (7, 30, 250), (0, 4, 4), (2, 0, 4)):
        assert 0 < orthogonalize_workspace_bytes(batch, m, n) <= 4096
    assert orthogonalize_workspace_bytes(1, 257, 256) > 3 * 2 * 257 * 256


@pytest.mark.gpu
def test_small_workspace_is_enough():
    g = torch.randn(100, 256, 256, device="cuda")
    need = orthogonalize_workspace_bytes(100, 256, 256)
    buf = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    got = orthogonalize(g, workspace=buf[256:256 + need])
    assert torch.equal(got, orthogonalize(g))
    assert (buf[:256] == 7).all() and (buf[256 + need:] == 7).all()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    orthogonalize(g)
    assert torch.cuda.max_memory_allocated() - before <= got.numel() * 2 + (1 << 16)
