"""Infinities and NaN in the block norm's backward reach what the formulas let them reach, whichever
kernel takes the rows.  What does not depend on the spoilt element has the bits of the clean run."""

import pytest
import torch

from lm_head_loss_streaming_b200 import block_norm_bwd, block_norm_fwd
from test_gpu_block_norm import BF, F32, HF, make

pytestmark = pytest.mark.gpu
ROW = 5


def both(t, dr, dh):
    kw = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    f = block_norm_fwd(t["x"], t["y"], residual_scale=0.75, block_scale=1.25, **kw)
    return block_norm_bwd(f, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)


def padded(v):
    """The same rows, further apart in memory than the outputs' rows by one element."""
    wide = torch.zeros(v.shape[0], v.shape[1] + 1, dtype=v.dtype, device=v.device)
    wide[:, :-1] = v
    return wide[:, :-1]


# Whole 16-byte pieces, rows off 16-byte boundaries, rows of several warps, and arrays whose rows lie
# differently (the general kernels).
@pytest.mark.parametrize("layout", ["plain", "apart"])
@pytest.mark.parametrize("d", [200, 201, 2048, 2053])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("dtype,gate_rows", [(BF, 0), (BF, 1), (HF, 40), (F32, 4)])
def test_spoilt_block_output(dtype, gate_rows, pre, post, bad, d, layout):
    t, dr, dh = make(40, d, dtype, gate_rows=gate_rows, post=post, pre=pre, seed=d)
    if layout == "apart":
        t["y"] = padded(t["y"])
    clean = both(t, dr, dh)
    c = d // 2
    t["y"][ROW, c] = bad
    got = both(t, dr, dh)
    others = [n for n in range(40) if n != ROW]
    assert torch.equal(got.dx[others], clean.dx[others])
    assert torch.equal(got.dy[others], clean.dy[others])
    if pre:
        # r of the row has the spoilt element, and so has its norm.
        assert got.dx[ROW].isnan().all() and got.dy[ROW].isnan().all()
        return
    assert torch.equal(got.dx[ROW], clean.dx[ROW])      # residual_scale d_residual
    if post:
        assert got.dy[ROW].isnan().all()                # through the norm of y
    else:
        assert torch.equal(got.dy[ROW], clean.dy[ROW])  # block_scale gate d_residual
        if gate_rows:
            rest = [k for k in range(d) if k != c]
            assert torch.equal(got.dgate[:, rest], clean.dgate[:, rest])
            per = 40 // gate_rows
            assert not got.dgate[ROW // per, c].isfinite()
            keep = [g for g in range(gate_rows) if g != ROW // per]
            assert torch.equal(got.dgate[keep], clean.dgate[keep])


@pytest.mark.parametrize("layout", ["plain", "apart"])
@pytest.mark.parametrize("d", [200, 201, 4096])
@pytest.mark.parametrize("name", ["x", "dr", "dh"])
def test_spoilt_stream_and_gradients(name, d, layout):
    """With both norms every element of the row depends on the spoilt one, no other row's does."""
    t, dr, dh = make(40, d, BF, gate_rows=1, seed=d)
    if layout == "apart":
        t["y"] = padded(t["y"])
    clean = both(t, dr, dh)
    {"x": t["x"], "dr": dr, "dh": dh}[name][ROW, 3] = float("nan")
    got = both(t, dr, dh)
    others = [n for n in range(40) if n != ROW]
    for k in ("dx", "dy"):
        a, b = getattr(got, k), getattr(clean, k)
        assert torch.equal(a[others], b[others])
        if name != "dr" or k == "dy":
            assert a[ROW].isnan().all()
        else:                                           # dx = residual_scale g, element by element
            assert a[ROW].isnan().sum() == 1 and a[ROW, 3].isnan()


def test_stream_alone_does_not_reach_gradients_without_a_norm():
    t, dr, _ = make(40, 136, BF, gate_rows=1, pre=False)
    clean = both(t, dr, None)
    t["x"][ROW, 3] = float("nan")
    got = both(t, dr, None)
    for k in ("dx", "dy", "dgate", "dw_post"):
        assert torch.equal(getattr(got, k), getattr(clean, k)), k
