"""The block norm where its kernels change hands: rows narrower than a 16-byte piece, gates of many
groups, arrays that all begin equally far from a 16-byte boundary.  Reference and tolerances are those
of test_gpu_block_norm."""

import pytest
import torch

from lm_head_loss_streaming_b200 import _lib, block_norm_fwd
from lm_head_loss_streaming_b200.norms import _DTYPE
from test_gpu_block_norm import BF, BWD, F32, HF, check, make, reference, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 8, 9])
@pytest.mark.parametrize("N,gate_rows,gate_dtype", [(2, 0, None), (3, 3, F32), (4, 1, BF),
                                                    (30, 6, F32), (301, 301, BF)])
def test_rows_narrower_than_a_piece(N, gate_rows, gate_dtype, d):
    t, dr, dh = make(N, d, BF, gate_rows=gate_rows, gate_dtype=gate_dtype, seed=N + d)
    run_case(t, dr, dh)
    if gate_dtype is not BF:
        for dtype in (HF, F32):
            t, dr, dh = make(N, d, dtype, gate_rows=gate_rows, gate_dtype=gate_dtype, seed=d)
            run_case(t, dr, dh)


# Groups by row classes (4, 2, 1 of them), as many as have workers of their own and more; whole
# pieces beside a weight that is not aligned.
@pytest.mark.parametrize("dtype,d,groups", [(BF, 1026, 148), (BF, 1026, 150), (BF, 1028, 296),
                                            (BF, 1028, 300), (F32, 258, 296), (F32, 258, 400),
                                            (BF, 1024, 75), (HF, 512, 700), (F32, 256, 1000)])
def test_gates_of_many_groups(dtype, d, groups):
    t, dr, dh = make(3 * groups, d, dtype, gate_rows=groups, seed=groups)
    run_case(t, dr, dh)
    odd = torch.empty(d + 1, dtype=dtype, device="cuda")[1:]
    odd.copy_(t["w_pre"])
    run_case(dict(t, w_pre=odd), dr, dh)


class Inside:
    """Tensors that begin `start` elements into a buffer of NaN."""

    def __init__(self, start):
        self.start, self.all = start, []

    def __call__(self, v):
        buf = torch.full((v.numel() + 2 * self.start + 8,), float("nan"), dtype=v.dtype, device="cuda")
        got = buf[self.start:self.start + v.numel()].view(v.shape)
        got.copy_(v)
        self.all.append((buf, v.numel()))
        return got

    def check(self):
        """Nothing was written around them."""
        for buf, n in self.all:
            assert buf[:self.start].isnan().all() and buf[self.start + n:].isnan().all()


# The wrapper's outputs are aligned, so that inputs which are not go to the general kernels; through
# the C entry the outputs may lie as the inputs do, and the ring takes the rows from there.
@pytest.mark.parametrize("dtype,start", [(BF, 1), (BF, 4), (HF, 7), (F32, 1), (F32, 3)])
@pytest.mark.parametrize("N,d,gate_rows", [(1, 8, 1), (23, 9, 0), (40, 15, 40), (23, 200, 1), (700, 201, 7),
                                           (23, 2048, 23), (31, 2053, 1), (9, 5001, 9), (300, 5000, 3),
                                           (33, 16380, 1)])
def test_arrays_that_begin_off_a_boundary(N, d, gate_rows, dtype, start):
    t, dr, dh = make(N, d, dtype, gate_rows=gate_rows, seed=N + d)
    f = block_norm_fwd(t["x"], t["y"], t["w_pre"], t["w_post"], t["gate"], 0.75, 1.25)
    place = Inside(start)
    u = {k: None if v is None else place(v) for k, v in t.items()}
    grads = place(dr), place(dh)
    got = dict(dx=place(torch.zeros_like(dr)), dy=place(torch.zeros_like(dr)),
               dgate=None if t["gate"] is None else place(torch.zeros_like(t["gate"])),
               dw_pre=place(torch.zeros(d, device="cuda")), dw_post=place(torch.zeros(d, device="cuda")))
    ws = torch.empty(_lib.slm_block_norm_workspace_bytes(N, d, gate_rows), dtype=torch.uint8,
                     device="cuda")
    at = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    dt = _DTYPE[dtype]
    st = _lib.slm_block_norm_bwd(
        dt, at(u["x"]), d, at(u["y"]), d, at(u["w_post"]), at(u["w_pre"]), dt, at(u["gate"]), dt,
        gate_rows, at(grads[0]), d, at(grads[1]), d, at(f.stats), at(f.stats[1]), N, d, 0.75, 1.25,
        0.0, at(got["dx"]), at(got["dy"]), at(got["dgate"]), at(got["dw_post"]), at(got["dw_pre"]),
        at(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    val, tol = reference(t, dr, dh, 0.75, 1.25, 1e-6, 0.0)
    check(got, val, tol, BWD)
    place.check()
