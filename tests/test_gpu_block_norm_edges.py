"""The block norm where its kernels change hands: rows narrower than a 16-byte piece, gates of many
groups.  Reference and tolerances are those of test_gpu_block_norm."""

import pytest
import torch

from test_gpu_block_norm import BF, F32, HF, make, run_case

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
