"""The block norm where its kernels change hands: rows narrower than a 16-byte piece.  Reference and
tolerances are those of test_gpu_block_norm."""

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
