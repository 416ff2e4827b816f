"""``orthogonalize`` where a launch is refused: nothing of the call may have happened."""

import pytest
import torch

from lm_head_loss_streaming_b200 import _lib, orthogonalize
from orth_util import spectrum

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(300, 200), (600, 1300), (300, 6000), (1100, 1100)])
def test_refused_launch_leaves_the_momentum(shape):
    g = spectrum(*shape, "noise", 1).float()
    mom = spectrum(*shape, "noise", 2).float()
    out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    old, twin = mom.clone(), mom.clone()
    assert _lib.slm_debug_set(4, 0) == 0             # the products' launch is refused
    try:
        with pytest.raises(_lib.SLMError) as e:
            orthogonalize(g, momentum=mom, out=out)
    finally:
        assert _lib.slm_debug_set(0, 0) == 0
    assert e.value.status == 8                       # SLM_ERR_CUDA
    torch.cuda.synchronize()
    assert torch.equal(mom, old) and (out == 7.0).all()
    want = orthogonalize(g, momentum=twin)
    assert torch.equal(orthogonalize(g, momentum=mom, out=out), want) and torch.equal(mom, twin)
