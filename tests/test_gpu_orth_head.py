"""``orthogonalize`` on the gradient that this framework makes itself: dW [V, d] in fp32 at the 8B and
the 1B vocabulary, with momentum.  (V x d of the former is 5.3e8: byte offsets beyond 32 bits.)"""

import pytest
import torch

from lm_head_loss_streaming_b200 import orthogonalize
from orth_util import STANDARD

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,d", [(128256, 4096), (32000, 2048)])
def test_weight_gradient_of_the_head(V, d):
    g = torch.Generator(device="cuda").manual_seed(V)
    # A few strong directions over noise, as a gradient has.
    k = d // 16
    grad = torch.randn(V, d, generator=g, device="cuda")
    strength = torch.arange(1, k + 1, device="cuda", dtype=torch.float32).rsqrt()
    grad.addmm_(torch.randn(V, k, generator=g, device="cuda") * strength,
                torch.randn(k, d, generator=g, device="cuda"), beta=0.5)
    grad *= 1e-3
    mom = torch.randn(V, d, generator=g, device="cuda") * 5e-4
    u = 0.95 * mom.double() + 0.05 * grad.double()
    got = orthogonalize(grad, momentum=mom, beta=0.95)
    # Three fp32 roundings of the momentum, as in test_gpu_orth; then the update along it.
    assert ((mom.double() - u).abs() <= 4 * 2.0 ** -24 * (u.abs() + 0.1 * grad.double().abs())).all()
    u = u.mul_(0.95).add_(0.05 * grad.double())
    u /= torch.linalg.vector_norm(u) + 1e-7
    # X_5 = X_0 Q: the polynomials' factors P(G_i) commute with the Gram matrix, G_{i+1} = P G_i P.
    gram = u.T @ u
    eye = torch.eye(d, dtype=torch.float64, device="cuda")
    q = eye
    for a, b, c in [STANDARD] * 5:
        p = a * eye + b * gram + c * (gram @ gram)
        q = q @ p
        gram = p @ gram @ p
    num = den = 0.0
    for rows in range(0, V, 16384):
        x = u[rows:rows + 16384] @ q
        num += (got[rows:rows + 16384].double() - x).square().sum().item()
        den += x.square().sum().item()
    assert (num / den) ** 0.5 <= 2.5e-3
