"""The Newton-Schulz iteration in 64 bits, exactly and with the operands' number formats.

The formats (two fp16 numbers for X, fp32 diagonals and fp16 off-diagonal entries for A and B,
each at its power-of-two scale) are part of what ``slm_orthogonalize`` documents.  Rounding in
the same places, with every sum and product in 64 bits, shows how far these formats alone take
a result from the exact iteration on the same input.  A kernel that follows them differs from
that emulation by fp32 sums only (relative 2^-24 per addition, against the operands' 2^-11), so
its error is another sample of the same size.  Matrices of up to 256 x 256 with a side of at
most 128 multiply both fp16 numbers of X in the update, others the first.
"""

import torch

STANDARD = (3.4445, -4.7750, 2.0315)


def _f16(t, scale):
    return (t * scale).to(torch.float16).double() / scale


def iterate(u, rows, eps, formats=False):
    """Result for one [m, n] matrix in 64 bits, before the final rounding to bf16."""
    x = u.double()
    x = x / (torch.linalg.vector_norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    both = x.shape[0] <= 128 and x.shape[1] <= 256
    for i, (a, b, c) in enumerate(rows):
        if not formats:
            A = x @ x.T
            x = a * x + (b * A + c * (A @ A)) @ x
            continue
        hi = _f16(x, 2.0 ** 14)
        x = hi + _f16(x - hi, 2.0 ** 14)
        A = hi @ hi.T
        D = A.diagonal().clone()
        R = _f16(A - D.diag(), 2.0 ** 14)
        B = b * (R + D.diag()) + c * (R @ R + (D[:, None] + D[None, :]) * R + (D * D).diag())
        DB = B.diagonal().clone()
        RB = _f16(B - DB.diag(), 2.0 ** 12)
        y = x if both else hi
        x = a * x + DB[:, None] * y + RB @ y
    return x.T if tall else x


def spectrum(m, n, kind, seed, device="cuda"):
    """[m, n] test matrices in 64 bits: noise, decaying, very badly conditioned, a few strong
    directions over a weak floor, low rank."""
    g = torch.Generator(device=device).manual_seed(seed)
    G = torch.randn(m, n, generator=g, device=device, dtype=torch.float64)
    if kind == "noise":
        return G
    k = min(m, n)
    i = torch.arange(1, k + 1, device=device, dtype=torch.float64)
    S = {"decay": 1 / i, "bad": 10 ** (-4 * i / k), "spikes": torch.where(i <= 3, 30.0 / i, 0.01),
         "rank": (i <= max(1, k // 4)).double()}[kind]
    U, _, Vh = torch.linalg.svd(G, full_matrices=False)
    return (U * S) @ Vh


def tolerance(exact, emulated):
    """Relative Frobenius error that a bf16 result may have.  Rounding to bf16 is off by at most
    2^-8 per element; taken together over at least 4096 elements, independent, its measured size
    on the exact result is right to a few per cent, and it adds in squares to the formats'
    error, which as another sample of thousands of roundings is allowed a quarter more.  Small
    matrices get the bound of the rounding and twice the formats' error instead."""
    n = torch.linalg.vector_norm(exact).item()
    e = torch.linalg.vector_norm(emulated - exact).item() / n
    r = torch.linalg.vector_norm(exact.to(torch.bfloat16).double() - exact).item() / n
    if exact.numel() >= 4096 and min(exact.shape) >= 32:
        return 1.25 * (r * r + e * e) ** 0.5
    return 2.0 ** -8 + 2 * e
