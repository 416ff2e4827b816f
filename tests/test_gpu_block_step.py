"""A training step of a draft block's end: the norms around the block (``block_norm``) make the
hidden states of the streaming loss and take the gradient that it returns, and an optimiser's
update (``orthogonalize``) is made of the weight gradients.

Each part is held to its own reference on the inputs that the part before really gave it: the
loss's gradient to the dense loss in 64 bits (1e-2 of the largest entry, as in the parity
tests), the norms' gradients to the formulas (the bounds of test_gpu_block_norm), the update to
the iteration (orth_util.tolerance).  The autograd chain must give the explicit calls' bits.
"""

import pytest
import torch

from lm_head_loss_streaming_b200 import (block_norm, block_norm_bwd, block_norm_fwd,
                                         lm_head_loss_bwd, lm_head_loss_fwd, orthogonalize,
                                         streaming_lm_head_loss)
from orth_util import STANDARD, iterate, tolerance
from test_gpu_block_norm import BWD, FWD, check, reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def inputs(N, d, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(
        x=rn(N, d).to(BF), z=rn(N, d).to(BF), proj=(rn(d, d) * d ** -0.5).to(BF),
        w_pre=(1 + 0.1 * rn(d)).to(BF), w_post=(1 + 0.1 * rn(d)).to(BF),
        gate=(0.5 + 0.1 * rn(1, d)).to(BF), W=(rn(V, d) * 0.05).to(BF),
        target=rn(N, d).to(BF),
        labels=torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32))


@pytest.mark.parametrize("kind,N,d,V", [("ce", 300, 256, 3001), ("kl_div", 257, 264, 2000),
                                        ("ce", 1, 128, 777)])
def test_step_part_by_part(kind, N, d, V):
    t = inputs(N, d, V, seed=N + d)
    t["labels"][::7] = -100
    y = t["z"] @ t["proj"]
    nrm = dict(x=t["x"], y=y, w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    par = {k: nrm[k] for k in ("w_pre", "w_post", "gate")}
    lab = t["labels"] if kind == "ce" else None
    tgt = None if kind == "ce" else t["target"]

    f = block_norm_fwd(t["x"], y, residual_scale=0.75, block_scale=1.25, **par)
    loss = lm_head_loss_fwd(kind, f.hidden, t["W"], lab, tgt)
    dH, dW = lm_head_loss_bwd(loss, f.hidden, t["W"], lab, tgt)
    b = block_norm_bwd(f, t["x"], y, d_hidden=dH, **par)

    # The loss on the hidden states that the norms made.
    h = f.hidden.double().requires_grad_()
    logp = (h @ t["W"].double().T).log_softmax(1)
    if kind == "ce":
        valid = lab != -100
        ref = -logp.gather(1, lab.clamp_min(0).long()[:, None])[:, 0][valid].sum()
        ref = ref / max(int(valid.sum()), 1)
    else:
        lp = (tgt.double() @ t["W"].double().T).log_softmax(1)
        ref = (lp.exp() * (lp - logp)).sum(1).mean()
    ref.backward()
    assert abs(loss.loss_mean.item() - ref.item()) <= 2e-3 * max(abs(ref.item()), 1e-2)
    assert (dH.double() - h.grad).abs().max() <= 1e-2 * h.grad.abs().max()

    # The norms' gradients of the gradient that the loss returned.
    val, tol = reference(nrm, None, dH, 0.75, 1.25, 1e-6, 0.0)
    check({**f.__dict__, **b.__dict__}, val, tol, ("residual",) + FWD + BWD)

    # The update of the projection (and of the head itself).
    d_proj = (t["z"].float().T @ b.dy.float())
    for grad in (d_proj, dW):
        u = orthogonalize(grad)
        if not grad.any():           # every label masked: the update of nothing is nothing
            assert not u.any()
            continue
        exact = iterate(grad, [STANDARD] * 5, 1e-7)
        emulated = iterate(grad, [STANDARD] * 5, 1e-7, formats=True)
        off = torch.linalg.vector_norm(u.double() - exact) / torch.linalg.vector_norm(exact)
        assert off.item() <= tolerance(exact, emulated)

    # The same through autograd.
    leaves = {k: v.clone().requires_grad_() for k, v in nrm.items()}
    W = t["W"].clone().requires_grad_()
    _, hidden = block_norm(residual_scale=0.75, block_scale=1.25, **leaves)
    streaming_lm_head_loss(hidden, W, lab, tgt, kind=kind).backward()
    assert torch.equal(leaves["x"].grad, b.dx) and torch.equal(leaves["y"].grad, b.dy)
    assert torch.equal(leaves["gate"].grad, b.dgate)
    assert torch.equal(leaves["w_pre"].grad, b.dw_pre.to(BF))
    assert torch.equal(leaves["w_post"].grad, b.dw_post.to(BF))
    assert torch.equal(W.grad, dW.to(BF))


def test_captured_step_replays_on_new_inputs():
    t = inputs(200, 256, 2000, seed=4)
    mom = torch.zeros(256, 256, device="cuda")

    def step(m):
        y = t["z"] @ t["proj"]
        par = {k: t[k] for k in ("w_pre", "w_post", "gate")}
        f = block_norm_fwd(t["x"], y, **par)
        loss = lm_head_loss_fwd("ce", f.hidden, t["W"], t["labels"])
        dH, dW = lm_head_loss_bwd(loss, f.hidden, t["W"], t["labels"])
        b = block_norm_bwd(f, t["x"], y, d_hidden=dH, **par)
        return b.dx, dW, orthogonalize(t["z"].float().T @ b.dy.float(), momentum=m)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(mom.clone())
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(mom)
    twin = mom.clone()
    for seed in (5, 6):
        for k, v in inputs(200, 256, 2000, seed).items():
            t[k].copy_(v)
        graph.replay()
        want = step(twin)
        torch.cuda.synchronize()
        assert torch.equal(mom, twin)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_traced_launches_have_their_classes():
    from lm_head_loss_streaming_b200 import _lib
    t = inputs(64, 128, 500, seed=1)
    torch.cuda.synchronize()
    _lib.slm_trace_enable(True)
    try:
        _lib.slm_trace_read()
        f = block_norm_fwd(t["x"], t["z"], t["w_pre"], t["w_post"])
        block_norm_bwd(f, t["x"], t["z"], t["w_pre"], t["w_post"], d_hidden=t["x"])
        orthogonalize(t["W"])
        orthogonalize(t["proj"])
        st, classes = _lib.slm_trace_read()
    finally:
        _lib.slm_trace_enable(False)
    assert st == 0
    assert classes["norm"][1] == 2 and classes["norm"][0] > 0      # forward, backward
    assert classes["orth"][1] == 3 and classes["orth"][0] > 0      # preparation, products; small
    assert sum(n for _, n in classes.values()) == 5
