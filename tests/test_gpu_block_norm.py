"""The fused norms, gate and residual of a block (``block_norm``) against the formulas in 64
bits, forward and backward.

Tolerances.  Every output is fp32 arithmetic rounded once to its type, so an element may be
off by half a step of its type, eps / 2 relative, plus the fp32 error.  A sum of d terms taken
in per-thread runs of at most d / 32 terms and a tree of at most 16 levels is off by at most
(d / 32 + 16) 2^-24 relative to the sum of its terms' magnitudes (all positive for the norms);
with the approximate 1 / sqrt (2 ulp) and the few products behind it, one norm factor carries
E = (d / 32 + 32) 2^-24.  An element of r carries E times its terms' magnitudes, and the norm
of r carries that on: R = 1 + sum(|r| mag_r) / sum(r^2) bounds how much a cancellation between
the stream and the block magnifies it.  A gradient is made of at most 8 such factors.  Sums
over N rows add (N + 64) 2^-24 times their terms' magnitudes.
"""

import pytest
import torch

from lm_head_loss_streaming_b200 import block_norm, block_norm_bwd, block_norm_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(N, d, dtype=BF, w_dtype=None, gate_rows=0, gate_dtype=None, post=True, pre=True,
         y=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w_dtype, gate_dtype = w_dtype or dtype, gate_dtype or dtype
    t = dict(x=rn(N, d).to(dtype), y=(0.7 * rn(N, d)).to(dtype) if y else None,
             w_pre=(1 + 0.2 * rn(d)).to(w_dtype) if pre else None,
             w_post=(1 + 0.2 * rn(d)).to(w_dtype) if post and y else None,
             gate=(0.5 + 0.3 * rn(gate_rows, d)).to(gate_dtype) if gate_rows and y else None)
    dr = rn(N, d).to(dtype)
    dh = rn(N, d).to(dtype) if pre else None
    return t, dr, dh


def reference(t, dr, dh, rs, bs, eps, o):
    """Values in 64 bits and the bound of each (see above)."""
    D = {k: None if v is None else v.double() for k, v in t.items()}
    x, y = D["x"], D["y"]
    N, d = x.shape
    E = (d / 32 + 32) * U
    dt = t["x"].dtype
    h = half_step(dt)
    val, tol = {}, {}

    def put(name, v, mag, dtype=None):
        s = h if dtype is None else half_step(dtype)
        val[name] = v
        tol[name] = s * v.abs() + (1 + s) * mag + torch.finfo(dtype or dt).tiny * s

    one = torch.ones((), dtype=torch.float64, device=x.device)
    per = 1
    gate = wq = one
    yh = iy = None
    r = rs * x
    mag = (rs * x).abs()
    if y is not None:
        if D["gate"] is not None:
            G = D["gate"].reshape(-1, d)
            per = N // G.shape[0]
            gate = G.repeat_interleave(per, 0)
        if D["w_post"] is not None:
            wq = D["w_post"] + o
            iy = 1 / (y.square().mean(1, keepdim=True) + eps).sqrt()
        else:
            iy = torch.ones(N, 1, dtype=torch.float64, device=x.device)
        yh = y * iy
        r = r + bs * gate * (yh * wq)
        mag = mag + (bs * gate * yh).abs() * (wq.abs() if wq is one else D["w_post"].abs() + abs(o))
        put("residual", r, E * mag)
    ir = torch.zeros(N, 1, dtype=torch.float64, device=x.device)
    R = torch.ones(N, 1, dtype=torch.float64, device=x.device)
    rh = torch.zeros_like(x)
    wp, wpm = torch.zeros_like(x), torch.zeros_like(x)
    if D["w_pre"] is not None:
        ir = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
        R = 1 + (mag * r.abs()).sum(1, keepdim=True) / (r.square().sum(1, keepdim=True) + d * eps)
        rh = r * ir
        wp, wpm = D["w_pre"] + o, D["w_pre"].abs() + abs(o)
        put("hidden", rh * wp, 2 * E * R * (ir * mag + rh.abs()) * wpm)
    if dr is None and dh is None:
        return val, tol
    g0 = torch.zeros_like(x) if dr is None else dr.double()
    dhd = torch.zeros_like(x) if dh is None else dh.double()
    u, um = dhd * wp, dhd.abs() * wpm
    rhm = ir * mag + rh.abs()          # magnitude behind rh
    c1 = (u * rh).mean(1, keepdim=True)
    c1m = (um * rhm).mean(1, keepdim=True)
    g = g0 + ir * (u - rh * c1)
    gm = g0.abs() + ir * (um + rhm * c1m)
    F = 8 * E * R
    put("dx", rs * g, abs(rs) * F * gm)
    S = (N + 64) * U
    if D["w_pre"] is not None:
        put("dw_pre", (dhd * rh).sum(0), (dhd.abs() * rhm * (F + S)).sum(0), F32)
    if y is not None:
        wqm = wq.abs() if D["w_post"] is None else D["w_post"].abs() + abs(o)
        a, am = bs * gate * wq, (bs * gate).abs() * wqm
        if D["w_post"] is not None:
            c2 = (a * yh * g).mean(1, keepdim=True)
            c2m = (am * yh.abs() * (gm + ir * rhm * c1m)).mean(1, keepdim=True)
            put("dy", iy * (a * g - yh * c2), iy * F * (am * gm + yh.abs() * c2m))
            put("dw_post", (bs * gate * yh * g).sum(0),
                ((bs * gate * yh).abs() * gm * (F + S)).sum(0), F32)
        else:
            put("dy", a * g, F * am * gm)
        if D["gate"] is not None:
            dg = bs * yh * wq * g
            dgm = abs(bs) * yh.abs() * wqm * gm * (F + (per + 64) * U)
            shape = t["gate"].shape
            put("dgate", dg.reshape(-1, per, d).sum(1).reshape(shape),
                dgm.reshape(-1, per, d).sum(1).reshape(shape), t["gate"].dtype)
    return val, tol


def check(got, val, tol, names):
    for k in names:
        if k not in val:
            assert got[k] is None, k
            continue
        v = got[k].double()
        assert v.shape == val[k].shape, k
        off = (v - val[k]).abs()
        bad = ~(off <= tol[k])
        assert not bad.any(), (k, off[bad].max().item(), tol[k][bad].min().item(),
                               int(bad.sum()))


FWD, BWD = ("hidden",), ("dx", "dy", "dgate", "dw_pre", "dw_post")


def run_case(t, dr, dh, rs=0.75, bs=1.25, eps=1e-6, o=0.0, views=None):
    kw = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    if t["y"] is None:
        rs = 1.0
    f = block_norm_fwd(t["x"], t["y"], residual_scale=rs, block_scale=bs, eps=eps,
                       weight_offset=o, **kw)
    b = block_norm_bwd(f, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)
    val, tol = reference(t, dr, dh, rs, bs, eps, o)
    names = FWD + BWD + (("residual",) if t["y"] is not None else ())
    check({**f.__dict__, **b.__dict__}, val, tol, names)
    return f, b


# Widths: one channel, below and above a warp, odd, whole 16-byte pieces, several pieces per
# thread, more than one block of threads per row; rows: one, few, ragged.
SHAPES = [(1, 1), (3, 7), (2, 64), (5, 100), (130, 256), (37, 1001), (1, 4096), (70, 2048),
          (33, 4096), (301, 520), (9, 8192), (17, 16384), (3, 16392), (2, 40000), (5, 33001), (1, 1001), (40, 5001), (21, 16387),
          (1700, 515), (700, 2049), (9, 9999)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_all_parts(shape, dtype):
    N, d = shape
    t, dr, dh = make(N, d, dtype, gate_rows=1, seed=N + d)
    run_case(t, dr, dh)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate_rows", [0, 1, 6, 30, 60])
@pytest.mark.parametrize("d", [96, 101, 1540, 4096, 4097])
def test_parts_and_gates(post, pre, gate_rows, d):
    t, dr, dh = make(60, d, BF, F32, gate_rows, F32 if gate_rows == 6 else BF, post, pre, seed=d)
    run_case(t, dr, dh, o=1.0 if gate_rows == 6 else 0.0)


@pytest.mark.parametrize("N,gate_rows", [(1000, 500), (1200, 2), (900, 300), (2048, 1),
                                         (1184, 37)])
def test_shared_gate_slices(N, gate_rows):
    for d in (72, 77, 2052):
        t, dr, dh = make(N, d, HF, gate_rows=gate_rows, seed=N)
        run_case(t, dr, dh)


@pytest.mark.parametrize("dtype,d", [(BF, 1000), (HF, 2057), (F32, 515), (BF, 6000)])
@pytest.mark.parametrize("start", [1, 3, 8])
def test_views_that_start_between_pieces(dtype, d, start):
    """Every array begins `start` elements into its buffer, the rows end to end from there, with
    neighbours that must be neither read into a row nor written."""
    N = 23
    t, dr, dh = make(N, d, dtype, gate_rows=1, seed=d)

    def inner(v):
        buf = torch.full((N * d + 2 * start,), float("nan"), dtype=dtype, device="cuda")
        buf[start:start + N * d] = v.reshape(-1)
        return buf[start:start + N * d].view(N, d)

    u = dict(t, x=inner(t["x"]), y=inner(t["y"]))
    res, hid = inner(torch.zeros_like(t["x"])), inner(torch.zeros_like(t["x"]))
    f = block_norm_fwd(u["x"], u["y"], t["w_pre"], t["w_post"], t["gate"], 0.75, 1.25,
                       residual=res, hidden=hid)
    b = block_norm_bwd(f, u["x"], u["y"], t["w_pre"], t["w_post"], t["gate"], inner(dr), inner(dh))
    val, tol = reference(t, dr, dh, 0.75, 1.25, 1e-6, 0.0)
    check({**f.__dict__, **b.__dict__}, val, tol, ("residual",) + FWD + BWD)
    for out in (res, hid):
        whole = torch.as_strided(out, (N * d + 2 * start,), (1,), out.storage_offset() - start)
        assert whole[:start].isnan().all() and whole[-start:].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 77, 4096])
def test_norm_alone(d, dtype):
    t, dr, dh = make(50, d, dtype, y=False, seed=d)
    run_case(t, None, dh)
    run_case(t, dr, dh)


@pytest.mark.parametrize("d", [512, 333])
def test_no_residual_gradient(d):
    t, _, dh = make(40, d, BF, gate_rows=1, seed=d)
    run_case(t, None, dh)


@pytest.mark.parametrize("dtype,d,pad", [(BF, 256, 8), (BF, 256, 3), (F32, 100, 4), (HF, 99, 1)])
def test_strided_and_offset_rows(dtype, d, pad):
    """Rows cut out of a wider tensor, at bases that are and are not 16-byte aligned."""
    t, dr, dh = make(45, d, dtype, gate_rows=1, seed=d + pad)

    def cut(v):
        wide = torch.full((v.shape[0], d + 2 * pad), float("nan"), dtype=dtype, device="cuda")
        wide[:, pad:pad + d] = v
        return wide[:, pad:pad + d]

    u = dict(t, x=cut(t["x"]), y=cut(t["y"]))
    f0, b0 = run_case(u, cut(dr), cut(dh))
    odd = torch.empty(2 * d + 3, dtype=dtype, device="cuda")[1:1 + d]   # an unaligned weight
    odd.copy_(t["w_pre"])
    run_case(dict(u, w_pre=odd), cut(dr), cut(dh))


def test_zero_rows_and_zero_values():
    t, dr, dh = make(0, 64, BF, gate_rows=0)
    f = block_norm_fwd(t["x"], t["y"], w_pre=t["w_pre"], w_post=t["w_post"])
    b = block_norm_bwd(f, t["x"], t["y"], w_pre=t["w_pre"], w_post=t["w_post"], d_residual=dr,
                       d_hidden=dh)
    assert f.residual.shape == (0, 64) and b.dx.shape == (0, 64)
    assert not b.dw_pre.any() and not b.dw_post.any()
    t, dr, dh = make(4, 64, F32)
    t["x"][1] = 0
    t["y"][1:3] = 0
    run_case(t, dr, dh)


def test_nan_and_infinity_stay_in_their_row():
    t, dr, dh = make(6, 200, BF, gate_rows=1)
    clean = block_norm_fwd(t["x"], t["y"], t["w_pre"], t["w_post"], t["gate"])
    t["x"][2, 5] = float("nan")
    t["y"][4, 7] = float("inf")
    f = block_norm_fwd(t["x"], t["y"], t["w_pre"], t["w_post"], t["gate"])
    keep = [0, 1, 3, 5]
    assert torch.equal(f.hidden[keep], clean.hidden[keep])
    assert torch.equal(f.residual[keep], clean.residual[keep])
    assert f.hidden[2].isnan().all() and f.residual[2].isnan().sum() == 1
    assert f.residual[4, 7].isnan()    # inf * (1 / inf)


@pytest.mark.parametrize("d", [128, 131, 4096])
def test_in_place_residual_and_given_outputs(d):
    t, _, _ = make(33, d, BF, gate_rows=1, seed=d)
    ref = block_norm_fwd(t["x"], t["y"], t["w_pre"], t["w_post"], t["gate"], 0.5, 2.0)
    x = t["x"].clone()
    h = torch.empty_like(x)
    got = block_norm_fwd(x, t["y"], t["w_pre"], t["w_post"], t["gate"], 0.5, 2.0, residual=x,
                         hidden=h)
    assert got.residual is x and got.hidden is h
    assert torch.equal(x, ref.residual) and torch.equal(h, ref.hidden)


@pytest.mark.parametrize("N,d,gate_rows", [(700, 1024, 1), (513, 136, 27), (64, 16384, 64),
                                           (700, 1023, 1), (513, 131, 27), (64, 9001, 64)])
def test_same_bits_each_time(N, d, gate_rows):
    t, dr, dh = make(N, d, BF, gate_rows=gate_rows, seed=3)
    a = run_case(t, dr, dh)
    for _ in range(3):
        b = run_case(t, dr, dh)
        for p, q in zip(a, b):
            for k, v in p.__dict__.items():
                if isinstance(v, torch.Tensor):
                    assert torch.equal(v, getattr(q, k)), k


def test_autograd_matches_differences():
    """Directional differences of the 64-bit formulas against the gradients (fp32 rows)."""
    t, dr, dh = make(12, 40, F32, gate_rows=3, seed=5)
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    r, h = block_norm(leaves["x"], leaves["y"], leaves["w_pre"], leaves["w_post"], leaves["gate"],
                      0.75, 1.25, 1e-6, 1.0)
    ((r * dr).sum() + (h * dh).sum()).backward()

    def loss(v):
        y = v["y"] / (v["y"].square().mean(1, keepdim=True) + 1e-6).sqrt() * (v["w_post"] + 1)
        q = 0.75 * v["x"] + 1.25 * v["gate"].repeat_interleave(4, 0) * y
        hh = q / (q.square().mean(1, keepdim=True) + 1e-6).sqrt() * (v["w_pre"] + 1)
        return ((q * dr.double()).sum() + (hh * dh.double()).sum()).item()

    base = {k: v.double() for k, v in t.items()}
    for k in t:
        e = torch.randn(t[k].shape, device="cuda", dtype=torch.float64,
                        generator=torch.Generator(device="cuda").manual_seed(7))
        step = 1e-5
        up, down = (loss({**base, k: base[k] + s * step * e}) for s in (1, -1))
        slope = (up - down) / (2 * step)
        got = (leaves[k].grad.double() * e).sum().item()
        # Central differences: O(step^2) and 1e-16 |loss| / step, both below 1e-6 here; the
        # gradients' own error is the fp32 one bounded above, below 1e-4 of the sum.
        scale = (leaves[k].grad.double() * e).abs().sum().item()
        assert abs(slope - got) <= 1e-4 * scale, k


def test_autograd_unused_outputs_and_types():
    t, _, _ = make(8, 64, BF, F32, gate_rows=1, gate_dtype=F32)
    for use in ("residual", "hidden"):
        leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
        r, h = block_norm(**leaves)
        (r if use == "residual" else h).float().square().sum().backward()
        for k, v in leaves.items():
            if use == "residual" and k == "w_pre":
                assert not v.grad.any()
            else:
                assert v.grad.dtype == v.dtype and v.grad.isfinite().all() and v.grad.any(), k
    x = t["x"].clone().requires_grad_()
    r, h = block_norm(x, w_pre=t["w_pre"])
    assert r is x
    (r.float().sum() + h.float().sum()).backward()
    assert x.grad.shape == x.shape


def test_other_stream_and_captured_graph():
    t, dr, dh = make(200, 1024, BF, gate_rows=4, seed=9)
    kw = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    f = block_norm_fwd(t["x"], t["y"], **kw)
    b = block_norm_bwd(f, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f2 = block_norm_fwd(t["x"], t["y"], **kw)
        b2 = block_norm_bwd(f2, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(f.hidden, f2.hidden) and torch.equal(b.dw_post, b2.dw_post)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3 = block_norm_fwd(t["x"], t["y"], **kw)
        b3 = block_norm_bwd(f3, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)
    t["x"].mul_(0.5)
    graph.replay()
    f = block_norm_fwd(t["x"], t["y"], **kw)
    b = block_norm_bwd(f, t["x"], t["y"], d_residual=dr, d_hidden=dh, **kw)
    torch.cuda.synchronize()
    for p, q in ((f, f3), (b, b3)):
        for k, v in p.__dict__.items():
            if isinstance(v, torch.Tensor):
                assert torch.equal(v, getattr(q, k)), k


def test_given_outputs_and_second_derivatives_are_known_to_autograd():
    x, y = (torch.randn(40, 64, device="cuda") for _ in range(2))
    w = torch.rand(64, device="cuda").requires_grad_()
    hidden = torch.empty_like(x)
    block_norm_fwd(x, y, w_pre=w.detach(), hidden=hidden)
    loss = (hidden * w).sum()                       # keeps hidden for w's gradient
    block_norm_fwd(y, x, w_pre=w.detach(), hidden=hidden)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    x.requires_grad_()
    dx, = torch.autograd.grad(block_norm(x, y, w_pre=w)[1].square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_statistics_of_another_type_or_layout_are_refused():
    x = torch.randn(40, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    fwd = block_norm_fwd(x, w_pre=w)
    from lm_head_loss_streaming_b200.norms import BlockNormResult
    for stats in (fwd.stats.double(), fwd.stats.repeat(1, 2)[:, ::2]):
        bad = BlockNormResult(None, None, stats, 1.0, 1.0, 0.0)
        with pytest.raises(ValueError, match="forward"):
            block_norm_bwd(bad, x, w_pre=w, d_hidden=x)
