"""Cases of the operators on either side of the streaming LM-head loss: the fused norm, gate and
residual of a draft block (``block_norm_fwd``, ``block_norm_bwd``), which makes the hidden states
that the loss reads and takes the gradient that it returns, and the orthogonalised update
(``orthogonalize``) that an optimiser makes of the resulting weight gradients.

Formulas.  block norm, per row of d channels, o the weight offset, norm(t) = t / sqrt(mean(t^2) + eps):
    v = norm(y) (w_post + o)        (v = y without w_post)
    r = residual_scale x + block_scale gate v
    h = norm(r) (w_pre + o)
orthogonalised update: m <- beta m + (1 - beta) g;  u = beta m + (1 - beta) g (u = g without momentum);
    X = u / (||u||_F + eps), then 5 times  X <- a X + (b A + c A^2) X  with A = X X^T.
"""

import math

import torch

own = False

EPS = 1e-6            # of the norms
ORTH_EPS = 1e-7
BETA = 0.95
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _norm(name, N, d, dtype, w_dtype, post, gate, pre, train, groups=1):
    """A block-norm case; gate: "none", "shared" ([groups, d]) or "token" ([N, d])."""
    c = {"op": "norm", "N": N, "d": d, "dtype": dtype, "w_dtype": w_dtype, "post": post,
         "gate": gate, "groups": groups if gate == "shared" else 1, "pre": pre, "train": train}
    return {"name": name, **c} if name else c


def _orth(name, batch, m, n, dtype, momentum):
    c = {"op": "orth", "batch": batch, "m": m, "n": n, "dtype": dtype, "momentum": momentum}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One token of a drafter being served, at the width of the 8B shape: latency alone.
        _norm("norm one token d4096", 1, 4096, "bf16", "bf16", True, "shared", True, False),
        # A batch of requests, one draft token each, plain residual add and next norm in fp16.
        _norm("norm 130 tokens d2048 fp16", 130, 2048, "fp16", "fp16", False, "none", True, False),
        # The rows of the 8B KL workload through the norms around a block, no gradients (the
        # target's side, or evaluation).
        _norm("norm 16384 x d4096", 16384, 4096, "bf16", "bf16", True, "shared", True, False),
        # The same rows in training: forward and every gradient.
        _norm("norm train 16384 x d4096", 16384, 4096, "bf16", "bf16", True, "shared", True, True),
        # The 1B width in training, with a per-token gate that a projection made.
        _norm("norm train 8192 x d2048 token gate", 8192, 2048, "bf16", "fp32", True, "token", True, True),
        # Odd width, ragged rows, fp32 stream, a gate per sequence (5 of them).
        _norm("norm train 1515 x d1001 fp32", 1515, 1001, "fp32", "fp32", True, "shared", True, True, 5),
        # The 405B width: rows of 32 KB.
        _norm("norm train 8192 x d16384", 8192, 16384, "bf16", "bf16", True, "shared", True, True),
        # A small projection's gradient (the width of the smallest workload): launch latency counts.
        _orth("orth 256 x 256", 1, 256, 256, "bf16", False),
        # A stack of small odd matrices updated in one call (per-head projections).
        _orth("orth 6 x 200 x 333 momentum", 6, 200, 333, "fp32", True),
        # A square weight at the 1B width.
        _orth("orth 2048 x 2048 momentum", 1, 2048, 2048, "bf16", True),
        # A square weight at the 8B width, fp32 gradients as this framework's dW.
        _orth("orth 4096 x 4096 momentum", 1, 4096, 4096, "fp32", True),
        # A tall one: an up projection, four times the 8B width.
        _orth("orth 16384 x 4096", 1, 16384, 4096, "bf16", False),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm; often a multiple of a power of two, often odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    if kind == 0:
        step = max(1, 1 << max(0, v.bit_length() - 3))
        v = v // step * step
    elif kind == 1:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    if rng.random() < 0.6:
        d = _spread(rng, 64, 16384)
        N = _spread(rng, 1, min(16384, (1 << 27) // d))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        w_dtype = rng.choice((dtype, "fp32"))
        post = rng.random() < 0.7
        gate = rng.choice(("none", "shared", "token"))
        divisors = [g for g in range(1, min(N, 64) + 1) if N % g == 0]
        return _norm(None, N, d, dtype, w_dtype, post, gate, rng.random() < 0.85, rng.random() < 0.6,
                     rng.choice(divisors))
    m = _spread(rng, 16, 8192)
    n = _spread(rng, 16, 8192)
    while min(m, n) ** 2 * max(m, n) > 1 << 37:
        m, n = max(16, m * 3 // 4), max(16, n * 3 // 4)
    most = max(1, min(8, (1 << 37) // (min(m, n) ** 2 * max(m, n)), (1 << 25) // (m * n)))
    return _orth(None, rng.randint(1, most), m, n, rng.choice(("bf16", "fp32")), rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dt = DTYPES[case["dtype"]]
    if case["op"] == "orth":
        b, m, n = case["batch"], case["m"], case["n"]
        # A gradient: a few strong directions over a broad floor of noise.
        k = max(1, min(m, n) // 16)
        strength = torch.arange(1, k + 1, device="cuda", dtype=torch.float32).rsqrt()
        s = {"grad": normal(b, m, n)}
        s["grad"].baddbmm_(normal(b, m, k) * strength, normal(b, k, n), beta=0.5)
        s["grad"] = s["grad"].mul_(1e-3).to(dt)
        s["momentum"] = normal(b, m, n).mul_(5e-4) if case["momentum"] else None
        return {"case": dict(case), **s}
    N, d = case["N"], case["d"]
    wt = DTYPES[case["w_dtype"]]
    # A residual stream with a few loud channels, the output of a block, weights around 1.
    loud = 1.0 + 7.0 * (torch.rand(d, generator=g, device="cuda") < 0.01)
    s = {"x": (normal(N, d) * loud).to(dt), "y": (normal(N, d) * 0.7).to(dt)}
    s["w_post"] = (1 + 0.2 * normal(d)).to(wt) if case["post"] else None
    s["w_pre"] = (1 + 0.2 * normal(d)).to(wt) if case["pre"] else None
    rows = {"none": 0, "shared": case["groups"], "token": N}[case["gate"]]
    s["gate"] = (0.5 + 0.3 * normal(rows, d)).to(dt) if rows else None
    if case["train"]:
        s["d_residual"] = (1e-2 * normal(N, d)).to(dt)
        s["d_hidden"] = (1e-2 * normal(N, d)).to(dt) if case["pre"] else None
    return {"case": dict(case), **s}


#: The residual and block scales of every case: a stream scaled down a little, a block's output up.
RESIDUAL_SCALE, BLOCK_SCALE = 0.75, 1.25


def _run_own(s):
    from lm_head_loss_streaming_b200 import block_norm_bwd, block_norm_fwd, orthogonalize

    if s["case"]["op"] == "orth":
        out = orthogonalize(s["grad"], momentum=s["momentum"], beta=BETA, nesterov=True, steps=STEPS,
                            coefficients=COEFFICIENTS, eps=ORTH_EPS)
        return {"update": out, "momentum": s["momentum"]}
    fwd = block_norm_fwd(s["x"], s["y"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                         residual_scale=RESIDUAL_SCALE, block_scale=BLOCK_SCALE, eps=EPS)
    got = {"residual": fwd.residual, "hidden": fwd.hidden}
    if s["case"]["train"]:
        grads = block_norm_bwd(fwd, s["x"], s["y"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                               d_residual=s["d_residual"], d_hidden=s["d_hidden"])
        got |= {"dx": grads.dx, "dy": grads.dy, "dgate": grads.dgate, "dw_pre": grads.dw_pre,
                "dw_post": grads.dw_post}
    return got


def _plain_orth(s):
    u = s["grad"].float()
    if s["momentum"] is not None:
        s["momentum"].copy_(BETA * s["momentum"] + (1 - BETA) * u)
        u = BETA * s["momentum"] + (1 - BETA) * u
    tall = u.shape[1] > u.shape[2]
    x = u / (u.square().sum(dim=(1, 2), keepdim=True).sqrt() + ORTH_EPS)
    if tall:
        x = x.transpose(1, 2)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        A = x @ x.transpose(1, 2)
        x = a * x + (b * A + c * (A @ A)) @ x
    if tall:
        x = x.transpose(1, 2)
    return {"update": x.to(torch.bfloat16).contiguous(), "momentum": s["momentum"]}


def _spread_gate(gate, N):
    """The gate's rows over the N rows that they stand for."""
    return gate.repeat_interleave(N // gate.shape[0], dim=0)


def _plain_norm(s):
    case, dt = s["case"], s["x"].dtype
    N, d = s["x"].shape
    x, y = s["x"].float(), s["y"].float()
    gate = 1.0 if s["gate"] is None else _spread_gate(s["gate"].float(), N)
    post, pre = s["w_post"] is not None, s["w_pre"] is not None
    wq = s["w_post"].float() if post else 1.0
    iy = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if post else 1.0
    yn = y * iy
    r = RESIDUAL_SCALE * x + BLOCK_SCALE * gate * (yn * wq)
    got = {"residual": r.to(dt), "hidden": None}
    if pre:
        wp = s["w_pre"].float()
        ir = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
        rn = r * ir
        got["hidden"] = (rn * wp).to(dt)
    if not case["train"]:
        return got
    g, dw_pre, dw_post, dgate = s["d_residual"].float(), None, None, None
    if pre:
        dh = s["d_hidden"].float()
        dw_pre = (dh * rn).sum(0)
        t = dh * wp
        g = g + ir * (t - rn * (t * rn).mean(1, keepdim=True))
    dv = BLOCK_SCALE * gate * g
    if s["gate"] is not None:
        dgate = BLOCK_SCALE * (yn * wq) * g
        dgate = dgate.view(s["gate"].shape[0], -1, d).sum(1).to(s["gate"].dtype)
    dy = dv
    if post:
        dw_post = (dv * yn).sum(0)
        t = dv * wq
        dy = iy * (t - yn * (t * yn).mean(1, keepdim=True))
    got |= {"dx": (RESIDUAL_SCALE * g).to(dt), "dy": dy.to(dt), "dgate": dgate, "dw_pre": dw_pre,
            "dw_post": dw_post}
    return got


def run(state):
    if own:
        return _run_own(state)
    return _plain_orth(state) if state["case"]["op"] == "orth" else _plain_norm(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orth":
        u, mom = s["grad"].double(), None
        if s["momentum"] is not None:
            mom = BETA * s["momentum"].double() + (1 - BETA) * u
            u = BETA * mom + (1 - BETA) * u
        # The polynomial's factors commute with the Gram matrix, so the iteration can run on it:
        # X_5 = X_0 Q with Q the product of the factors P(G_i), G_{i+1} = P G_i P.
        u = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + ORTH_EPS)
        left = u.shape[1] <= u.shape[2]
        gram = u @ u.mT if left else u.mT @ u
        eye = torch.eye(gram.shape[1], dtype=torch.float64, device="cuda")
        q = eye.expand_as(gram)
        a, b, c = COEFFICIENTS
        for _ in range(STEPS):
            p = a * eye + b * gram + c * (gram @ gram)
            q = p @ q
            gram = p @ gram @ p
        return {"update": q @ u if left else u @ q, "momentum": mom}

    # The norms as autograd sees them, in 64 bits, a slab of rows at a time.
    N, d = case["N"], case["d"]
    per = N // s["gate"].shape[0] if s["gate"] is not None else 1
    slab = max(1, (1 << 25) // d // per) * per
    leaf = {k: s[k].double().requires_grad_(case["train"]) for k in ("w_pre", "w_post", "gate") if s[k] is not None}
    rows = {k: [] for k in ("residual", "hidden", "dx", "dy")}
    for at in range(0, N, slab):
        n = slice(at, min(N, at + slab))
        x = s["x"][n].double().requires_grad_(case["train"])
        y = s["y"][n].double().requires_grad_(case["train"])
        v = y
        if "w_post" in leaf:
            v = leaf["w_post"] * y / (y.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
        if "gate" in leaf:
            k = torch.arange(n.start, n.stop, device="cuda") // per
            v = v * leaf["gate"][k]
        r = RESIDUAL_SCALE * x + BLOCK_SCALE * v
        total = 0
        if case["train"]:
            total = (r * s["d_residual"][n].double()).sum()
        rows["residual"].append(r.detach())
        if "w_pre" in leaf:
            h = leaf["w_pre"] * r / (r.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
            rows["hidden"].append(h.detach())
            if case["train"]:
                total = total + (h * s["d_hidden"][n].double()).sum()
        if case["train"]:
            total.backward()
            rows["dx"].append(x.grad)
            rows["dy"].append(y.grad)
    got = {k: torch.cat(v) if v else None for k, v in rows.items()}
    if not case["train"]:
        return {"residual": got["residual"], "hidden": got["hidden"]}
    grad = {k: t.grad for k, t in leaf.items()}
    return {**got, "dgate": grad.get("gate"), "dw_pre": grad.get("w_pre"), "dw_post": grad.get("w_post")}


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "orth":
        b, m, n = case["batch"], case["m"], case["n"]
        k, l = min(m, n), max(m, n)
        # The symmetric products at half their full cost: k k l for A, k k k for A^2; 2 k k l for the update.
        return {"bytes": b * m * n * (e + 2 + (8 if case["momentum"] else 0)),
                "flops": STEPS * b * (3 * k * k * l + k * k * k)}
    N, d, w = case["N"], case["d"], BYTES[case["w_dtype"]]
    gate = {"none": 0, "shared": case["groups"], "token": N}[case["gate"]] * d
    weights = d * (case["post"] + case["pre"])
    size = N * d * e * (3 + case["pre"]) + gate * e + weights * w
    flops = N * d * (4 + 4 * case["post"] + 4 * case["pre"])
    if case["train"]:
        # d_residual and d_hidden in, dx and dy out, the gate's and the weights' gradients out.
        size += N * d * e * (3 + case["pre"]) + gate * e + weights * 4
        flops += N * d * (6 + 8 * case["post"] + 8 * case["pre"])
    return {"bytes": size, "flops": flops}
