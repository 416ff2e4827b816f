"""``orthogonalize`` against the Newton-Schulz iteration in 64 bits; the tolerances are those of
``orth_util.tolerance``.  The momentum is three fp32 roundings away from its formula:
4 * 2^-24 of its terms' magnitudes."""

import pytest
import torch

from lm_head_loss_streaming_b200 import orthogonalize, orthogonalize_workspace_bytes
from orth_util import STANDARD, iterate, spectrum, tolerance

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROWS = [STANDARD] * 5


def check(got, u, rows=ROWS, eps=1e-7):
    """One matrix's result against the exact iteration on u."""
    exact = iterate(u, rows, eps)
    emulated = iterate(u, rows, eps, formats=True)
    assert got.dtype == BF and got.shape == u.shape
    off = torch.linalg.vector_norm(got.double() - exact) / torch.linalg.vector_norm(exact)
    tol = tolerance(exact, emulated)
    assert off.item() <= tol, (off.item(), tol)


# One element, rows and columns, below / at / above the 64-wide K block, the 128- and 256-wide
# tiles, odd sizes, several tiles with ragged ends, very wide and very tall.
SHAPES = [(1, 1), (1, 9), (9, 1), (5, 3), (16, 16), (33, 64), (64, 33), (65, 127), (128, 128),
          (129, 257), (128, 256), (256, 128), (200, 129), (130, 250), (255, 256), (256, 256),
          (257, 255), (384, 500), (700, 300), (520, 777),
          (1024, 1024), (1100, 900), (40, 5000), (5000, 40)]


@pytest.mark.parametrize("dtype", [BF, F32, HF])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype):
    g = spectrum(*shape, "noise", sum(shape)).to(dtype)
    check(orthogonalize(g), g)


@pytest.mark.parametrize("kind", ["decay", "bad", "spikes", "rank"])
@pytest.mark.parametrize("shape", [(256, 256), (200, 900), (900, 200)])
def test_spectra(shape, kind):
    g = (1e-3 * spectrum(*shape, kind, 1)).to(F32)
    check(orthogonalize(g), g)


def test_diagonal_and_repeated_rows():
    g = torch.eye(300, device="cuda") * 1e-4
    check(orthogonalize(g), g)
    g = torch.ones(130, 70, device="cuda")      # rank one, every entry of A alike
    check(orthogonalize(g), g)


@pytest.mark.parametrize("batch,m,n", [(1, 64, 64), (200, 256, 130), (7, 30, 250), (3, 100, 257), (5, 257, 100), (2, 600, 600),
                                       (80, 40, 30)])
def test_stacks(batch, m, n):
    g = torch.stack([(10.0 ** (i % 5 - 2)) * spectrum(m, n, "noise", i) for i in range(batch)])
    g = g.to(F32)
    got = orthogonalize(g)
    for i in range(batch):
        check(got[i], g[i])
    lone = orthogonalize(g[batch - 1])
    assert torch.equal(lone, got[batch - 1])    # a matrix's result does not depend on the stack


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_momentum(dtype, nesterov):
    b, m, n, beta = 2, 150, 203, 0.9
    mom = torch.stack([spectrum(m, n, "noise", 10 + i) for i in range(b)]).to(F32)
    for step in range(3):
        g = torch.stack([spectrum(m, n, "decay", 20 + step + i) for i in range(b)]).to(dtype)
        want = beta * mom.double() + (1 - beta) * g.double()
        size = beta * mom.double().abs() + (1 - beta) * g.double().abs()
        got = orthogonalize(g, momentum=mom, beta=beta, nesterov=nesterov)
        assert ((mom.double() - want).abs() <= 4 * 2.0 ** -24 * size).all()
        u = beta * mom.double() + (1 - beta) * g.double() if nesterov else mom.double()
        for i in range(b):
            check(got[i], u[i])


def test_beta_ends():
    g, mom = spectrum(70, 80, "noise", 1).to(F32), spectrum(70, 80, "noise", 2).to(F32)
    old = mom.clone()
    check(orthogonalize(g, momentum=mom, beta=1.0, nesterov=False), old)
    assert torch.equal(mom, old)
    orthogonalize(g, momentum=mom, beta=0.0)
    assert torch.equal(mom, g)


def test_strided_gradients():
    wide = spectrum(100, 400, "noise", 3).to(BF)
    g = wide[:, 7:7 + 301]
    check(orthogonalize(g), g)
    stack = spectrum(90, 500, "noise", 4).to(F32).reshape(3, 30, 500)[:, ::2, :111]
    got = orthogonalize(stack)
    for i in range(3):
        check(got[i], stack[i])
    assert torch.equal(got, orthogonalize(stack.contiguous()))


@pytest.mark.parametrize("steps,rows", [
    (1, [STANDARD]), (3, [STANDARD] * 3), (6, [(1.5, -0.5, 0.0)] * 6), (1, [(1.0, 0.0, 0.0)]),
    (4, [(2.0, -1.5, 0.5), STANDARD, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)])])
def test_coefficients(steps, rows):
    g = spectrum(140, 170, "decay", 5).to(F32)
    check(orthogonalize(g, steps=steps, coefficients=rows), g, rows)
    if len(set(rows)) == 1:
        assert torch.equal(orthogonalize(g, steps=steps, coefficients=rows[0]),
                           orthogonalize(g, steps=steps, coefficients=rows))


def test_result_is_orthogonal_enough():
    """Independent of the reference: the singular values end within the polynomial's band."""
    g = spectrum(200, 300, "noise", 6).to(BF)
    s = torch.linalg.svdvals(orthogonalize(g).double())
    # p maps [0.01, 1] into [0.68, 1.21] in five steps; noise of this shape starts above 0.01.
    assert s.max() <= 1.22 and s.min() >= 0.66


def test_zeros_nan_and_neighbours():
    g = torch.stack([spectrum(60, 70, "noise", i) for i in range(4)]).to(F32)
    alone = orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    got = orthogonalize(g)
    assert not got[1].any() and got[2].isnan().all()
    wide = torch.stack([spectrum(60, 270, "noise", i) for i in range(3)]).to(F32)
    wide[1, 5, 260] = float("nan")
    many = orthogonalize(wide)
    assert many[1].isnan().all() and torch.equal(many[2], orthogonalize(wide[2]))
    assert torch.equal(got[0], alone[0]) and torch.equal(got[3], alone[3])
    g[2, 3, 4] = float("inf")
    assert orthogonalize(g)[2].isnan().all()


def test_scale_range():
    """Gradients near the ends of fp32's and bf16's range, whose squares leave it."""
    base = spectrum(64, 96, "noise", 7)
    for scale, dtype in ((1e-4, F32), (1e30, F32), (1e30, BF), (1e4, HF)):
        g = (scale * base).to(dtype)
        check(orthogonalize(g), g)
    g = (1e-30 * base).to(F32)
    check(orthogonalize(g, eps=1e-36), g, eps=1e-36)


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 4)):
        assert orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def test_given_buffers_streams_and_graph():
    g = spectrum(300, 200, "noise", 8).to(BF)
    want = orthogonalize(g)
    ws = torch.empty(orthogonalize_workspace_bytes(1, 300, 200), dtype=torch.uint8, device="cuda")
    out = torch.empty(300, 200, dtype=BF, device="cuda")
    assert orthogonalize(g, out=out, workspace=ws) is out and torch.equal(out, want)
    odd = torch.empty(300 * 200 + 1, dtype=BF, device="cuda")[1:].view(300, 200)
    assert torch.equal(orthogonalize(g, out=odd), want)     # an output off 16-byte alignment
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = orthogonalize(g)
        twin = orthogonalize(g.float())
    here = orthogonalize(g)                                  # two calls at once
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, want) and torch.equal(here, want) and torch.equal(twin, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonalize(g)
    g.copy_(spectrum(300, 200, "noise", 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, orthogonalize(g))


def test_momentum_graph_advances_each_replay():
    g, mom = spectrum(80, 90, "noise", 1).to(F32), torch.zeros(80, 90, device="cuda")
    orthogonalize(g, momentum=mom.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonalize(g, momentum=mom)
    twin = torch.zeros_like(mom)
    for _ in range(3):
        graph.replay()
        want = orthogonalize(g, momentum=twin)
        torch.cuda.synchronize()
        assert torch.equal(mom, twin) and torch.equal(got, want)


@pytest.mark.parametrize("shape", [(2, 600, 300), (260, 1030)])
def test_same_bits_each_time(shape):
    g = torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    want = orthogonalize(g)
    for _ in range(5):
        assert torch.equal(orthogonalize(g), want)


@pytest.mark.parametrize("shape", [(200, 150), (300, 200), (600, 1300)])
def test_wait_runs_out_reports_timeout_and_the_next_call_is_right(shape):
    from lm_head_loss_streaming_b200 import _lib
    g = spectrum(*shape, "noise", 11).to(BF)
    ws = torch.empty(orthogonalize_workspace_bytes(1, *shape), dtype=torch.uint8, device="cuda")
    want = orthogonalize(g)
    assert _lib.slm_debug_set(1, 100_000_000) == 0   # ~0.05-0.1 s per wait
    try:
        orthogonalize(g, workspace=ws)
        st = _lib.slm_device_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    finally:
        assert _lib.slm_debug_set(0, 0) == 0
    assert st == 7, _lib.status_string(st)   # SLM_ERR_TIMEOUT
    assert torch.equal(orthogonalize(g, workspace=ws), want)
    st = _lib.slm_device_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0


def test_many_calls_on_several_streams():
    """Calls whose blocks wait for one another, at once on four streams."""
    gs = [spectrum(400 + 64 * i, 900 - 50 * i, "noise", i).to(F32) for i in range(4)]
    want = [orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    got = [[] for _ in gs]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(orthogonalize(gs[i]))
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(g, want[i]) for g in got[i])


# Few tiles over a long side: the Gram product's long axis is shared out.  Parts that end inside a
# 64-wide K block, one or several tiles, one or several matrices, with and without room for X's
# tiles in tensor memory.
@pytest.mark.parametrize("batch,m,n", [(1, 64, 2048), (1, 2049, 64), (1, 300, 8192), (1, 8191, 300),
                                       (2, 130, 4100), (3, 4097, 257), (8, 100, 4000),
                                       (1, 520, 5001), (1, 5003, 1000), (1, 3, 20000)])
def test_long_axis_in_parts(batch, m, n):
    g = torch.stack([spectrum(m, n, "noise", 7 + i) for i in range(batch)]).to(BF)
    got = orthogonalize(g)
    for i in range(batch):
        check(got[i], g[i])
    assert torch.equal(got, orthogonalize(g))


def test_long_axis_in_parts_wait_runs_out():
    test_wait_runs_out_reports_timeout_and_the_next_call_is_right((300, 6000))


def test_writes_in_place_are_known_to_autograd():
    g = spectrum(30, 40, "noise", 1).to(F32)
    mom, out = torch.zeros_like(g), torch.empty(30, 40, dtype=BF, device="cuda")
    before = mom._version, out._version
    orthogonalize(g, momentum=mom, out=out)
    assert mom._version > before[0] and out._version > before[1]


@pytest.mark.parametrize("m,n", [(40, 64), (40, 300)])
@pytest.mark.parametrize("size", [1e-37, 2e38])
def test_scales_beyond_fp32(m, n, size):
    """||u|| whose reciprocal, or its product with the kernels' scale, leaves fp32."""
    g = spectrum(m, n, "noise", 3)
    g = (g / g.abs().max() * size).to(F32)
    u = g.where(g.abs() >= 2.0 ** -126, 0)     # subnormal elements count as zeros
    check(orthogonalize(g, eps=2e-38), u, eps=2e-38)
    assert not orthogonalize(torch.zeros_like(g), eps=2e-38).any()
