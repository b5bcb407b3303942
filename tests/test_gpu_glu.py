"""w4a16_glu and its gradient against their 64-bit forms and against
differences: sizes around every tile, both activations, types, special values,
streams, graphs, autograd."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._train import activation, glu_grad_reference, glu_reference, hidden, stored, weight, within

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def gradient(M, I, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1e-4 * torch.exp(torch.randn(M, 1, generator=g)) * torch.randn(M, I, generator=g)).to(dtype).cuda()


# I around the 64 pairs of a unit, odd ones among them; K with staged rows
SHAPES = [(1, 1, 16), (1, 64, 256), (2, 63, 48), (15, 65, 272), (16, 200, 512), (33, 99, 144),
          (64, 128, 256), (65, 130, 400), (128, 17, 1024), (129, 301, 528), (200, 640, 256),
          (300, 129, 2064), (513, 64, 272)]


@pytest.mark.parametrize("M,I,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(M, I, K, act):
    w, W = weight(2 * I, K, seed=M + I + K)
    x = hidden(M, K, seed=M)
    want, tol = glu_reference(x, W, act)
    for dtype in (torch.bfloat16, torch.float32):
        got = nv.w4a16_glu(x, *w, activation=act, out_dtype=dtype)
        assert got.shape == (M, I) and got.dtype == dtype
        within(got, want, stored(want, tol, dtype), dtype)


@pytest.mark.parametrize("M,I,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward(M, I, K, act, dtype):
    w, W = weight(2 * I, K, seed=M + I + K)
    x, dh = hidden(M, K, seed=M), gradient(M, I, M * I, dtype)
    want, tol = glu_grad_reference(dh, x, W, w[2], act)
    for out in (torch.bfloat16, torch.float32):
        got = nv.w4a16_glu_backward(dh, x, *w, activation=act, out_dtype=out)
        assert got.shape == (M, K) and got.dtype == out
        within(got, want, stored(want, tol, out), out)


def test_backward_is_the_slope_of_forward():
    """Central differences of the 64-bit form along random directions, step
    1e-4 of x: off by 1e-8 of the third derivative and by 1e-11 of rounding,
    far below the kernel's own bound."""
    w, W = weight(2 * 150, 272, seed=1)
    x, dh = hidden(20, 272, seed=2, outliers=0), gradient(20, 150, 3, torch.float32)
    for act in ACTS:
        dx = nv.w4a16_glu_backward(dh, x, *w, activation=act, out_dtype=torch.float32)
        _, tol = glu_grad_reference(dh, x, W, w[2], act)
        g = torch.Generator(device="cuda").manual_seed(4)
        for _ in range(3):
            v = torch.randn(20, 272, device="cuda", generator=g, dtype=torch.float64)

            def f(s):
                gu = (x.double() + s * v) @ W.T
                return (dh.double() * activation(gu[:, :150], act)[0] * gu[:, 150:]).sum(1)

            slope = (f(1e-4) - f(-1e-4)) / 2e-4
            bound = (tol * v.abs()).sum(1) + 1e-5 * (dx.double() * v).abs().sum(1)
            within((dx.double() * v).sum(1), slope, bound)


@pytest.mark.parametrize("M", [7, 260])
@pytest.mark.parametrize("act", ACTS)
def test_large_and_special_values(M, act):
    """Gates far beyond where the exponential ends, and rows with Inf or NaN."""
    w, W = weight(2 * 90, 256, seed=5)
    x = hidden(M, 256, seed=6)
    x[0] = 0.0
    x[1] *= 1e4
    x[2] *= 1e-30
    x[3] *= 1e12
    bad = [4, 5]
    x[4, 3], x[5, 200] = float("inf"), float("nan")
    ok = torch.ones(M, dtype=torch.bool)
    ok[bad] = False
    h = nv.w4a16_glu(x, *w, activation=act, out_dtype=torch.float32)
    want, tol = glu_reference(x[ok], W, act)
    within(h[ok], want, stored(want, tol, torch.float32))
    assert not bool(torch.isfinite(h[bad]).any())
    dh = gradient(M, 90, 7, torch.float32)
    dh[6] = 0.0
    dx = nv.w4a16_glu_backward(dh, x, *w, activation=act, out_dtype=torch.float32)
    want, tol = glu_grad_reference(dh[ok], x[ok], W, w[2], act)
    within(dx[ok], want, stored(want, tol, torch.float32) + 2.0 ** -126)
    assert not bool(torch.isfinite(dx[bad]).any())
    assert bool((dx[6] == 0).all())


def test_a_gradient_that_is_not_finite_stays_in_its_token():
    w, W = weight(2 * 90, 256, seed=5)
    x, dh = hidden(7, 256, seed=6), gradient(7, 90, 7, torch.float32)
    dh[2, 5], dh[3, 89] = float("nan"), float("inf")
    dx = nv.w4a16_glu_backward(dh, x, *w, out_dtype=torch.float32)
    assert not bool(torch.isfinite(dx[2:4]).any())
    ok = [0, 1, 4, 5, 6]
    want, tol = glu_grad_reference(dh[ok], x[ok], W, w[2], "silu")
    within(dx[ok], want, stored(want, tol, torch.float32))


def test_nan_scale_raises_the_status():
    w, _ = weight(2 * 70, 512, seed=8)
    scales = w[1].view(torch.uint8).clone()
    scales[70 + 13, 5] = 0xFF  # an up row
    x, dh = hidden(9, 512, seed=9), gradient(9, 70, 10, torch.bfloat16)
    ws = torch.empty(nv.w4a16_glu_backward_workspace_bytes(9, 70, 512), dtype=torch.uint8, device="cuda")
    h = nv.w4a16_glu(x, w[0], scales, w[2], workspace=ws)
    assert nv.nvfp4_read_device_status(ws) == nv.Status.ERR_NONFINITE
    assert bool(torch.isnan(h[:, 13]).all()) and int(torch.isnan(h).sum()) == 9
    nv.w4a16_glu(x, *w, workspace=ws)
    assert nv.nvfp4_read_device_status(ws) == nv.Status.OK
    nv.w4a16_glu_backward(dh, x, w[0], scales, w[2], workspace=ws)
    assert nv.nvfp4_read_device_status(ws) == nv.Status.ERR_NONFINITE


def test_empty():
    w, _ = weight(64, 32, seed=11)
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    assert nv.w4a16_glu(x, *w).shape == (0, 32)
    assert nv.w4a16_glu_backward(torch.empty(0, 32, device="cuda"), x, *w).shape == (0, 32)
    none = (torch.empty(0, 16, dtype=torch.uint8, device="cuda"),
            torch.empty(0, 2, dtype=torch.uint8, device="cuda"), w[2])
    x = hidden(3, 32, seed=12)
    assert nv.w4a16_glu(x, *none).shape == (3, 0)
    dx = nv.w4a16_glu_backward(torch.empty(3, 0, device="cuda"), x, *none)
    assert bool((dx == 0).all())


def test_results_and_their_neighbours():
    w, W = weight(2 * 99, 144, seed=13)
    for M in (5, 100, 260):
        x, dh = hidden(M, 144, seed=M), gradient(M, 99, M, torch.bfloat16)
        h = torch.full((M + 30, 99), 3.0, dtype=torch.bfloat16, device="cuda")
        assert nv.w4a16_glu(x, *w, out=h[:M]).data_ptr() == h.data_ptr()
        dx = torch.full((M + 30, 144), 3.0, device="cuda")
        nv.w4a16_glu_backward(dh, x, *w, out=dx[:M])
        assert bool((h[M:] == 3.0).all()) and bool((dx[M:] == 3.0).all())
        assert torch.equal(h[:M], nv.w4a16_glu(x, *w))
        assert torch.equal(dx[:M], nv.w4a16_glu_backward(dh, x, *w, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [9, 90, 400])
def test_same_bits_each_time_on_streams_and_in_graphs(M):
    w, W = weight(2 * 500, 528, seed=14)
    x, dh = hidden(M, 528, seed=15), gradient(M, 500, 16, torch.bfloat16)

    def both(stream=None):
        return nv.w4a16_glu(x, *w, stream=stream), nv.w4a16_glu_backward(dh, x, *w, stream=stream)

    first = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(both(), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(other, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (17, 18):
        x.copy_(hidden(M, 528, seed))
        dh.copy_(gradient(M, 500, seed, torch.bfloat16))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, both()))


@pytest.mark.parametrize("act", ACTS)
def test_graph(act):
    w, W = weight(2 * 70, 272, seed=19)
    x = hidden(12, 272, seed=20).requires_grad_(True)
    h = nv.w4a16_glu(x, *w, activation=act)
    assert torch.equal(h.detach(), nv.w4a16_glu(x.detach(), *w, activation=act))
    g = gradient(12, 70, 21, torch.bfloat16)
    (dx,) = torch.autograd.grad(h, x, g, retain_graph=True)
    assert torch.equal(dx, nv.w4a16_glu_backward(g, x.detach(), *w, activation=act))
    (dx,) = torch.autograd.grad(h.float().sum(), x)
    want, tol = glu_grad_reference(torch.ones(12, 70, device="cuda"), x.detach(), W, w[2], act)
    within(dx, want, stored(want, tol, dx.dtype))
    with torch.no_grad():
        assert not nv.w4a16_glu(x, *w).requires_grad
