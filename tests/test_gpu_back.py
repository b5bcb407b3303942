"""w4a16_lm_head_backward, the product back through a packed weight, against
its 64-bit form: sizes around every tile, types, special values, empty calls,
pieces, streams, graphs."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._train import back_reference, hidden, stored, weight, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def gradient(M, N, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(3.0 * torch.randn(M, 1, generator=g))  # tokens differ by several binades
    return (1e-5 * size * torch.randn(M, N, generator=g)).to(dtype).cuda()


def check(dy, w, W, **kw):
    got = nv.w4a16_lm_head_backward(dy, *w, **kw)
    want, tol = back_reference(dy, W)
    within(got, want, stored(want, tol, got.dtype))
    return got


# token tiles 16 .. 48 (deep rings), 64 .. 128; weight rows around a stage of
# 256; columns around tiles of 128 and pairs of 256, staged rows where K % 256 !=
# 0; many tiles; stages of 128 rows, where gradient and weight are large; pairs of
# CTAs, where 256 x 256 tiles fill 76 of them three times, with and without tiles
# that are split, or once with more than 65536 rows
SHAPES = [(1, 1, 16), (1, 700, 48), (3, 255, 144), (16, 256, 128), (17, 257, 256), (33, 1000, 272),
          (48, 64, 1024), (49, 513, 400), (64, 2000, 512), (100, 31, 96), (127, 300, 640),
          (128, 256, 256), (129, 4099, 1008), (255, 77, 128), (256, 511, 384), (257, 1500, 512),
          (300, 640, 2064), (700, 2049, 272),
          (512, 300, 9728), (500, 1111, 10000), (1000, 300, 5120),
          (700, 40001, 272), (99, 100_100, 640),
          (512, 300, 29184), (500, 1111, 29456), (1000, 300, 15104), (1280, 65664, 3904)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(M, N, K, dtype):
    w, W = weight(N, K, seed=M + N + K)
    check(gradient(M, N, M * N, dtype), w, W)


@pytest.mark.parametrize("M", [5, 130, 520])
def test_fp32_result(M):
    w, W = weight(900, 304, seed=M)
    got = check(gradient(M, 900, M, torch.bfloat16), w, W, out_dtype=torch.float32)
    assert got.dtype == torch.float32
    out = torch.empty(M, 304, device="cuda")
    assert nv.w4a16_lm_head_backward(gradient(M, 900, M, torch.bfloat16), *w, out=out) is out
    assert torch.equal(out, got)


def test_uint8_scales_and_given_workspace():
    w, W = weight(300, 272, seed=1)
    dy = gradient(40, 300, 2, torch.float32)
    n = nv.w4a16_lm_head_backward_workspace_bytes(40, 300, 272)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    got = check(dy, (w[0], w[1].view(torch.uint8), w[2]), W, workspace=ws[:n])
    assert nv.nvfp4_read_device_status(ws) == nv.Status.OK
    assert bool((ws[n:] == 255).all())
    assert torch.equal(got, nv.w4a16_lm_head_backward(dy, *w))


@pytest.mark.parametrize("M", [20, 300])
def test_special_values_stay_in_their_token(M):
    w, W = weight(500, 256, seed=3)
    dy = gradient(M, 500, 4, torch.float32)
    dy[1] = 0.0
    dy[2] = 1e-38 * torch.sign(dy[2])      # near the smallest normal number
    dy[3] = 1e36 * torch.sign(dy[3])
    ok = torch.ones(M, dtype=torch.bool)
    dy[4, 7], dy[5, 499] = float("nan"), float("inf")
    ok[4:6] = False
    got = nv.w4a16_lm_head_backward(dy, *w, out_dtype=torch.float32)
    assert not bool(torch.isfinite(got[4]).any()) and not bool(torch.isfinite(got[5]).any())
    want, tol = back_reference(dy[ok], W)
    within(got[ok], want, stored(want, tol, torch.float32) + 2.0 ** -126)
    assert bool((got[1] == 0).all())


def test_nan_scale_raises_the_status():
    w, W = weight(500, 512, seed=5)
    scales = w[1].view(torch.uint8).clone()
    scales[321, 17] = 0x7F
    for M in (3, 130, 300):
        ws = torch.empty(nv.w4a16_lm_head_backward_workspace_bytes(M, 500, 512), dtype=torch.uint8,
                         device="cuda")
        got = nv.w4a16_lm_head_backward(gradient(M, 500, 6, torch.bfloat16), w[0], scales, w[2],
                                        workspace=ws)
        assert nv.nvfp4_read_device_status(ws) == nv.Status.ERR_NONFINITE
        bad = torch.zeros(512, dtype=torch.bool)
        bad[17 * 16:18 * 16] = True
        assert bool(torch.isnan(got[:, bad]).all()) and bool(torch.isfinite(got[:, ~bad]).all())


def test_empty():
    w, _ = weight(64, 32, seed=7)
    assert nv.w4a16_lm_head_backward(torch.empty(0, 64, device="cuda"), *w).shape == (0, 32)
    none = (torch.empty(0, 16, dtype=torch.uint8, device="cuda"),
            torch.empty(0, 2, dtype=torch.uint8, device="cuda"), w[2])
    out = torch.full((3, 32), 7.0, device="cuda")
    nv.w4a16_lm_head_backward(torch.empty(3, 0, device="cuda"), *none, out=out)
    assert bool((out == 0).all())


def test_pieces_of_a_long_call():
    """More fp16 gradient than is held at a time: 384 and 44 tokens."""
    N = 600_000
    w, W = weight(N, 16, seed=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(428, N, device="cuda", generator=g).to(torch.bfloat16)
    check(dy, w, W)


def test_rows_behind_the_result_are_left_alone():
    w, W = weight(300, 144, seed=10)
    for M in (5, 100, 260):
        buf = torch.full((M + 40, 144), 3.0, dtype=torch.bfloat16, device="cuda")
        nv.w4a16_lm_head_backward(gradient(M, 300, M, torch.bfloat16), *w, out=buf[:M])
        assert bool((buf[M:] == 3.0).all())


@pytest.mark.parametrize("M", [9, 90, 400])
def test_same_bits_each_time_on_streams_and_in_graphs(M):
    w, W = weight(3000, 528, seed=11)
    dy = gradient(M, 3000, 12, torch.bfloat16)
    first = check(dy, w, W)
    for _ in range(4):
        assert torch.equal(nv.w4a16_lm_head_backward(dy, *w), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = nv.w4a16_lm_head_backward(dy, *w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = nv.w4a16_lm_head_backward(dy, *w)
    new = gradient(M, 3000, 13, torch.bfloat16)
    keep = dy.clone()
    for source in (new, keep):
        dy.copy_(source)
        graph.replay()
        assert torch.equal(held, nv.w4a16_lm_head_backward(source, *w))


def test_logits_carry_the_gradient():
    """w4a16_lm_head on x that requires a gradient."""
    w, W = weight(700, 272, seed=14)
    x = hidden(33, 272, seed=15).requires_grad_(True)
    for dtype in (torch.float32, torch.bfloat16):
        logits = nv.w4a16_lm_head(x, *w, out_dtype=dtype)
        assert logits.requires_grad and logits.dtype == dtype
        g = gradient(33, 700, 16, dtype)
        (dx,) = torch.autograd.grad(logits, x, g)
        want, tol = back_reference(g, W)
        within(dx, want, stored(want, tol, dx.dtype))
    with torch.no_grad():
        assert not nv.w4a16_lm_head(x, *w).requires_grad
    out = torch.empty(33, 700, device="cuda")
    assert nv.w4a16_lm_head(x, *w, out=out) is out and not out.requires_grad
    assert torch.equal(out, nv.w4a16_lm_head(x.detach(), *w))
    # a gradient that is a view (of a sum: one element for all)
    (dx,) = torch.autograd.grad(nv.w4a16_lm_head(x, *w).sum(), x)
    want, tol = back_reference(torch.ones(33, 700, device="cuda"), W)
    within(dx, want, stored(want, tol, dx.dtype))
