"""w4a16_cross_entropy and its gradient against their 64-bit forms and against
differences: sizes around every tile, targets of every kind, logits that move
the reference, special values, pieces, streams, graphs, autograd."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._operators import dequant
from tests._train import entropy_grad_reference, entropy_reference, hidden, stored, weight, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(M, N, K, seed, std=0.05, spread=20.0):
    """Hidden states whose targets are anything from unlikely to all but
    certain; some positions without a target."""
    w, W = weight(N, K, seed, std)
    g = torch.Generator().manual_seed(seed + 1)
    t = torch.randint(0, N, (M,), generator=g)
    pull = spread * torch.rand(M, 1, generator=g)
    rows = W[t.cuda()]
    x = torch.randn(M, K, generator=g).cuda() + pull.cuda() * rows / (rows * rows).sum(1, keepdim=True)
    t[torch.rand(M, generator=g) < 0.15] = -100
    if M > 6:
        t[M // 2] = N          # outside as well
        t[M // 3] = N - 1
        t[M - 1] = 0
    return x.to(torch.bfloat16), t.cuda(), w, W


def check(x, t, w, W, a=None, b=None, stream=None):
    M = x.shape[0]
    r = entropy_reference(x, W, t)
    loss, lse = nv.w4a16_cross_entropy(x, *w, t)
    within(lse, r["lse"], r["lse_tol"], "lse")
    within(loss, r["loss"], r["loss_tol"], "loss")
    loss2, lse2, mean = nv.w4a16_cross_entropy(x, *w, t, with_mean=True)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    within(mean, r["mean"], r["mean_tol"], "mean")
    g = torch.Generator().manual_seed(M)
    a = torch.randn(M, generator=g).cuda() if a is None else a
    b = 0.3 * torch.randn(M, generator=g).cuda() if b is None else b
    for out in (torch.bfloat16, torch.float32):
        for gb in (b, None):
            dx = nv.w4a16_cross_entropy_backward(mean, *w, t, loss, a, gb, out_dtype=out)
            want, tol = entropy_grad_reference(r, W, a, torch.zeros_like(b) if gb is None else gb)
            within(dx, want, stored(want, tol, out), (out, gb is None))
    return loss, lse, mean


# token tiles and pairs as in the product back; vocabularies around a unit of
# 128, a group of 32 and a stage of 256 rows; sums of the logits in one part and
# in several (K above 1792)
SHAPES = [(1, 1, 16), (1, 2, 32), (1, 33, 256), (2, 128, 272), (5, 129, 48), (16, 300, 512),
          (17, 1000, 144), (49, 257, 1552), (64, 700, 272), (100, 95, 1024), (128, 513, 256),
          (130, 2000, 1616), (256, 384, 144), (300, 1111, 528), (520, 4099, 272), (40, 800, 3328),
          (512, 700, 9984)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sizes(M, N, K):
    check(*make(M, N, K, seed=M + N + K))


@pytest.mark.parametrize("M", [6, 140, 300])
def test_units_that_are_cut_between_ctas(M):
    """More units than SMs, so that some are cut in the k direction."""
    check(*make(M, 128 * 170 + 5, 528, seed=M))


@pytest.mark.parametrize("M", [3, 130])
def test_certain_targets_keep_their_small_loss(M):
    """1 - p down to 1e-12: the loss is not a difference of large numbers."""
    x, t, w, W = make(M, 900, 256, seed=7, spread=60.0)
    loss, _, _ = check(x, t, w, W)
    assert bool((loss[t >= 0] < 1e-9).any()) and bool((loss[(t >= 0) & (t < 900)] > 0).all())


def test_references_that_rise_late():
    """The largest logit but the target's in the last rows of the vocabulary,
    higher and higher above the rest: most groups were stored at a lower
    reference.  Also all logits equal, and far below 0."""
    M, N, K = 64, 40_000, 256
    w, W = weight(N, K, seed=9)
    g = torch.Generator().manual_seed(10)
    x = torch.randn(M, K, generator=g).cuda()
    rows = W[N - 1 - torch.arange(M).cuda()]
    x += torch.linspace(0, 90, M)[:, None].cuda() * rows / (rows * rows).sum(1, keepdim=True)
    x[5] = 0.0
    x = x.to(torch.bfloat16)
    t = torch.randint(0, N, (M,), generator=g).cuda()
    first = check(x, t, w, W)
    for _ in range(5):
        again = nv.w4a16_cross_entropy(x, *w, t, with_mean=True)
        assert all(torch.equal(p, q) for p, q in zip(again, first))


def test_large_logits():
    """Logits of thousands (one row has all the mass), and of 1e30."""
    x, t, w, W = make(40, 700, 256, seed=11)
    check((x.float() * 300).to(torch.bfloat16), t, w, W)
    loss, lse, mean = nv.w4a16_cross_entropy((x.float() * 1e30).to(torch.bfloat16), *w, t, with_mean=True)
    z = (x.float() * 1e30).to(torch.bfloat16).double() @ W.T
    within(lse, z.amax(1), 1e-5 * z.abs().amax(1))
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(mean).all())


@pytest.mark.parametrize("M", [5, 140])
@pytest.mark.parametrize("low", [2, 3, 5, 9, 17, 30, 36, 200, 3000])
def test_logits_far_below_zero(M, low):
    """Every logit around -low: below and above where one reference ends.  The
    mean keeps its accuracy relative to itself."""
    N, K = 700, 256
    rng = torch.Generator().manual_seed(low)
    packed = torch.randint(0, 8, (N, K // 2), generator=rng) * 17  # two equal positive codes
    scales = (40 + 400 * torch.rand(N, K // 16, generator=rng)).to(torch.float8_e4m3fn)
    W = dequant(packed.to(torch.uint8), scales, torch.tensor(1e-4)).cuda()
    w = packed.to(torch.uint8).cuda(), scales.cuda(), torch.tensor([1e-4]).cuda()
    x = (-low / W.sum(1).mean() * (1 + 0.05 * torch.randn(M, K, generator=rng).cuda())).to(torch.bfloat16)
    t = torch.randint(0, N, (M,), generator=rng).cuda()
    t[1] = -1
    _, _, mean = check(x, t, w, W)
    r = entropy_reference(x, W, t)
    # fp16's 2^-11 of each probability and its sums, and exp(z - lse), off by as
    # much as z and lse are: z's error is that of 256 products, each sum of 16 of
    # them truncated by up to 2^-23 of it (3000 / 2^19 = 0.006 for the last case)
    # (a column that the likely rows leave at 0 has only terms far below the
    # largest, each kept to 2^-23 of that, which is at most 1)
    rel = 2.0 ** -10 + 2 * r["lse_tol"][:, None]
    assert bool(((mean - r["mean"]).abs() <= rel * r["mean"].abs() + 2.0 ** -23 * W.abs().sum(0)).all())


@pytest.mark.parametrize("M", [12, 260])
def test_special_values_stay_in_their_token(M):
    x, t, w, W = make(M, 600, 256, seed=12)
    x[1] = 0.0
    x[3, 5], x[4, 77] = float("nan"), float("inf")
    t[3], t[4] = 17, -1
    ok = torch.ones(M, dtype=torch.bool)
    ok[3:5] = False
    got = nv.w4a16_cross_entropy(x, *w, t, with_mean=True)
    assert bool(torch.isnan(got[1][3:5]).all()) and bool(torch.isnan(got[0][3]))
    assert bool(torch.isnan(got[2][3:5]).all())
    r = entropy_reference(x[ok], W, t[ok])
    for v, name in zip(got, ("loss", "lse", "mean")):
        within(v[ok], r[name], r[name + "_tol"], name)
    # a position that counts nowhere has gradient 0, whatever it holds
    a = torch.ones(M, device="cuda")
    dx = nv.w4a16_cross_entropy_backward(got[2], *w, t, got[0], a)
    assert bool((dx[4] == 0).all()) and bool(torch.isnan(dx[3]).all())
    # nor has one whose gradients are 0: a masked position with a target
    for b in (None, torch.zeros(M, device="cuda")):
        a[3] = 0.0
        dx = nv.w4a16_cross_entropy_backward(got[2], *w, t, got[0], a, b)
        assert bool((dx[3:5] == 0).all()) and bool(torch.isfinite(dx).all())


def test_nan_scale_raises_the_status():
    x, t, w, W = make(9, 600, 512, seed=13)
    scales = w[1].view(torch.uint8).clone()
    scales[599, 3] = 0x7F
    ws = torch.empty(nv.w4a16_cross_entropy_workspace_bytes(9, 600, 512, True), dtype=torch.uint8,
                     device="cuda")
    loss, lse, _ = nv.w4a16_cross_entropy(x, w[0], scales, w[2], t, with_mean=True, workspace=ws)
    assert nv.nvfp4_read_device_status(ws) == nv.Status.ERR_NONFINITE
    assert bool(torch.isnan(lse).all())
    nv.w4a16_cross_entropy(x, *w, t, workspace=ws)
    assert nv.nvfp4_read_device_status(ws) == nv.Status.OK


def test_empty_and_given_workspace():
    x, t, w, W = make(40, 300, 144, seed=14)
    loss, lse, mean = nv.w4a16_cross_entropy(x[:0], *w, t[:0], with_mean=True)
    assert loss.shape == (0,) and lse.shape == (0,) and mean.shape == (0, 144)
    assert nv.w4a16_cross_entropy_backward(mean, *w, t[:0], loss, loss).shape == (0, 144)
    n = nv.w4a16_cross_entropy_workspace_bytes(40, 300, 144, True)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    got = nv.w4a16_cross_entropy(x, *w, t, with_mean=True, workspace=ws[:n])
    assert all(torch.equal(p, q) for p, q in zip(got, nv.w4a16_cross_entropy(x, *w, t, with_mean=True)))
    assert bool((ws[n:] == 255).all())
    out = torch.full((45, 144), 3.0, device="cuda")
    nv.w4a16_cross_entropy_backward(got[2], *w, t, got[0], got[1], out=out[:40])
    assert bool((out[40:] == 3.0).all())


def test_pieces_of_a_long_call():
    """More probabilities than are held at a time: 384 and 44 tokens."""
    check(*make(428, 600_000, 16, seed=15))


def test_gradient_against_differences():
    """Central differences of the 64-bit loss along random directions, step
    1e-4 of x: off by 1e-8 of the third derivative and 1e-11 of rounding."""
    x, t, w, W = make(20, 500, 272, seed=16, spread=10.0)
    loss, lse, mean = nv.w4a16_cross_entropy(x, *w, t, with_mean=True)
    r = entropy_reference(x, W, t)
    a, b = torch.full((20,), 0.7, device="cuda"), torch.full((20,), 0.2, device="cuda")
    dx = nv.w4a16_cross_entropy_backward(mean, *w, t, loss, a, b, out_dtype=torch.float32).double()
    _, tol = entropy_grad_reference(r, W, a, b)
    g = torch.Generator(device="cuda").manual_seed(17)
    for _ in range(3):
        v = torch.randn(20, 272, device="cuda", generator=g, dtype=torch.float64)

        def f(s):
            z = (x.double() + s * v) @ W.T
            q = torch.logsumexp(z, 1)
            has = (t >= 0) & (t < 500)
            return torch.where(has, 0.7 * (q - z.gather(1, t.clamp(0, 499)[:, None])[:, 0]), 0.0) + 0.2 * q

        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        within((dx * v).sum(1), slope, (tol * v.abs()).sum(1) + 1e-5 * (dx * v).abs().sum(1) + 1e-7)


def test_graph():
    """loss and lse carry the gradient; ignored positions and views of
    gradients among it."""
    x, t, w, W = make(50, 900, 272, seed=18)
    x.requires_grad_(True)
    loss, lse = nv.w4a16_cross_entropy(x, *w, t)
    plain = nv.w4a16_cross_entropy(x.detach(), *w, t)
    assert torch.equal(loss.detach(), plain[0]) and torch.equal(lse.detach(), plain[1])
    r = entropy_reference(x.detach(), W, t)
    n = int(((t >= 0) & (t < 900)).sum())
    cases = [(loss.sum() / n, torch.full((50,), 1 / n), torch.zeros(50)),
             (lse.mean(), torch.zeros(50), torch.full((50,), 1 / 50)),
             (loss.sum() / n + 1e-2 * (lse * lse).mean(), torch.full((50,), 1 / n),
              (2e-2 / 50 * plain[1]).cpu())]
    for value, a, b in cases:
        (dx,) = torch.autograd.grad(value, x, retain_graph=True)
        assert dx.dtype == torch.bfloat16
        want, tol = entropy_grad_reference(r, W, a.cuda(), b.cuda())
        within(dx, want, stored(want, tol + 2.0 ** -20 * want.abs(), dx.dtype))
    with torch.no_grad():
        assert not any(v.requires_grad for v in nv.w4a16_cross_entropy(x, *w, t))
    assert not any(v.requires_grad for v in nv.w4a16_cross_entropy(x, *w, t, with_mean=True))


@pytest.mark.parametrize("M", [9, 90, 400])
def test_same_bits_each_time_on_streams_and_in_graphs(M):
    x, t, w, W = make(M, 20_000, 528, seed=19)
    a = torch.randn(M, device="cuda")

    def both(stream=None):
        loss, lse, mean = nv.w4a16_cross_entropy(x, *w, t, with_mean=True, stream=stream)
        return loss, lse, mean, nv.w4a16_cross_entropy_backward(mean, *w, t, loss, a, lse, stream=stream)

    first = both()
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(both(), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(other, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (20, 21):
        nx, nt, _, _ = make(M, 20_000, 528, seed)
        x.copy_(nx)
        t.copy_(nt)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(held, both()))


def test_two_captured_calls_on_one_workspace():
    """Replayed one after the other, each as if it were alone."""
    x, t, w, W = make(33, 3000, 272, seed=22)
    y, u, _, _ = make(33, 3000, 272, seed=23)
    ws = torch.empty(nv.w4a16_cross_entropy_workspace_bytes(33, 3000, 272, True), dtype=torch.uint8,
                     device="cuda")
    want = [nv.w4a16_cross_entropy(p, *w, q, with_mean=True) for p, q in ((x, t), (y, u))]
    graphs = []
    for p, q in ((x, t), (y, u)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = nv.w4a16_cross_entropy(p, *w, q, with_mean=True, workspace=ws)
        graphs.append((graph, held))
    for i in (0, 1, 0, 0, 1):
        graphs[i][0].replay()
        assert all(torch.equal(p, q) for p, q in zip(graphs[i][1], want[i]))
