"""The training calls together, as a model's last layer and loss use them: a
gated block, its down projection, the residual and the cross entropy over the
lm_head, with the gradient through all of it."""
import threading

import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._train import activation, hidden, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("call", ["lm_head", "back", "glu", "glu_backward", "cross_entropy"])
def test_first_call_of_a_thread(call):
    """A thread that has made no CUDA call, as an autograd thread is at first."""
    w, _ = weight(512, 256, seed=1)
    x, dy = hidden(20, 256, seed=2), hidden(20, 512, seed=3)
    t = torch.arange(20, device="cuda")
    calls = {"lm_head": lambda: nv.w4a16_lm_head(x, *w), "back": lambda: nv.w4a16_lm_head_backward(dy, *w),
             "glu": lambda: nv.w4a16_glu(x, *w),
             "glu_backward": lambda: nv.w4a16_glu_backward(dy[:, :256].contiguous(), x, *w),
             "cross_entropy": lambda: nv.w4a16_cross_entropy(x, *w, t, with_mean=True)[2]}
    want = calls[call]()
    torch.cuda.synchronize()
    got = []
    thread = threading.Thread(target=lambda: got.append(calls[call]()))
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert got and torch.equal(got[0], want)


@pytest.mark.parametrize("M", [1, 50, 300])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_block_and_loss(M, act):
    """Against the same chain in 64 bits by autograd.  Each of the three
    bf16 roundings on the way forward (h, y, x + y) moves what follows by at
    most 2^-8 of itself, at random, and so does each of the four on the way
    back; the largest of the errors stays below 4 times the root of their
    squares' sum."""
    K, I, V = 272, 400, 3000
    w13, W13 = weight(2 * I, K, seed=1)
    w2, W2 = weight(K, I, seed=2)
    head, H = weight(V, K, seed=3)
    x = hidden(M, K, seed=4, outliers=0).requires_grad_(True)
    t = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(5)).cuda()
    if M > 1:
        t[M // 2] = -100

    def own(x):
        y = nv.w4a16_lm_head(nv.w4a16_glu(x, *w13, activation=act), *w2, out_dtype=torch.bfloat16)
        loss, lse = nv.w4a16_cross_entropy(x + y, *head, t)
        return loss.sum() + 1e-2 * (lse * lse).sum()

    def plain(x):
        gu = x @ W13.T
        y = (activation(gu[:, :I], act)[0] * gu[:, I:]) @ W2.T
        z = (x + y) @ H.T
        lse = torch.logsumexp(z, 1)
        loss = torch.where(t >= 0, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
        return loss.sum() + 1e-2 * (lse * lse).sum()

    value = own(x)
    (dx,) = torch.autograd.grad(value, x)
    X = x.detach().double().requires_grad_(True)
    want = plain(X)
    (dX,) = torch.autograd.grad(want, X)
    assert abs(float(value.detach()) - float(want.detach())) <= 4 * 2.0 ** -8 * 3 ** 0.5 * abs(float(want.detach()))
    err = (dx.double() - dX).norm(dim=1) / dX.norm(dim=1)
    assert float(err.max()) <= 4 * 2.0 ** -8 * 7 ** 0.5


def test_captured_training_step():
    """Forward and backward pass of the chain captured into one CUDA graph."""
    K, I, V, M = 272, 400, 3000, 64
    w13, _ = weight(2 * I, K, seed=1)
    w2, _ = weight(K, I, seed=2)
    head, _ = weight(V, K, seed=3)
    x = hidden(M, K, seed=4)
    t = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(5)).cuda()
    a = torch.full((M,), 1.0 / M, device="cuda")

    def step():
        h = nv.w4a16_glu(x, *w13)
        y = nv.w4a16_lm_head(h, *w2, out_dtype=torch.bfloat16)
        loss, lse, mean = nv.w4a16_cross_entropy(x + y, *head, t, with_mean=True)
        dr = nv.w4a16_cross_entropy_backward(mean, *head, t, loss, a)
        dh = nv.w4a16_lm_head_backward(dr, *w2)
        return loss, dr + nv.w4a16_glu_backward(dh, x, *w13)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (6, 7):
        x.copy_(hidden(M, K, seed))
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(held, step()))
