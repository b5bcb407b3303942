"""The memory of the training calls on a stream other than the current one:
neither results nor workspaces are memory whose last use is still queued on
the current stream, and two calls on two streams do not meet."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._train import hidden, weight

pytestmark = pytest.mark.gpu

M, V, I, K = 150, 2000, 300, 272


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def inputs(seed):
    w13, _ = weight(2 * I, K, seed=seed)
    head, _ = weight(V, K, seed=seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    return {"x": hidden(M, K, seed=seed + 3), "w13": w13, "head": head,
            "t": torch.randint(0, V, (M,), generator=g).cuda(),
            "dh": torch.randn(M, I, generator=g).cuda(),
            "dy": torch.randn(M, V, generator=g).to(torch.bfloat16).cuda(),
            "a": torch.randn(M, generator=g).cuda()}


def calls(d, stream):
    loss, lse, mean = nv.w4a16_cross_entropy(d["x"], *d["head"], d["t"], with_mean=True, stream=stream)
    return [loss, lse, mean,
            nv.w4a16_cross_entropy_backward(mean, *d["head"], d["t"], loss, d["a"], stream=stream),
            nv.w4a16_lm_head_backward(d["dy"], *d["head"], stream=stream),
            nv.w4a16_glu(d["x"], *d["w13"], stream=stream),
            nv.w4a16_glu_backward(d["dh"], d["x"], *d["w13"], stream=stream)]


def test_memory_still_in_use_on_the_current_stream_is_not_reused():
    d = inputs(1)
    want = [t.cpu() for t in calls(d, None)]
    torch.cuda.synchronize()
    sizes = (nv.w4a16_cross_entropy_workspace_bytes(M, V, K, True),
             nv.w4a16_lm_head_backward_workspace_bytes(M, V, K), nv.w4a16_glu_workspace_bytes(M, I, K),
             nv.w4a16_glu_backward_workspace_bytes(M, I, K), M * K * 4, M * K * 2, M * I * 2, 1024, 2048)
    s = torch.cuda.Stream()
    free = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(3)]
    torch.cuda._sleep(40_000_000)  # what the current stream does below waits for some 20 ms
    for t in free:
        t.fill_(255)
    del t, free
    got = calls(d, s)
    s.synchronize()
    with torch.cuda.stream(s):
        early = [t.cpu() for t in got]
    torch.cuda.synchronize()
    for now, a, b in zip(early, got, want):
        assert torch.equal(now, b) and torch.equal(a.cpu(), b)


def test_results_used_by_the_current_stream_are_not_given_out_on_the_other():
    """Freed while the current stream still has to read them."""
    d = inputs(11)
    want = [t.clone() for t in calls(d, None)]
    out = [torch.empty_like(t) for t in want]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = calls(d, s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(40_000_000)
    for o, h in zip(out, held):
        o.copy_(h)
    sizes = [t.numel() * t.element_size() for t in held]
    del held, h
    with torch.cuda.stream(s):
        junk = [torch.zeros(b, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))
    assert all(bool((j == 0).all()) for j in junk)


def test_calls_on_two_streams_at_once():
    d = [inputs(21), inputs(31)]
    want = [[t.clone() for t in calls(e, None)] for e in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [calls(e, s) for e, s in zip(d, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_gradients_of_broadcast_sums_and_a_frozen_x():
    """loss.sum() hands a gradient of stride 0 back; without one nothing is kept."""
    d = inputs(41)
    x = d["x"].clone().requires_grad_(True)
    loss, lse = nv.w4a16_cross_entropy(x, *d["head"], d["t"])
    (dx,) = torch.autograd.grad(loss.sum() + lse.sum(), x)
    y = nv.w4a16_glu(x, *d["w13"])
    (dy,) = torch.autograd.grad(y.float().sum(), x)
    (dz,) = torch.autograd.grad(nv.w4a16_lm_head(x, *d["head"]).sum(), x)
    one = torch.ones(M, device="cuda")
    loss2, _, mean = nv.w4a16_cross_entropy(d["x"], *d["head"], d["t"], with_mean=True)
    assert torch.equal(loss, loss2) and not loss2.requires_grad
    assert torch.equal(dx, nv.w4a16_cross_entropy_backward(mean, *d["head"], d["t"], loss2, one, one))
    assert torch.equal(dy, nv.w4a16_glu_backward(torch.ones(M, I, device="cuda", dtype=torch.bfloat16),
                                                 d["x"], *d["w13"]))
    assert torch.equal(dz, nv.w4a16_lm_head_backward(torch.ones(M, V, device="cuda"), *d["head"]))
    with torch.no_grad():
        assert not nv.w4a16_cross_entropy(x, *d["head"], d["t"])[0].requires_grad
        assert not nv.w4a16_glu(x, *d["w13"]).requires_grad
