"""Token log probabilities, entropy, ranks, alternatives and their gradient
against plain 64-bit forms: odd vocabularies, strided and unaligned rows,
masked, empty, tied and non-finite rows, offsets past 32 bits.

Tolerances of the forward (fp32): a term exp(d) is off by 2^-22 plus
|d| 2^-23 of itself, and |d| weighted by the terms is below 13 for fewer than
2^18 columns; a sum over at most 1024 terms per thread and 20 merges rounds
by (1024 + 20) 2^-24.  So S and T are within 7e-5 of themselves, which bounds
lse by 7e-5 + 2^-22 (|lse| + |max|) and the entropy by 7e-5 (2 entropy + 1)
plus 2^-22 of the same terms."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._operators import bf16_half_ulp, logprobs_grad_reference, logprobs_reference

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def make(M, N, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N + pad, generator=g) * 2.5
    x[torch.arange(M), torch.randint(0, N, (M,), generator=g)] += 9.0
    x = x.to(dtype)
    tok = torch.randint(0, N, (M,), generator=g)
    tok[::3] = x[::3, :N].float().argmax(1)
    return x[:, :N], tok


def check(got, x, tok, k, s=1.0):
    lp, ent, lse, ranks, ids, top = (t.cpu() for t in got)
    w = logprobs_reference(x, tok, k, s)
    size = torch.where(torch.isfinite(w[2]), w[2].abs(), 0.0) + \
        (s * torch.nan_to_num(x.double(), nan=0.0, posinf=0.0, neginf=0.0).amax(1)).abs()

    def near(a, b, tol, what):
        same = (a.double() == b) | (torch.isnan(a) & torch.isnan(b))
        assert bool((same | ((a.double() - b).abs() <= tol)).all()), (what, a, b)

    rounding = 7e-5 + 2.0 ** -22 * size
    near(lse, w[2], rounding, "lse")
    near(lp, w[0], rounding, "logprobs")
    near(ent, w[1], rounding + 1.4e-4 * w[1].abs(), "entropy")
    assert torch.equal(ranks, w[3])
    assert torch.equal(ids, w[4])
    near(top, w[5], rounding[:, None], "top_logprobs")


@pytest.mark.parametrize("M,N,k", [(1, 128256, 20), (1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 17, 17),
                                   (5, 127, 100), (4, 4096, 128), (33, 32003, 7), (7, 50257, 64),
                                   (64, 8191, 1), (310, 1537, 5), (2, 151936, 128), (1, 262144, 3),
                                   (20, 33000, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward(M, N, k, dtype):
    x, tok = make(M, N, dtype, seed=M + N)
    check(nv.token_logprobs(x.cuda(), tok.cuda(), k), x, tok, k)


@pytest.mark.parametrize("s", [0.25, 1.0 / 0.7, 40.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_temperature(s, dtype):
    x, tok = make(9, 5000, dtype, seed=1)
    s = float(torch.tensor(s, dtype=torch.float32))
    check(nv.token_logprobs(x.cuda(), tok.cuda(), 4, inv_temperature=s), x, tok, 4, s)


@pytest.mark.parametrize("pad,start", [(1, 0), (3, 1), (64, 0), (5, 2), (7, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(pad, start, dtype):
    M, N = 12, 2049
    x, tok = make(M, N, dtype, seed=pad)
    flat = torch.zeros(start + M * (N + pad), dtype=dtype)
    view = flat[start:].view(M, N + pad)[:, :N]
    view.copy_(x)
    dev = flat.cuda()[start:].view(M, N + pad)[:, :N]
    check(nv.token_logprobs(dev, tok.cuda(), 6), x, tok, 6)
    lse = torch.logsumexp(x.double(), 1).float()
    ent, a, b = torch.zeros(M), torch.randn(M), torch.randn(M)
    g = nv.token_logprobs_backward(dev, tok.cuda(), lse.cuda(), ent.cuda(), a.cuda(), b.cuda())
    check_grad(g, x, tok, 1.0, lse, ent, a, b)


def special_rows(dtype):
    N = 3001
    low = torch.finfo(dtype).min
    x = torch.randn(12, N, generator=torch.Generator().manual_seed(0)).to(dtype)
    x[0] = -INF                                   # nothing is left
    x[1] = -INF
    x[1, 2000] = 3.0                              # one token is left
    x[2, ::2] = -INF
    x[3] = 1.5                                    # all tied
    x[4] = low                                    # all at the type's lowest value
    x[5, 10:] = low                               # masked with it
    x[6, 0], x[6, 1] = 0.0, -0.0
    x[6, 2:] = -1.0
    x[7, :1500] = 2.0                             # a large tie at the top
    x[8] = -INF
    x[8, :5] = low
    x[9] = torch.linspace(-90, 90, N).to(dtype)
    x[10, 77] = float("nan")
    x[11, 5] = INF
    tok = torch.tensor([4, 2000, 3, 9, 0, 11, 1, 1600, 2, 3000, 5, 6])
    return x, tok


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [0, 1, 5, 128])
def test_special_rows(dtype, k):
    x, tok = special_rows(dtype)
    got = nv.token_logprobs(x.cuda(), tok.cuda(), k)
    check([t[:10] for t in got], x[:10], tok[:10], k)
    lp, ent, lse, ranks, ids, top = (t.cpu() for t in got)
    assert lp[0] == -INF and ent[0] == 0 and lse[0] == -INF and ranks[0] == 1
    assert lp[1] == 0 and ent[1] == 0
    for t in (lp, ent, lse):
        assert bool(torch.isnan(t[10:]).all())
    if k:
        assert ids[10, 0] == 77 and ids[11, 0] == 5


def test_rows_without_a_token():
    x, tok = make(6, 999, torch.float32, seed=2)
    tok[:] = torch.tensor([-1, 0, 999, -100, 998, 2 ** 40])
    got = nv.token_logprobs(x.cuda(), tok.cuda(), 3)
    check(got, x, tok, 3)
    assert got[0][[0, 2, 3, 5]].tolist() == [0] * 4 and got[3][[0, 2, 3, 5]].tolist() == [0] * 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_candidates_at_the_bound(dtype):
    """Every logit ties (or two values alternate) over a whole vocabulary and
    over several CTAs of a row: the lowest columns win."""
    N = 70000
    x = torch.full((3, N), 0.5, dtype=dtype)
    x[1, 1::2] = 1.0
    x[2, N - 3:] = 2.0
    tok = torch.tensor([5, 1, N - 1])
    for k in (1, 33, 128):
        check(nv.token_logprobs(x.cuda(), tok.cuda(), k), x, tok, k)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    N, ld = 1000, 2 ** 31 + 24
    buf = torch.empty(ld + N, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(buf, (2, N), (ld, 1))
    x, tok = make(2, N, torch.bfloat16, seed=3)
    view.copy_(x)
    got = nv.token_logprobs(view, tok.cuda(), 5)
    check(got, x, tok, 5)
    a = torch.randn(2)
    lse, ent = got[2].cpu(), got[1].cpu()
    g = nv.token_logprobs_backward(view, tok.cuda(), got[2], got[1], a.cuda(), a.cuda(), out=view)
    check_grad(g, x, tok, 1.0, lse, ent, a, a)


# ---------------------------------------------------------------- gradient
def check_grad(got, x, tok, s, lse, ent, a, b):
    want, tol = logprobs_grad_reference(x, tok, s, lse, ent, a, b)
    if got.dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(want.abs() + tol)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol.clamp(min=1e-300)).max()), err.max())


@pytest.mark.parametrize("M,N", [(1, 1), (2, 3), (3, 4097), (19, 50257), (2, 128256), (300, 1003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s", [1.0, 1.5])
def test_gradient_against_the_formula(M, N, dtype, s):
    x, tok = make(M, N, dtype, seed=N + 1)
    if M > 2:
        tok[1] = -1
        x[2, ::3] = -INF
        tok[2] = 1
    g = torch.Generator().manual_seed(5)
    a, b = torch.randn(M, generator=g), torch.randn(M, generator=g) * 0.1
    _, ent, lse, *_ = nv.token_logprobs(x.cuda(), tok.cuda(), inv_temperature=s)
    got = nv.token_logprobs_backward(x.cuda(), tok.cuda(), lse, ent, a.cuda(), b.cuda(), s)
    check_grad(got, x, tok, s, lse.cpu(), ent.cpu(), a, b)
    # without an entropy gradient, and in place
    dev = x.cuda().clone()
    got = nv.token_logprobs_backward(dev, tok.cuda(), lse, None, a.cuda(), None, s, out=dev)
    assert got.data_ptr() == dev.data_ptr()
    check_grad(got, x, tok, s, lse.cpu(), ent.cpu(), a, torch.zeros(M))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 3])
def test_large_gradient(dtype, pad):
    """Logits and gradient of more than 32 MB together, rows on and off
    16-byte boundaries, into a new tensor and in place."""
    M, N = 75, 120001
    x, tok = make(M, N, dtype, seed=9, pad=pad)
    tok[4] = -1
    x[7, 1::2] = -INF
    tok[7] = 0
    dev = x.cuda() if pad == 0 else torch.empty(M, N + pad, dtype=dtype, device="cuda")[:, :N].copy_(x)
    g = torch.Generator().manual_seed(8)
    a, b = torch.randn(M, generator=g), torch.randn(M, generator=g) * 0.1
    _, ent, lse, *_ = nv.token_logprobs(dev, tok.cuda())
    args = (tok.cuda(), lse, ent, a.cuda(), b.cuda())
    check_grad(nv.token_logprobs_backward(dev, *args), x, tok, 1.0, lse.cpu(), ent.cpu(), a, b)
    check_grad(nv.token_logprobs_backward(dev, *args, out=dev), x, tok, 1.0, lse.cpu(), ent.cpu(), a, b)


def test_gradient_against_differences():
    """Directional differences of f = sum a logprob + b entropy in 64 bits:
    central differences of step 1e-4 are off by about 1e-8 of f's third
    derivative, well inside 1e-4 of |a| + |b| times the direction."""
    M, N, s = 6, 700, 1.25
    x, tok = make(M, N, torch.float32, seed=4)
    tok[3] = -1
    g = torch.Generator().manual_seed(6)
    a, b = torch.randn(M, generator=g), torch.randn(M, generator=g)
    _, ent, lse, *_ = nv.token_logprobs(x.cuda(), tok.cuda(), inv_temperature=s)
    grad = nv.token_logprobs_backward(x.cuda(), tok.cuda(), lse, ent, a.cuda(), b.cuda(), s).cpu()

    def f(y):
        lp, H, *_ = logprobs_reference(y, tok, 0, s)
        return a.double() * lp + b.double() * H

    for _ in range(8):
        d = torch.randn(M, N, generator=g, dtype=torch.float64)
        slope = (f(x.double() + 1e-4 * d) - f(x.double() - 1e-4 * d)) / 2e-4
        got = (grad.double() * d).sum(1)
        assert bool(((got - slope).abs() <= 1e-4 * (a.abs() + b.abs()) * d.abs().amax(1)).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_special_rows(dtype):
    x, tok = special_rows(dtype)
    x, tok = x[:10], tok[:10]
    a, b = torch.ones(10), torch.full((10,), 0.5)
    _, ent, lse, *_ = nv.token_logprobs(x.cuda(), tok.cuda())
    got = nv.token_logprobs_backward(x.cuda(), tok.cuda(), lse, ent, a.cuda(), b.cuda())
    assert bool((got[0] == 0).all())
    check_grad(got, x, tok, 1.0, lse.cpu(), ent.cpu(), a, b)


def test_deterministic_on_another_stream_and_in_a_graph():
    x, tok = make(37, 40001, torch.bfloat16, seed=7)
    x, tok = x.cuda(), tok.cuda()
    first = nv.token_logprobs(x, tok, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = nv.token_logprobs(x, tok, 12)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = nv.token_logprobs(x, tok, 12)
    x.add_(1.0)
    want = nv.token_logprobs(x, tok, 12)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_empty_batch_and_refusals():
    x = torch.zeros(4, 10, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert nv.token_logprobs(x[:0], t[:0], 3)[4].shape == (0, 3)
    for bad in (dict(k=11), dict(k=-1), dict(inv_temperature=0.0), dict(inv_temperature=INF),
                dict(inv_temperature=float("nan"))):
        with pytest.raises(nv.NVFP4Error) as err:
            nv.token_logprobs(x, t, **bad)
        assert err.value.status == nv.Status.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error):
        nv.token_logprobs(x[:, :0], t)
    with pytest.raises(ValueError, match="contiguous"):
        nv.token_logprobs(torch.zeros(10, 4, device="cuda").t(), t)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        nv.token_logprobs(x.half(), t)
    with pytest.raises(ValueError, match="token_ids"):
        nv.token_logprobs(x, t.int())
    with pytest.raises(ValueError, match="overlap"):
        nv.token_logprobs(x[:1].expand(4, 10), t)
    f = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="entropy"):
        nv.token_logprobs_backward(x, t, f, None, f, f)
    with pytest.raises(ValueError, match="out"):
        nv.token_logprobs_backward(x, t, f, f, f, f, out=torch.zeros(4, 10, device="cuda").half())
