"""token_logprobs on logits that require a gradient: the graph leads to
token_logprobs_backward."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests.test_gpu_logprobs import check, check_grad, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_logprobs,with_entropy", [(True, True), (True, False), (False, True)])
def test_graph(dtype, with_logprobs, with_entropy):
    M, N, s = 7, 4099, 1.25
    x, tok = make(M, N, dtype, seed=1, pad=3)
    tok[3] = -1
    g = torch.Generator().manual_seed(2)
    a = torch.randn(M, generator=g) * with_logprobs
    b = torch.randn(M, generator=g) * with_entropy
    buf = torch.zeros(M, N + 3, dtype=dtype, device="cuda")
    buf[:, :N] = x.cuda()
    buf.requires_grad_(True)
    got = nv.token_logprobs(buf[:, :N], tok.cuda(), 4, inv_temperature=s)
    check([t.detach() for t in got], x, tok, 4, s)
    loss = 0.0
    if with_logprobs:
        loss = loss + (a.cuda() * got[0]).sum()
    if with_entropy:
        loss = loss + (b.cuda() * got[1]).sum()
    loss.backward()
    assert bool((buf.grad[:, N:] == 0).all())
    check_grad(buf.grad[:, :N], x, tok, s, got[2].detach().cpu(), got[1].detach().cpu(), a, b)


def test_gradients_given_as_views():
    """A mean's gradient is one element for all rows."""
    x, tok = make(6, 500, torch.float32, seed=3)
    logits = x.cuda().requires_grad_(True)
    lp, ent, lse, *_ = nv.token_logprobs(logits, tok.cuda())
    (lp.mean() + 0.5 * ent.mean()).backward()
    check_grad(logits.grad, x, tok, 1.0, lse.detach().cpu(), ent.detach().cpu(), torch.full((6,), 1 / 6),
               torch.full((6,), 0.5 / 6))


def test_what_has_no_gradient():
    x, tok = make(6, 500, torch.float32, seed=4)
    x, tok = x.cuda(), tok.cuda()
    logits = x.clone().requires_grad_(True)
    out = nv.token_logprobs(logits, tok, 3)
    assert not out[3].requires_grad and not out[4].requires_grad
    for at in (2, 5):
        with pytest.raises(RuntimeError, match="logprobs and entropy only"):
            (out[0].sum() + out[at].sum()).backward(retain_graph=True)
    with torch.no_grad():
        plain = nv.token_logprobs(logits, tok, 3)
    assert not any(t.requires_grad for t in plain)
    assert not any(t.requires_grad for t in nv.token_logprobs(x, tok, 3))
    assert all(torch.equal(p, q) for p, q in zip(plain, out))
    with torch.no_grad():  # what the gradient needs was overwritten
        logits.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out[0].sum().backward()
