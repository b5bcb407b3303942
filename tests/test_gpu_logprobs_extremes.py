"""Token log probabilities and their gradient at the ends of fp32's range: the
largest finite logits, temperatures near 2^-128, and large gradient weights."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests.test_gpu_logprobs import check, make

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def dominated(M, N, dtype, value):
    """Rows of ordinary logits in which one is `value` (and in every other row
    half of the others are masked)."""
    x, tok = make(M, N, dtype, seed=N)
    x[1::2, ::2] = -INF
    x[torch.arange(M), torch.arange(M) * 7 % N] = value
    tok[:2] = torch.arange(2) * 7 % N
    return x, tok


@pytest.mark.parametrize("M,N", [(3, 61), (6, 5003), (2, 70001), (130, 36001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s,value", [(1.0, None), (0.25, None), (0.75, 3.0e38), (100.0, 3.0e36),
                                     (1.0e6, 1.0e31)])
def test_a_logit_near_the_largest_number(M, N, dtype, s, value):
    x, tok = dominated(M, N, dtype, torch.finfo(dtype).max if value is None else value)
    s = float(torch.tensor(s, dtype=torch.float32))
    got = nv.token_logprobs(x.cuda(), tok.cuda(), 3, inv_temperature=s)
    check(got, x, tok, 3, s)
    assert bool((got[1] == 0).all())


@pytest.mark.parametrize("N", [9, 5003, 70001])
@pytest.mark.parametrize("s", [1.0e38, 2.5e38, 3.3e38])
def test_temperature_near_zero(N, s):
    g = torch.Generator().manual_seed(N)
    x = torch.randn(4, N, generator=g) * 2e-38
    x[1, ::2] = -INF
    tok = torch.randint(0, N, (4,), generator=g)
    tok[1] = 1
    s = float(torch.tensor(s, dtype=torch.float32))
    check(nv.token_logprobs(x.cuda(), tok.cuda(), 3, inv_temperature=s), x, tok, 3, s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b", [1e9, 1e30])
def test_gradient_of_masked_columns_with_a_large_weight(dtype, b):
    """p log p is 0 at a masked column whatever the entropy's gradient is."""
    x, tok = make(5, 4099, dtype, seed=1)
    x[:, ::2] = -INF
    tok[:] = 1
    _, ent, lse, *_ = nv.token_logprobs(x.cuda(), tok.cuda())
    g = nv.token_logprobs_backward(x.cuda(), tok.cuda(), lse, ent, torch.zeros(5).cuda(),
                                   torch.full((5,), b).cuda())
    assert bool((g[:, ::2] == 0).all()) and bool(torch.isfinite(g).all())
    one = nv.token_logprobs_backward(x.cuda(), tok.cuda(), lse, ent, torch.zeros(5).cuda(),
                                     torch.ones(5).cuda())
    assert bool(((g.double() / b - one.double()).abs() <= 2.0 ** -7 * one.double().abs() + 1e-30).all())
