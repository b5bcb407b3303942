"""The kernels that take shares of more than 32768 logits: 512 threads, eight
vectors ahead where the grid is one CTA an SM and four where it is more, with
the ties, masks and special rows that leave the first bound."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._routes import kernels
from tests.test_gpu_logprobs import check, make

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def launched(x, tok, k, depth):
    names = kernels(lambda: nv.token_logprobs(x, tok, k))
    assert any("logprobs_kernel" in n and f"512, {depth}>" in n for n in names), names


@pytest.mark.parametrize("M,N,k,depth", [(64, 151936, 8, 8), (40, 151936, 4, 4), (130, 36001, 0, 8), (140, 33003, 5, 8),
                                         (170, 40001, 3, 4), (304, 33000, 20, 4), (330, 34001, 17, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward(M, N, k, depth, dtype):
    x, tok = make(M, N, dtype, seed=M + N)
    dev, t = x.cuda(), tok.cuda()
    check(nv.token_logprobs(dev, t, k), x, tok, k)
    launched(dev, t, k, depth)


@pytest.mark.parametrize("M,depth", [(130, 8), (170, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 30, 128])
def test_special_rows(M, depth, dtype, k):
    N = 36003
    low = torch.finfo(dtype).min
    x, tok = make(M, N, dtype, seed=k, pad=5)
    x = x.clone()
    x[0] = -INF
    x[1] = -INF
    x[1, 30000] = 3.0
    x[2] = 1.5
    x[3, ::2] = -INF
    x[4] = low
    x[5, 10:] = low
    x[6] = 0.5
    x[6, 1::2] = 1.0
    x[7, :20000] = 2.0
    x[8] = -INF
    x[8, 35990:] = torch.arange(13).to(dtype)
    x[9, :] = torch.linspace(-90, 90, N).to(dtype)
    tok[:10] = torch.tensor([4, 30000, 35000, 2, 9, 11, 1, 25000, 35995, 0])
    dev, t = x.cuda(), tok.cuda()
    check(nv.token_logprobs(dev, t, k), x, tok, k)
    launched(dev, t, k, depth)
    x[10, 35000] = float("nan")
    x[11, 5] = INF
    lp, ent, lse, _, ids, _ = nv.token_logprobs(x.cuda(), t, k)
    for out in (lp, ent, lse):
        assert bool(torch.isnan(out[10:12]).all()) and not bool(torch.isnan(out[12:]).any())
    assert ids[10, 0] == 35000 and ids[11, 0] == 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_temperature(dtype):
    x, tok = make(150, 36000, dtype, seed=4)
    s = float(torch.tensor(1.0 / 0.7, dtype=torch.float32))
    check(nv.token_logprobs(x.cuda(), tok.cuda(), 4, inv_temperature=s), x, tok, 4, s)
