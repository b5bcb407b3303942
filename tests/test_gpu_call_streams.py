"""The memory of the compiled calls.  Given a stream other than the current one, their results and
workspaces are not memory whose last use is still queued on the current
stream."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests.test_gpu_logprobs import check as check_logprobs
from tests.test_gpu_logprobs import make as make_logits
from tests.test_gpu_moe import check, make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def test_memory_still_in_use_on_the_current_stream_is_not_reused():
    args = make(64, 16, 4, 512, 256, seed=21)
    dev = on_gpu(*args)
    logits = torch.randn(64, 16, device="cuda")
    big, tok = make_logits(40, 5001, torch.float32, seed=3)
    bd, td = big.cuda(), tok.cuda()
    n = nv.w4a16_moe_workspace_bytes(64, 4, 512, 256)
    sizes = (n, n, 64 * 512 * 2, 4096, 8192, 16384, 40 * 5001 * 4)
    grads = torch.randn(40, device="cuda")
    lse = torch.logsumexp(bd, 1)
    ent = torch.ones(40, device="cuda")

    def calls(stream):
        return [nv.w4a16_moe(*dev, stream=stream), *nv.moe_route(logits, 4, stream=stream),
                *nv.token_logprobs(bd, td, 5, stream=stream),
                nv.token_logprobs_backward(bd, td, lse, ent, grads, stream=stream)]

    want = [t.cpu() for t in calls(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    free = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(3)]
    torch.cuda._sleep(40_000_000)  # what the current stream does below waits for some 20 ms
    for t in free:
        t.fill_(255)
    del t, free
    got = calls(s)
    s.synchronize()
    with torch.cuda.stream(s):
        early = [t.cpu() for t in got]
    torch.cuda.synchronize()
    for now, a, b in zip(early, got, want):
        assert torch.equal(now, b) and torch.equal(a.cpu(), b)
    check(got[0], args)
    check_logprobs(got[3:9], big, tok, 5)


def test_results_used_by_the_current_stream_are_not_given_out_on_the_other():
    """Freed while the current stream still has to read them."""
    logits, tok = (t.cuda() for t in make_logits(64, 40001, torch.float32, seed=5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = nv.token_logprobs(logits, tok, 20)[5].clone()
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    held = nv.token_logprobs(logits, tok, 20, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(40_000_000)
    out.copy_(held[5])
    del held
    with torch.cuda.stream(s):
        junk = [torch.zeros(64 * 20 * 12 + 4096, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((j == 0).all()) for j in junk)


def test_workspace_has_its_bytes():
    """A view with enough elements over a small storage is refused."""
    dev = on_gpu(*make(3, 4, 2, 64, 32, seed=1))
    n = nv.w4a16_moe_workspace_bytes(3, 2, 64, 32)
    small = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for view in (small.expand(n), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            nv.w4a16_moe(*dev, workspace=view)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        nv.w4a16_moe(*dev, workspace=torch.zeros(n, dtype=torch.uint8))


def test_out_of_memory_is_torchs_own_exception():
    """As the calls that allocate through torch.empty raise it; the allocator
    is told that it has no memory left."""
    logits = torch.randn(300, 40001, device="cuda")
    tok = torch.zeros(300, dtype=torch.int64, device="cuda")
    vec = torch.zeros(300, device="cuda")
    dev = on_gpu(*make(512, 8, 8, 1024, 512, seed=1))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() /
                                               torch.cuda.get_device_properties(0).total_memory)
    held = []
    try:
        with pytest.raises(torch.OutOfMemoryError):  # what is free of the memory held already
            while True:
                held.append(torch.empty(16 << 20, dtype=torch.uint8, device="cuda"))
        for call in (lambda: torch.empty_like(logits),
                     lambda: nv.token_logprobs_backward(logits, tok, vec, vec, vec),
                     lambda: nv.w4a16_moe(*dev)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        held.clear()
    nv.w4a16_moe(*dev)
    torch.cuda.synchronize()


@pytest.mark.parametrize("k", [-1, 11, 1000, 1 << 40, (1 << 62) + 3])
def test_k_out_of_range_is_a_shape_error_of_any_size(k):
    x = torch.zeros(4, 10, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    for call in (lambda: nv.token_logprobs(x, tok, k), lambda: nv.moe_route(x, k),
                 lambda: nv.moe_route(x, k, expert_ids=torch.zeros(4, max(k, 0), dtype=torch.int32, device="cuda")
                                      if k < 2000 else None)):
        with pytest.raises(nv.NVFP4Error) as err:
            call()
        assert err.value.status == nv.Status.ERR_SHAPE
