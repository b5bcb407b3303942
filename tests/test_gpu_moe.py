"""The router's choice and the few-token expert layer against plain 64-bit
forms: odd sizes, absent and repeated experts, special values, determinism,
streams and CUDA graphs with new routing."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests._operators import bf16_half_ulp, moe_reference, random_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


# ------------------------------------------------------------------ router
def route_reference(logits, k, scoring, renormalize, bias, scale):
    x = logits.double()
    s = torch.softmax(x, 1) if scoring == "softmax" else torch.sigmoid(x)
    s = torch.where(torch.isneginf(x).all(1, keepdim=True), 0.0, s)
    key = x if bias is None else s + bias.double()
    ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
    w = s.gather(1, ids)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return ids, w * scale


@pytest.mark.parametrize("M,E,k", [(1, 128, 8), (5, 1, 1), (3, 33, 32), (130, 64, 1), (65, 256, 8),
                                   (9, 257, 5), (4, 512, 32), (1000, 96, 6), (2, 7, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring,renormalize", [("softmax", True), ("softmax", False),
                                                 ("sigmoid", True), ("sigmoid", False)])
def test_route(M, E, k, dtype, scoring, renormalize):
    """bf16 logits of a narrow spread tie often: the lower expert comes first.
    Weights: exp, the sum of E terms and two divisions in fp32, (E + 16) 2^-23
    relative at the most."""
    g = torch.Generator().manual_seed(M * 1000 + E + k)
    x = (torch.randn(M, E, generator=g) * 1.5).to(dtype)
    ids, w = nv.moe_route(x.cuda(), k, renormalize=renormalize, scoring=scoring, scale=1.25)
    want_ids, want_w = route_reference(x, k, scoring, renormalize, None, 1.25)
    assert torch.equal(ids.cpu().long(), want_ids)
    err = (w.cpu().double() - want_w).abs()
    assert bool((err <= (E + 16) * 2.0 ** -23 * want_w.abs()).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_bias_chooses_but_does_not_weigh(scoring):
    """Biases a multiple of 0.25 apart with scores below 0.2 of each other
    leave no near ties; the weights are the unbiased scores."""
    M, E, k = 40, 24, 6
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, E, generator=g) * 0.1
    bias = torch.randperm(E, generator=g).float() * 0.25
    ids, w = nv.moe_route(x.cuda(), k, scoring=scoring, bias=bias.cuda())
    want_ids, want_w = route_reference(x, k, scoring, True, bias, 1.0)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert bool(((w.cpu().double() - want_w).abs() <= (E + 16) * 2.0 ** -23 * want_w).all())


def test_route_special_rows():
    inf = float("inf")
    x = torch.zeros(6, 40)
    x[0] = -inf                       # every expert masked
    x[1, :38] = -inf                  # fewer experts than k
    x[2, 5] = float("nan")
    x[3] = 0.0
    x[3, 7] = -0.0                    # equal to +0
    x[4] = torch.finfo(torch.float32).min  # the lowest finite value everywhere
    x[5, 20] = 80.0
    ids, w = (t.cpu() for t in nv.moe_route(x.cuda(), 4))
    assert ids[0].tolist() == [0, 1, 2, 3] and w[0].tolist() == [0, 0, 0, 0]
    assert ids[1].tolist() == [38, 39, 0, 1] and w[1].tolist() == [0.5, 0.5, 0, 0]
    assert ids[2, 0] == 5 and bool(torch.isnan(w[2]).all())
    assert ids[3].tolist() == [0, 1, 2, 3]
    assert ids[4].tolist() == [0, 1, 2, 3] and w[4].tolist() == [0.25] * 4
    assert ids[5, 0] == 20 and w[5, 0] == 1.0
    empty_ids, empty_w = nv.moe_route(torch.empty(0, 40, device="cuda"), 4)
    assert empty_ids.shape == (0, 4) and empty_w.shape == (0, 4)


@pytest.mark.parametrize("E", [7, 64, 100, 256, 400])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_ties(E, scoring):
    """fp32 logits that differ in their last bits only, equal ones among
    them, and NaNs of either sign: the exact order, the lower expert first."""
    g = torch.Generator().manual_seed(E)
    x = torch.ones(64, E) + torch.randint(0, 9, (64, E), generator=g) * 2.0 ** -23
    x[32:] *= -1
    x[5, 3], x[5, 6] = float("nan"), -float("nan")
    k = min(E, 8)
    ids, w = nv.moe_route(x.cuda(), k, scoring=scoring)
    want, want_w = route_reference(torch.nan_to_num(x, nan=1e4), k, scoring, True, None, 1.0)
    assert torch.equal(ids.cpu().long(), want)
    live = torch.arange(64) != 5
    assert bool(((w.cpu().double() - want_w).abs()[live] <= (E + 16) * 2.0 ** -23).all())
    assert bool(torch.isnan(w[5]).all())


def test_route_unaligned_rows():
    """A base and rows off a 16-byte boundary."""
    for E, at in ((128, 1), (130, 0), (250, 3)):
        buf = torch.randn(at + 9 * E, generator=torch.Generator().manual_seed(E))
        for t in (buf, buf.to(torch.bfloat16)):
            x = t.cuda()[at:].view(9, E)
            ids, _ = nv.moe_route(x, 6)
            want, _ = route_reference(x.cpu(), 6, "softmax", True, None, 1.0)
            assert torch.equal(ids.cpu().long(), want)


# ------------------------------------------------------------ expert layer
def make(M, E, k, H, I, seed, absent=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H, generator=g)
    x[:, ::37] *= 30.0
    ids = torch.argsort(torch.rand(M, E, generator=g), 1)[:, :k].to(torch.int32)
    ids[torch.rand(M, k, generator=g) < absent] = -1
    w = torch.rand(M, k, generator=g)
    return (x.to(torch.bfloat16), ids.contiguous(), w, random_experts(E, 2 * I, H, seed + 1),
            random_experts(E, H, I, seed + 2))


def on_gpu(x, ids, w, w13, w2):
    return (x.cuda(), ids.cuda(), w.cuda(), *(t.cuda() for t in w13), *(t.cuda() for t in w2))


def check(out, args, what=""):
    ref, tol = moe_reference(*args)
    if out.dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(ref.abs() + tol)
    err = (out.double().cpu() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


SHAPES = [
    (1, 8, 2, 256, 128), (1, 128, 8, 2048, 768), (1, 1, 1, 16, 16), (2, 3, 3, 16, 48),
    (3, 5, 2, 80, 48), (4, 6, 2, 272, 896), (5, 8, 4, 2880, 720), (7, 9, 1, 512, 1040),
    (8, 4, 2, 4352, 64), (33, 16, 4, 320, 256), (64, 32, 8, 512, 272), (40, 2, 2, 256, 512),
    (100, 3, 2, 1024, 320), (257, 40, 5, 192, 64), (2, 4, 2, 8208, 80), (3, 4, 2, 64, 12304),
]


@pytest.mark.parametrize("M,E,k,H,I", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_moe(M, E, k, H, I, out_dtype):
    args = make(M, E, k, H, I, seed=M + H)
    out = nv.w4a16_moe(*on_gpu(*args), out_dtype=out_dtype)
    check(out, args)


# more work: the FP4 tensor-core route, with inner sizes that are and are not
# multiples of 256, 64 and 32, units and tiles that are cut, row counts that
# are not multiples of 128, and more pairs of an expert than a tile takes
WIDE = [
    (16, 8, 4, 1024, 512), (24, 6, 2, 4352, 272), (33, 16, 4, 2048, 144), (300, 3, 3, 256, 144),
    (17, 512, 8, 1024, 336), (8, 8, 2, 4096, 528), (1, 64, 64, 720, 720), (9, 4, 1, 8192, 464),
    (512, 12, 8, 128, 64), (512, 12, 8, 80, 112), (40, 10, 3, 16, 16384), (70, 5, 2, 16128, 16),
]


@pytest.mark.parametrize("M,E,k,H,I", WIDE)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_moe_wide(M, E, k, H, I, out_dtype):
    args = make(M, E, k, H, I, seed=M + H + 1)
    args[1][M // 2, 0] = -1
    check(nv.w4a16_moe(*on_gpu(*args), out_dtype=out_dtype), args)


# rows of an odd number of 8-byte pieces, at the longest and the shortest
@pytest.mark.parametrize("M,E,k,H,I", [(16, 8, 4, 4080, 2864), (24, 4, 2, 48, 4080),
                                       (32, 5, 1, 16, 16), (60, 9, 3, 1008, 176)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_moe_wide_odd_rows(M, E, k, H, I, out_dtype):
    args = make(M, E, k, H, I, seed=2 * H + I)
    check(nv.w4a16_moe(*on_gpu(*args), out_dtype=out_dtype), args)


def test_moe_wide_absent_repeated_special_and_dirty():
    x, ids, w, w13, w2 = make(64, 16, 8, 512, 256, seed=15, absent=0.4)
    ids[0] = -1
    ids[1, :] = 3
    ids[2, 0], ids[2, 1], ids[3, 0] = 16, 2 ** 31 - 1, -2 ** 31
    dev = on_gpu(x, ids, w, w13, w2)
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(64, 8, 512, 256), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    clean = nv.w4a16_moe(*dev, out_dtype=torch.float32, workspace=ws)
    check(clean, (x, ids, w, w13, w2))
    assert bool((clean[0] == 0).all())
    assert nv.nvfp4_read_device_status(ws) == nv.Status.OK
    for fill in (0, 127, 255):  # NaN and every other byte left in the workspace
        ws.fill_(fill)
        assert torch.equal(nv.w4a16_moe(*dev, out_dtype=torch.float32, workspace=ws), clean)
    ids[4:7, 0] = 5  # each of these tokens has an expert
    clean = nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2), workspace=ws)
    x[4, 9], x[5, 511] = float("inf"), float("nan")
    x[6] = 0.0
    x[7] = (x[7].float() * 2.0 ** -120).to(torch.bfloat16)
    out = nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2), workspace=ws)
    same = torch.ones(64, dtype=torch.bool)
    same[4:8] = False
    assert torch.equal(out[same], clean[same])
    assert not bool(torch.isfinite(out[4:6]).any())
    assert bool((out[6] == 0).all()) and bool(torch.isfinite(out[7]).all())
    none = nv.w4a16_moe(*on_gpu(x, torch.full_like(ids, -1), w, w13, w2), workspace=ws)
    assert bool((none == 0).all())


def test_moe_wide_nan_block_scale_raises_the_status():
    """... in an expert that is read, and not in the rows behind it."""
    x, ids, w, w13, w2 = make(48, 6, 4, 720, 336, seed=4)
    ids[:] = torch.tensor([0, 1, 3, 4], dtype=torch.int32)
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(48, 4, 720, 336), dtype=torch.uint8, device="cuda")
    for at, e, status in ((1, 3, nv.Status.ERR_NONFINITE), (2, 1, nv.Status.ERR_NONFINITE),
                          (1, 2, nv.Status.OK), (2, 5, nv.Status.OK), (0, 0, nv.Status.OK)):
        bad = [x, list(w13), list(w2)]
        if at:
            s = bad[at][1].clone().view(torch.uint8)
            s[e, 3, 5] = 0x7F
            bad[at][1] = s.view(torch.float8_e4m3fn)
        nv.w4a16_moe(*on_gpu(x, ids, w, *bad[1:]), workspace=ws)
        assert nv.nvfp4_read_device_status(ws) == status, (at, e)


@pytest.mark.parametrize("M,E,k,H,I", [(5, 8, 4, 512, 256), (64, 16, 8, 256, 80), (9, 512, 8, 64, 32)])
def test_moe_absent_and_repeated_experts(M, E, k, H, I):
    """Ids outside [0, E) add nothing, a token without experts gets zeros, and
    an expert chosen twice counts twice."""
    x, ids, w, w13, w2 = make(M, E, k, H, I, seed=5, absent=0.4)
    ids[0] = -1
    ids[1, :] = 3
    ids[2, 0] = E
    ids[2, 1] = 2 ** 31 - 1
    ids[3, 0] = -2 ** 31
    out = nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2), out_dtype=torch.float32)
    assert bool((out[0] == 0).all())
    check(out, (x, ids, w, w13, w2))
    none = nv.w4a16_moe(*on_gpu(x, torch.full_like(ids, -1), w, w13, w2))
    assert bool((none == 0).all())


def test_moe_most_pairs():
    """4096 pairs, nearly all on one expert: segments that read its weights again."""
    args = make(512, 8, 8, 128, 64, seed=11)
    args[1][:, :7] = 2
    check(nv.w4a16_moe(*on_gpu(*args), out_dtype=torch.float32), args)


def test_moe_special_values_stay_in_their_token():
    x, ids, w, w13, w2 = make(6, 4, 2, 512, 256, seed=2)
    clean = nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2))
    x[1, 100] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 0.0
    x[5] = (x[5].float() * 2.0 ** -120).to(torch.bfloat16)
    out = nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2))
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert not bool(torch.isfinite(out[1]).any())
    assert bool(torch.isnan(out[3]).all())
    assert bool((out[4] == 0).all()) and bool(torch.isfinite(out[5]).all())


def test_moe_gate_extremes():
    """Gates from about -3e4 to 3e4: exp(-g) overflows, silu underflows."""
    x, ids, w, w13, w2 = make(4, 4, 2, 256, 128, seed=8)
    x = (x.float() * 3000.0).to(torch.bfloat16)
    check(nv.w4a16_moe(*on_gpu(x, ids, w, w13, w2), out_dtype=torch.float32), (x, ids, w, w13, w2))


def test_moe_nan_block_scale_raises_the_status():
    x, ids, w, w13, w2 = make(2, 4, 1, 512, 256, seed=4)
    ids[:] = torch.tensor([[1], [2]], dtype=torch.int32)
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(2, 1, 512, 256), dtype=torch.uint8, device="cuda")
    for at, e, status in ((w13, 2, nv.Status.ERR_NONFINITE), (w2, 1, nv.Status.ERR_NONFINITE),
                          (w2, 3, nv.Status.OK), (None, 0, nv.Status.OK)):
        bad13, bad2 = list(w13), list(w2)
        if at is not None:
            s = at[1].clone().view(torch.uint8)
            s[e, 3, 5] = 0xFF
            (bad13 if at is w13 else bad2)[1] = s.view(torch.float8_e4m3fn)
        ws.fill_(255)
        nv.w4a16_moe(*on_gpu(x, ids, w, bad13, bad2), workspace=ws)
        assert nv.nvfp4_read_device_status(ws) == status, (e, status)


@pytest.mark.parametrize("M,E,k,H,I", [(1, 128, 8, 2048, 768), (48, 16, 4, 320, 720),
                                        (64, 32, 8, 1024, 528)])
def test_moe_deterministic_on_a_dirty_workspace_and_another_stream(M, E, k, H, I):
    args = on_gpu(*make(M, E, k, H, I, seed=6))
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(M, k, H, I), dtype=torch.uint8, device="cuda")
    first = nv.w4a16_moe(*args, workspace=ws)
    ws.fill_(255)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = nv.w4a16_moe(*args, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    for _ in range(20):
        nv.w4a16_moe(*args, out=again, workspace=ws)
    assert torch.equal(first, again)


def test_moe_unaligned_weights():
    """Codes on a 16-byte but not a 32-byte boundary: the narrow reads."""
    x, ids, w, w13, w2 = make(3, 4, 2, 512, 256, seed=9)
    dev = list(on_gpu(x, ids, w, w13, w2))
    want = nv.w4a16_moe(*dev)
    for at in (3, 6):
        buf = torch.empty(dev[at].numel() + 64, dtype=torch.uint8, device="cuda")
        moved = buf[16:16 + dev[at].numel()].view(dev[at].shape)
        moved.copy_(dev[at])
        dev[at] = moved
    assert torch.equal(nv.w4a16_moe(*dev), want)


def test_moe_graph_with_new_routing():
    M, E, k, H, I = 16, 24, 4, 512, 256
    x, ids, w, w13, w2 = make(M, E, k, H, I, seed=12)
    dev = on_gpu(x, ids, w, w13, w2)
    logits = torch.empty(M, E, device="cuda").normal_()
    out = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(M, k, H, I), dtype=torch.uint8, device="cuda")

    def layer():
        nv.moe_route(logits, k, expert_ids=dev[1], weights=dev[2])
        nv.w4a16_moe(*dev, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in range(3):
        logits.copy_(torch.randn(M, E, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        check(out, (x, dev[1].cpu(), dev[2].cpu(), w13, w2), f"replay {seed}")


def test_moe_empty_batch_and_refusals():
    x, ids, w, w13, w2 = make(3, 4, 2, 64, 32, seed=1)
    dev = on_gpu(x, ids, w, w13, w2)
    out = nv.w4a16_moe(dev[0][:0], dev[1][:0], dev[2][:0], *dev[3:])
    assert out.shape == (0, 64)
    with pytest.raises(nv.NVFP4Error) as err:  # more pairs than the call takes
        big = torch.zeros(4097, 64, dtype=torch.bfloat16, device="cuda")
        nv.w4a16_moe(big, torch.zeros(4097, 1, dtype=torch.int32, device="cuda"),
                     torch.zeros(4097, 1, device="cuda"), *dev[3:])
    assert err.value.status == nv.Status.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error) as err:
        nv.w4a16_moe(*dev, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == nv.Status.ERR_WORKSPACE
    with pytest.raises(ValueError, match="expert_ids"):
        nv.w4a16_moe(dev[0], dev[1].long(), *dev[2:])
    with pytest.raises(ValueError, match="w13_packed"):
        nv.w4a16_moe(*dev[:3], dev[3][:, :32].contiguous(), *dev[4:])
    with pytest.raises(ValueError, match="weights"):
        nv.w4a16_moe(dev[0], dev[1], dev[2].t().contiguous().t(), *dev[3:])
    with pytest.raises(ValueError, match="scoring"):
        nv.moe_route(torch.zeros(2, 8, device="cuda"), 2, scoring="relu")
    with pytest.raises(nv.NVFP4Error):
        nv.moe_route(torch.zeros(2, 8, device="cuda"), 9)


def test_memory_of_a_call_on_another_stream_is_not_given_out_early():
    args = make(64, 16, 4, 512, 256, seed=21)
    dev = on_gpu(*args)
    logits = torch.randn(64, 16, device="cuda")
    n = nv.w4a16_moe_workspace_bytes(64, 4, 512, 256)

    def fill():
        return [torch.full((b,), 255, dtype=torch.uint8, device="cuda") for b in (n, n, 4096, 4096)]

    nv.w4a16_moe(*dev)  # every kernel is loaded before the clock runs
    nv.moe_route(logits, 4)
    assert all(bool((j == 255).all()) for j in fill())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)  # the calls below wait for some 20 ms
    out = nv.w4a16_moe(*dev, stream=s)
    nv.moe_route(logits, 4, stream=s)
    junk = fill()
    torch.cuda.synchronize()
    assert all(bool((j == 255).all()) for j in junk)
    check(out, args)


@pytest.mark.parametrize("M,k", [(300, 8), (2048, 2)])
def test_moe_wide_without_any_expert(M, k):
    """Nothing for either product, places of an earlier use in the workspace."""
    x, ids, w, *weights = on_gpu(*make(M, 8, k, 256, 144, seed=31))
    ws = torch.empty(nv.w4a16_moe_workspace_bytes(M, k, 256, 144), dtype=torch.uint8, device="cuda")
    none = torch.full_like(ids, -1)
    for fill in (0, 1, 127, 255) * 5:
        ws.fill_(fill)
        assert bool((nv.w4a16_moe(x, none, w, *weights, workspace=ws) == 0).all())
