"""Shapes of the router and of the expert layer that are shown to take the
route, tile and scan they are meant for."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests import _moe_bounds as mb
from tests._operators import bf16_half_ulp
from tests._routes import kernels
from tests.test_gpu_moe import make, on_gpu, route_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def check(args, out_dtype, fp4):
    dev = on_gpu(*args)
    out = nv.w4a16_moe(*dev, out_dtype=out_dtype).double().cpu()
    if fp4:
        held = mb.held_pieces(6 if out_dtype == torch.bfloat16 else 8)
        ref, tol = mb.layer(*args, held, held)
    else:
        ref, tol = mb.layer(*args, mb.held_fp16, mb.held_two_fp16, steps=8)
    if out_dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(ref.abs() + tol)
    err = (out - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    names = kernels(lambda: nv.w4a16_moe(*dev, out_dtype=out_dtype))
    assert any("moe_tc_kernel" in n for n in names) == fp4, names
    assert any("moe_gemm_kernel" in n for n in names) != fp4, names


# FP4 route: tiles of 8 pairs (up to 8 tokens), more than two experts a lane
# of the scan, up to 64 slots of a token, long rows
@pytest.mark.parametrize("M,E,k,H,I", [(8, 8, 6, 256, 272), (1, 8, 64, 720, 1200), (7, 3, 3, 4096, 528),
                                       (8, 512, 8, 1024, 816), (60, 512, 64, 128, 112),
                                       (33, 300, 60, 128, 208), (450, 73, 9, 64, 80),
                                       (64, 65, 33, 128, 336), (9, 4, 8, 8192, 464)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_moe_fp4_shapes(M, E, k, H, I, out_dtype):
    args = make(M, max(E, k), k, H, I, seed=M + H + 5) if E >= k else repeated(M, E, k, H, I)
    args[1][M // 2, 0] = -1
    check(args, out_dtype, True)


def repeated(M, E, k, H, I):
    x, _, w, w13, w2 = make(M, E, 1, H, I, seed=M + H + 5)
    g = torch.Generator().manual_seed(M)
    return x, torch.randint(0, E, (M, k), generator=g, dtype=torch.int32), \
        torch.rand(M, k, generator=g), w13, w2


# few-pair route: one expert with 9 to 16, 17 to 32 and more pairs
@pytest.mark.parametrize("M,E,k,H,I", [(12, 64, 2, 1024, 512), (32, 64, 2, 1024, 512),
                                       (100, 64, 2, 512, 256), (29, 64, 2, 272, 336), (1, 200, 70, 128, 80)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_moe_popular_expert(M, E, k, H, I, out_dtype):
    args = make(M, E, k, H, I, seed=M + H + 7)
    args[1][:, 0] = 3
    check(args, out_dtype, False)


@pytest.mark.parametrize("M,E,k", [(7, 24, 6), (300, 100, 8), (129, 256, 8), (40, 384, 8), (5, 512, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("apart", [0.25, 0.0])
def test_route_with_a_bias(M, E, k, dtype, scoring, apart):
    """Logits on a grid of 1/16, so that scores tie exactly or are further apart
    than fp32 rounds them, with biases 0.25 apart or none to speak of."""
    g = torch.Generator().manual_seed(M + E)
    x = (torch.randint(-8, 9, (M, E), generator=g) / 16.0).to(dtype)
    bias = torch.randperm(E, generator=g).float() * apart
    ids, w = nv.moe_route(x.cuda(), k, scoring=scoring, bias=bias.cuda(), scale=2.5)
    want_ids, want_w = route_reference(x, k, scoring, True, bias, 2.5)
    assert torch.equal(ids.cpu().long(), want_ids)
    assert bool(((w.cpu().double() - want_w).abs() <= (E + 16) * 2.0 ** -23 * want_w).all())
    _, raw = nv.moe_route(x.cuda(), k, scoring=scoring, bias=bias.cuda(), renormalize=False)
    _, want_raw = route_reference(x, k, scoring, False, bias, 1.0)
    assert bool(((raw.cpu().double() - want_raw).abs() <= (E + 16) * 2.0 ** -23 * want_raw).all())
