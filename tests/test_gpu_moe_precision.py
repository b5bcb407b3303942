"""What w4a16_moe holds of x and h on either route, with outlier channels
that the weights ignore: the token's other channels keep their precision,
and the result does not depend on how many tokens share the call."""
import pytest
import torch

import nvfp4_weight_only_rows_gb300 as nv
from tests import _moe_bounds as mb
from tests._operators import bf16_half_ulp
from tests.test_gpu_moe import make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()


def layer_args(M, E, k, H, I, outlier, seed, block=False):
    """Channel 5 is an outlier that the weights ignore, or with the 15 others of its block."""
    x, ids, w, w13, w2 = make(M, E, k, H, I, seed)
    if outlier:
        x[:, 5] = outlier * (1.0 + torch.arange(M) / M)
        w13[0][:, :, 2] &= 0x0F          # channel 5: high nibble of byte 2
        if block:
            w13[0][:, :, :8] = 0
        s = w13[1].float()               # h's channel 9, about 50 times the others
        s[:, [9, I + 9]] *= 7.0
        w13[1][:] = s.clamp(max=448.0).to(torch.float8_e4m3fn)
        w2[0][:, :, 4] &= 0x0F
    return x, ids, w, w13, w2


def check(args, out_dtype, steps, held_x, held_h):
    out = nv.w4a16_moe(*on_gpu(*args), out_dtype=out_dtype).double().cpu()
    ref, tol = mb.layer(*args, held_x, held_h, steps=steps)
    if out_dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(ref.abs() + tol)
    err = (out - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("M,E,k,H,I", [(1, 4, 1, 64, 256), (4, 4, 2, 256, 256), (8, 16, 4, 128, 512),
                                       (5, 8, 4, 272, 336)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("outlier", [0, 3000.0])
def test_few_pairs(M, E, k, H, I, out_dtype, outlier):
    args = layer_args(M, E, k, H, I, outlier, seed=M + I)
    check(args, out_dtype, 8, mb.held_fp16, mb.held_two_fp16)


@pytest.mark.parametrize("M,E,k,H,I", [(16, 4, 2, 256, 256), (40, 5, 3, 512, 128), (30, 4, 4, 336, 272)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("outlier", [0, 30.0, 3000.0, 30000.0])
def test_fp4_route(M, E, k, H, I, out_dtype, outlier):
    args = layer_args(M, E, k, H, I, outlier, seed=M + I)
    held = mb.held_pieces(6 if out_dtype == torch.bfloat16 else 8)
    check(args, out_dtype, 16, held, held)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("outlier", [3000.0, 30000.0])
def test_fp4_route_beside_an_ignored_block(out_dtype, outlier):
    args = layer_args(64, 4, 2, 2048, 32, outlier, seed=2, block=True)
    held = mb.held_pieces(6 if out_dtype == torch.bfloat16 else 8)
    check(args, out_dtype, 16, held, held)
