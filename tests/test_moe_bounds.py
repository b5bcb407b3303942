"""The bounds of tests/_moe_bounds.py hold for the roundings they stand for
and not for coarser ones (on the CPU, every rounding emulated)."""
import pytest
import torch

from tests import _moe_bounds as mb
from tests.test_gpu_moe import make


def rows(outlier, seed=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(16, 1024, generator=g) * torch.rand(16, 1024, generator=g)
    v[:, 77] = outlier
    return v.double()


@pytest.mark.parametrize("outlier", [1.0, 30.0, 3000.0, 30000.0])
@pytest.mark.parametrize("pieces", [6, 8])
def test_pieces(outlier, pieces):
    v = rows(outlier)
    bound = mb.held_pieces(pieces)(v)
    assert bool(((mb.pieces_of(v.float(), pieces) - v.float().double()).abs() <= bound).all())
    # two pieces less, or all of a row on one scale (6e-6 of its largest: less
    # than six pieces of a block leave, unless the block is far below the row)
    if outlier >= 30.0 or pieces == 8:
        flat = (mb.pieces_of(v.float(), pieces, 1.0) - v.float().double()).abs()
        assert not bool((flat <= bound).all())
    fewer = (mb.pieces_of(v.float(), pieces - 2) - v.float().double()).abs()
    assert not bool((fewer <= bound).all())


@pytest.mark.parametrize("at", [1e-3, 1e-5, 1e-7])
def test_blocks_far_below_the_row(at):
    v = rows(1.0)
    v[:, 512:] *= at
    v = v.float()
    assert bool(((mb.pieces_of(v, 8) - v.double()).abs() <= mb.held_pieces(8)(v.double())).all())


def test_two_fp16():
    v = rows(30.0).float().double()
    assert bool(((mb.two_fp16(v) - v).abs() <= mb.held_two_fp16(v)).all())
    assert not bool(((mb.one_fp16(v) - v).abs() <= mb.held_two_fp16(v)).all())


def test_the_layers_bound_shows_a_coarser_h():
    """... in an fp32 result, and where a bf16 result is rounded once more."""
    x, ids, w, w13, w2 = make(4, 4, 2, 256, 256, seed=3)
    ref, tol = mb.layer(x, ids, w, w13, w2, mb.held_fp16, mb.held_two_fp16)
    half = torch.pow(2.0, torch.floor(torch.log2(ref.abs())) - 8)
    for hold, within in ((mb.two_fp16, True), (mb.one_fp16, False)):
        got, _ = mb.layer(x, ids, w, w13, w2, mb.held_fp16, mb.held_two_fp16, hold=hold)
        assert bool(((got - ref).abs() <= tol).all()) == within
        assert bool(((got.bfloat16().double() - ref).abs() <= tol + half).all()) == within
