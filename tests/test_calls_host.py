"""What the compiled calls refuse of their tensors, on tensors without memory:
every refusal comes before anything is allocated or launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import nvfp4_weight_only_rows_gb300 as nv


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.fixture
def fake():
    if torch.cuda.device_count() == 1:  # such a tensor takes its device's context
        pytest.skip("tensors of a second device need none or two")
    with FakeTensorMode() as mode:
        yield mode


def empty(shape, dtype=torch.float32, device="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=device)


def moe_args():
    M, k, E, H, I = 3, 2, 4, 64, 32
    u8 = torch.uint8
    return [empty((M, H), torch.bfloat16), empty((M, k), torch.int32), empty((M, k)),
            empty((E, 2 * I, H // 2), u8), empty((E, 2 * I, H // 16), u8), empty((E,)),
            empty((E, H, I // 2), u8), empty((E, H, I // 16), u8), empty((E,))]


NAMES = ["x", "expert_ids", "weights", "w13_packed", "w13_scales", "w13_global", "w2_packed",
         "w2_scales", "w2_global"]


@pytest.mark.parametrize("at", range(1, 9))
def test_w4a16_moe_on_two_devices(fake, at):
    args = moe_args()
    args[at] = empty(args[at].shape, args[at].dtype, "cuda:1")
    with pytest.raises(ValueError, match=f"{NAMES[at]} is on cuda:1, not on cuda:0"):
        nv.w4a16_moe(*args)


def test_w4a16_moe_workspace(fake):
    args = moe_args()
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        nv.w4a16_moe(*args, workspace=empty((1 << 20,), torch.uint8, "cuda:1"))
    for view in (empty((256,), torch.uint8).expand(4096, 256), empty((1 << 20,), torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            nv.w4a16_moe(*args, workspace=view)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        nv.w4a16_moe(*args, workspace=empty((1 << 20,), torch.uint8, "cpu"))


def test_the_others_on_two_devices(fake):
    x, t, f, other = empty((4, 10)), empty((4,), torch.int64), empty((4,)), empty((4,), device="cuda:1")
    with pytest.raises(ValueError, match="bias is on cuda:1"):
        nv.moe_route(x, 2, bias=empty((10,), device="cuda:1"))
    with pytest.raises(ValueError, match="token_ids is on cuda:1"):
        nv.token_logprobs(x, empty((4,), torch.int64, "cuda:1"))
    for bad in (1, 2, 3, 4):
        args = [t, f, f, f, f]
        args[bad] = other
        with pytest.raises(ValueError, match="is on cuda:1, not on cuda:0"):
            nv.token_logprobs_backward(x, *args)


@pytest.mark.parametrize("name", ["expert_ids", "weights"])
def test_given_results_on_another_device(fake, name):
    dtype = {"expert_ids": torch.int32, "weights": torch.float32}[name]
    with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
        nv.moe_route(empty((4, 10)), 2, **{name: empty((4, 2), dtype, "cuda:1")})
    with pytest.raises(ValueError, match="out is on cuda:1"):
        nv.w4a16_moe(*moe_args(), out=empty((3, 64), torch.bfloat16, "cuda:1"))
    f = empty((4,))
    with pytest.raises(ValueError, match="out is on cuda:1"):
        nv.token_logprobs_backward(empty((4, 10)), empty((4,), torch.int64), f, f, f, f,
                                   out=empty((4, 10), device="cuda:1"))
