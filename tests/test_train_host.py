"""Argument checks of the calls that train through NVFP4 weights, at the C
boundary and in Python (CPU only: every case fails before a CUDA call)."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    import nvfp4_weight_only_rows_gb300 as nv

    return nv.load_library()


vp = ctypes.c_void_p
fake, off2, off4, off8 = vp(1 << 20), vp((1 << 20) + 2), vp((1 << 20) + 4), vp((1 << 20) + 8)
BIG = 1 << 40


def test_lm_head_backward(lib):
    size = lib.w4a16_lm_head_backward_workspace_bytes
    assert size(4, 8, 24) == 0 and size(-1, 8, 32) == 0 and size(4, -1, 32) == 0 and size(4, 8, 0) == 0
    assert size(4, 8, 1 << 31) == 0
    assert size(0, 8, 32) >= 256 and size(4, 0, 32) >= 256
    assert size(4, 1001, 32) >= 4 * 1008 * 2  # fp16 rows of a multiple of 8
    # pieces: the workspace stops growing with the tokens
    assert size(1_000_000, 128256, 4096) < 1 << 30

    def f(g=fake, dt=0, M=4, N=8, p=fake, s=fake, gl=fake, K=32, dx=fake, out=1, ws=fake, n=BIG):
        return lib.w4a16_lm_head_backward(g, dt, M, N, p, s, gl, K, dx, out, ws, n, None)

    for bad in (dict(M=-1), dict(N=-1), dict(K=24), dict(K=0), dict(M=1 << 31), dict(N=1 << 31),
                dict(K=1 << 31)):
        assert f(**bad) == 1, bad
    assert f(dt=2) == 5 and f(out=7) == 5
    assert f(M=0, g=None, dx=None, ws=None, n=0) == 0
    assert f(g=None) == 3 and f(p=None) == 3 and f(s=None) == 3 and f(gl=None) == 3 and f(dx=None) == 3
    assert f(ws=None) == 4 and f(n=300) == 4
    assert f(g=off8) == 2 and f(p=off8) == 2 and f(s=off8) == 2 and f(gl=off2) == 2 and f(dx=off8) == 2
    assert f(ws=vp((1 << 20) + 128)) == 2


def test_cross_entropy(lib):
    size = lib.w4a16_cross_entropy_workspace_bytes
    assert size(4, 0, 32, 0) == 0 and size(4, 8, 24, 0) == 0 and size(-1, 8, 32, 1) == 0
    assert size(0, 8, 32, 1) >= 256
    assert size(200, 1001, 32, 1) >= size(200, 1001, 32, 0) + 200 * 1001 * 2
    assert size(1_000_000, 128256, 4096, 1) < 3 << 30

    def f(x=fake, M=4, K=32, p=fake, s=fake, gl=fake, N=8, t=fake, loss=fake, lse=fake, mean=fake,
          ws=fake, n=BIG):
        return lib.w4a16_cross_entropy(x, M, K, p, s, gl, N, t, loss, lse, mean, ws, n, None)

    for bad in (dict(M=-1), dict(N=0), dict(N=-1), dict(K=24), dict(K=0), dict(N=1 << 31)):
        assert f(**bad) == 1, bad
    assert f(M=0, x=None, t=None, ws=None, n=0) == 0
    for name in ("x", "p", "s", "gl", "t", "loss", "lse"):
        assert f(**{name: None}) == 3, name
    assert f(ws=None) == 4 and f(n=300) == 4 and f(mean=None, n=300) == 4
    for bad in (dict(x=off8), dict(p=off8), dict(s=off8), dict(gl=off2), dict(t=off4), dict(loss=off2),
                dict(lse=off2), dict(mean=off8), dict(ws=vp((1 << 20) + 128))):
        assert f(**bad) == 2, bad

    def g(mean=fake, M=4, K=32, p=fake, s=fake, gl=fake, N=8, t=fake, loss=fake, a=fake, b=None, dx=fake,
          out=1):
        return lib.w4a16_cross_entropy_backward(mean, M, K, p, s, gl, N, t, loss, a, b, dx, out, None)

    for bad in (dict(M=-1), dict(N=0), dict(K=24)):
        assert g(**bad) == 1, bad
    assert g(out=2) == 5
    assert g(M=0, mean=None, dx=None) == 0
    for name in ("mean", "p", "s", "gl", "t", "loss", "a", "dx"):
        assert g(**{name: None}) == 3, name
    for bad in (dict(mean=off8), dict(t=off4), dict(loss=off2), dict(a=off2), dict(b=off2), dict(dx=off8)):
        assert g(**bad) == 2, bad


def test_glu(lib):
    for size in (lib.w4a16_glu_workspace_bytes, lib.w4a16_glu_backward_workspace_bytes):
        assert size(4, 8, 24) == 0 and size(-1, 8, 32) == 0 and size(4, -1, 32) == 0
        assert size(4, 1 << 30, 32) == 0  # 2 I rows
        assert size(0, 8, 32) >= 256 and size(4, 0, 32) >= 256
    assert lib.w4a16_glu_backward_workspace_bytes(100, 999, 32) >= 100 * 1998 * 2

    def f(x=fake, M=4, K=32, p=fake, s=fake, gl=fake, I=8, act=0, o=fake, out=1, ws=fake, n=BIG):
        return lib.w4a16_glu(x, M, K, p, s, gl, I, act, o, out, ws, n, None)

    def g(dh=fake, dt=1, x=fake, M=4, K=32, p=fake, s=fake, gl=fake, I=8, act=1, o=fake, out=1, ws=fake,
          n=BIG):
        return lib.w4a16_glu_backward(dh, dt, x, M, K, p, s, gl, I, act, o, out, ws, n, None)

    for call in (f, g):
        for bad in (dict(M=-1), dict(I=-1), dict(K=24), dict(I=1 << 30)):
            assert call(**bad) == 1, bad
        assert call(out=2) == 5 and call(act=2) == 5 and call(act=-1) == 5
        assert call(M=0, x=None, o=None, ws=None, n=0) == 0
        for name in ("x", "p", "s", "gl", "o"):
            assert call(**{name: None}) == 3, name
        assert call(ws=None) == 4 and call(n=300) == 4
        for bad in (dict(x=off8), dict(p=off8), dict(s=off8), dict(gl=off2), dict(o=off8),
                    dict(ws=vp((1 << 20) + 128))):
            assert call(**bad) == 2, bad
    assert f(I=0, o=None) == 0
    assert g(dt=2) == 5 and g(dh=None) == 3 and g(dh=off8) == 2


# ------------------------------------------------------------------ Python
@pytest.fixture
def device(lib):
    if torch.cuda.device_count() == 1:  # such a tensor takes its device's context
        pytest.skip("tensors of a second device need none or two")
    with FakeTensorMode() as mode:
        yield mode


def empty(shape, dtype=torch.float32, device="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=device)


def weights(N=10, K=32, device="cuda:0"):
    return [empty((N, K // 2), torch.uint8, device), empty((N, K // 16), torch.uint8, device),
            empty((1,), device=device)]


def calls():
    import nvfp4_weight_only_rows_gb300 as nv

    M, N, K, I = 3, 10, 32, 5
    x, t, f = empty((M, K), torch.bfloat16), empty((M,), torch.int64), empty((M,))
    return {
        "back": (nv.w4a16_lm_head_backward, ["grad_logits", "packed", "scales", "global_scale"],
                 [empty((M, N)), *weights()]),
        "loss": (nv.w4a16_cross_entropy, ["x", "packed", "scales", "global_scale", "targets"], [x, *weights(), t]),
        "grad": (nv.w4a16_cross_entropy_backward,
                 ["mean", "packed", "scales", "global_scale", "targets", "loss", "grad_loss", "grad_lse"],
                 [empty((M, K)), *weights(), t, f, f, f]),
        "glu": (nv.w4a16_glu, ["x", "w13_packed", "w13_scales", "w13_global"], [x, *weights(2 * I)]),
        "glu_grad": (nv.w4a16_glu_backward, ["grad", "x", "w13_packed", "w13_scales", "w13_global"],
                     [empty((M, I)), x, *weights(2 * I)]),
    }


@pytest.mark.parametrize("name", ["back", "loss", "grad", "glu", "glu_grad"])
def test_tensors_that_do_not_fit(device, name):
    call, names, args = calls()[name]
    for at, what in enumerate(names):
        def refused(t, match):
            with pytest.raises(ValueError, match=match):
                call(*args[:at], t, *args[at + 1:])

        refused(args[at].to(torch.int16), f"{what} must")            # type
        if what != "grad" and at:
            refused(empty(args[at].shape, args[at].dtype, "cuda:1"), f"{what} is on cuda:1")
        refused(empty(args[at].shape, args[at].dtype, "cpu"), "must be a CUDA tensor|is on c")
        refused(empty((*args[at].shape, 2), args[at].dtype), "must")  # dimensions
        refused(7, f"{what} must be a tensor")
        if args[at].dim() == 2:
            rows, cols = args[at].shape
            refused(empty((rows, 2 * cols), args[at].dtype)[:, ::2], f"{what} must be contiguous")


def test_results_workspaces_and_names(device):
    all_calls = calls()
    for name, shape in (("back", (3, 32)), ("grad", (3, 32)), ("glu", (3, 5)), ("glu_grad", (3, 32))):
        call, _, args = all_calls[name]
        with pytest.raises(ValueError, match="out must be float32 or bfloat16"):
            call(*args, out=empty(shape, torch.float16))
        with pytest.raises(ValueError, match="out must have shape"):
            call(*args, out=empty((shape[0] + 1, shape[1])))
        with pytest.raises(ValueError, match="out is on cuda:1"):
            call(*args, out=empty(shape, device="cuda:1"))
        with pytest.raises(ValueError, match="out must be float32 or bfloat16"):
            call(*args, out_dtype=torch.float16)
    for name in ("back", "loss", "glu", "glu_grad"):
        call, _, args = all_calls[name]
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(*args, workspace=empty((1 << 20,), torch.uint8)[::2])
        with pytest.raises(ValueError, match="workspace is on cuda:1"):
            call(*args, workspace=empty((1 << 20,), torch.uint8, "cuda:1"))
    for name in ("glu", "glu_grad"):
        call, _, args = all_calls[name]
        with pytest.raises(ValueError, match="activation must be one of"):
            call(*args, activation="relu")
        odd = weights(11)
        with pytest.raises(ValueError, match="even number"):
            call(*args[:-3], *odd)
