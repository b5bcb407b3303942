"""Argument checks of the router, the expert layer and the token log
probabilities at the C boundary (CPU only: every case fails before a CUDA
call)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    import nvfp4_weight_only_rows_gb300 as nv

    return nv.load_library()


vp = ctypes.c_void_p
fake, off2, off4, off8 = vp(1 << 20), vp((1 << 20) + 2), vp((1 << 20) + 4), vp((1 << 20) + 8)


def test_moe_route(lib):
    f = lib.moe_route
    assert f(fake, 0, -1, 8, 2, 0, 1, None, 1.0, fake, fake, None) == 1
    assert f(fake, 0, 4, 0, 1, 0, 1, None, 1.0, fake, fake, None) == 1
    assert f(fake, 0, 4, 513, 1, 0, 1, None, 1.0, fake, fake, None) == 1
    assert f(fake, 0, 4, 8, 9, 0, 1, None, 1.0, fake, fake, None) == 1     # k > E
    assert f(fake, 0, 4, 64, 33, 0, 1, None, 1.0, fake, fake, None) == 1   # k > 32
    assert f(fake, 0, 4, 8, 0, 0, 1, None, 1.0, fake, fake, None) == 1
    assert f(fake, 2, 4, 8, 2, 0, 1, None, 1.0, fake, fake, None) == 5     # dtype
    assert f(fake, 0, 4, 8, 2, 2, 1, None, 1.0, fake, fake, None) == 5     # scoring
    assert f(None, 0, 0, 8, 2, 0, 1, None, 1.0, None, None, None) == 0     # empty
    assert f(None, 0, 4, 8, 2, 0, 1, None, 1.0, fake, fake, None) == 3
    assert f(fake, 0, 4, 8, 2, 0, 1, None, 1.0, fake, None, None) == 3
    assert f(off2, 0, 4, 8, 2, 0, 1, None, 1.0, fake, fake, None) == 2
    assert f(fake, 0, 4, 8, 2, 0, 1, off2, 1.0, fake, fake, None) == 2


def test_w4a16_moe(lib):
    size = lib.w4a16_moe_workspace_bytes
    assert size(4, 2, 64, 40) == 0 and size(4, 2, 72, 32) == 0 and size(-1, 2, 64, 32) == 0
    assert size(4097, 1, 64, 32) == 0 and size(2049, 2, 64, 32) == 0 and size(1, 4097, 64, 32) == 0
    assert size(4, 2, 64, 32768 + 16) == 0 and size(4, 0, 64, 32) == 0
    assert size(4, 2, 64, 32) >= 4 * 2 * (64 + 2 * 32) * 4

    def f(M=4, k=2, H=64, I=32, E=8, ids=fake, x=fake, p13=fake, out=fake, code=1, ws=fake,
          n=1 << 24):
        return lib.w4a16_moe(x, M, k, H, I, E, ids, fake, p13, fake, fake, fake, fake, fake, out,
                             code, ws, n, None)

    for bad in (dict(M=-1), dict(k=0), dict(H=72), dict(I=40), dict(H=0), dict(E=0), dict(E=513),
                dict(M=2049), dict(H=32768 + 16)):
        assert f(**bad) == 1, bad
    assert f(code=2) == 5
    assert f(M=0, x=None, ws=None, n=0) == 0
    assert f(x=None) == 3 and f(ids=None) == 3 and f(p13=None) == 3 and f(out=None) == 3
    assert f(ws=None) == 4 and f(n=1024) == 4
    assert f(x=off8) == 2 and f(p13=off8) == 2 and f(ids=off2) == 2 and f(out=off8) == 2
    assert f(ws=vp((1 << 20) + 128)) == 2


def test_token_logprobs(lib):
    def f(M=4, N=100, ld=100, s=1.0, k=3, code=0, x=fake, t=fake, ids=fake, top=fake, ranks=fake):
        return lib.token_logprobs(x, code, M, N, ld, t, s, k, fake, fake, fake, ranks, ids, top,
                                  None)

    for bad in (dict(M=-1), dict(N=0), dict(ld=99), dict(s=0.0), dict(s=-1.0), dict(k=-1),
                dict(s=float("nan")), dict(s=float("inf")), dict(k=129, N=1000, ld=1000),
                dict(k=101), dict(N=1 << 31, ld=1 << 31)):
        assert f(**bad) == 1, bad
    assert f(code=3) == 5
    assert f(M=0, x=None) == 0
    assert f(x=None) == 3 and f(t=None) == 3 and f(ids=None) == 3 and f(top=None) == 3
    assert f(x=off2) == 2 and f(t=off4) == 2 and f(ranks=off4) == 2


def test_token_logprobs_backward(lib):
    def f(M=4, N=100, ld=100, s=1.0, code=0, x=fake, H=fake, gH=fake, out=fake, ldg=100):
        return lib.token_logprobs_backward(x, code, M, N, ld, fake, s, fake, H, fake, gH, out, ldg,
                                           None)

    for bad in (dict(M=-1), dict(N=0), dict(ld=99), dict(ldg=99), dict(s=0.0)):
        assert f(**bad) == 1, bad
    assert f(code=3) == 5
    assert f(M=0, x=None) == 0
    assert f(x=None) == 3 and f(out=None) == 3 and f(H=None) == 3
    assert f(out=off2) == 2 and f(H=off2) == 2
