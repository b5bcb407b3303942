"""The expert layer in 64 bits with an error bound that follows what each
route of w4a16_moe documents for the numbers it holds, and, on the CPU, the
roundings that those bounds have to tell apart."""
from __future__ import annotations

import torch

from tests._operators import dequant


def blocks_max(v, n):
    """The largest magnitude of each n consecutive values of a row, at every one of them."""
    K = v.shape[1]
    pad = torch.nn.functional.pad(v.abs(), (0, -K % n))
    return pad.unflatten(1, (-1, n)).amax(2).repeat_interleave(n, 1)[:, :K]


def held_fp16(v):
    """x on the few-pair route: fp16 after a power of two per 256 values, exact for a
    bf16 within 2^28 of the largest of them (2^14 .. 2^15 then, half a step of
    the fp16 subnormals is 2^-25)."""
    return 2.0 ** -39 * blocks_max(v, 256)


def held_two_fp16(v):
    """h there: what a first fp16 leaves, at most 2^-11, is held by a second."""
    return 2.0 ** -22 * v.abs() + 2.0 ** -39 * blocks_max(v, 256)


def held_pieces(pieces):
    """x and h on the FP4 route: at most 0.177 of a block of 16 is left by
    each NVFP4 piece.  The residual is multiplied by 4 before the next, on a
    row whose largest value is 2^10 .. 2^11; a scale below the E4M3 normals is
    off by 2^-10, that is 6 2^-10 of a value, at 4^-q of the row's scale in
    piece q.  Summed over the pieces that is below 3.5 times the last one's."""
    def bound(v):
        return 1.001 * 0.1771 ** pieces * blocks_max(v, 16) + \
            3.5 * 6 * 2.0 ** -20 * 4.0 ** (1 - pieces) * v.abs().amax(1, keepdim=True)
    return bound


def layer(x, ids, weights, w13, w2, held_x, held_h, steps=16, hold=None):
    """(out, tolerance of an fp32 result), float64 [M, H].  hold(h): h as a route
    would hold it, for `out` (for tests of the bound itself).

    Products are exact.  A tensor-core sum of K terms, one truncation per
    `steps` of them and one fold per 256, is off by (K / steps + K / 256 + 16)
    2^-23 of the sum of magnitudes.  |silu'| <= 1.1; exp of a rounded argument
    is off by |g| 2^-23, it and the division and scalings by 2^-20.  The
    combine adds k + 3 roundings."""
    M, H = x.shape
    E, I = w2[0].shape[0], w2[0].shape[2] * 2
    X = x.double()
    out, tol = torch.zeros(M, H, dtype=torch.float64), torch.zeros(M, H, dtype=torch.float64)
    k = ids.shape[1]

    def rel(K):
        return (K / steps + K / 256 + 16) * 2.0 ** -23

    for e in range(E):
        m, j = torch.nonzero(ids == e, as_tuple=True)
        if m.numel() == 0:
            continue
        A, B = dequant(*(t[e] for t in w13)), dequant(*(t[e] for t in w2))
        gu = X[m] @ A.T
        dgu = rel(H) * (X[m].abs() @ A.abs().T) + held_x(X[m]) @ A.abs().T
        g, u = gu[:, :I], gu[:, I:]
        silu = g / (1.0 + torch.exp(-g))
        h = silu * u
        dh = 1.1 * dgu[:, :I] * (u.abs() + dgu[:, I:]) + silu.abs() * dgu[:, I:] \
            + (2.0 ** -20 + g.abs() * 2.0 ** -23) * h.abs() + held_h(h)
        w = weights[m, j].double()[:, None]
        out.index_add_(0, m, w * ((h if hold is None else hold(h)) @ B.T))
        ymag = w.abs() * (h.abs() @ B.abs().T)
        tol.index_add_(0, m, w.abs() * (dh @ B.abs().T) + (rel(I) + (k + 3) * 2.0 ** -23) * ymag)
    return out, tol


# ------------------------------------------------- what the bounds tell apart
_GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e2m1(q):
    """To the nearest code, ties to the even one."""
    a = q.abs().clamp(max=6.0)
    mid = (_GRID[1:] + _GRID[:-1]) / 2
    i = torch.searchsorted(mid, a)
    i = torch.where((i < 7) & (a == mid[i.clamp(max=6)]) & (i % 2 == 1), i + 1, i)
    return torch.sign(q) * _GRID[i]


def pieces_of(v, pieces, grow=4.0):
    """v [rows, K] as `pieces` NVFP4 values, the residual times `grow` before each next."""
    up = 2.0 ** (10 - torch.floor(torch.log2(v.abs().amax(1, keepdim=True))))
    r = (v * up).float().unflatten(1, (-1, 16))
    total, f = torch.zeros(r.shape, dtype=torch.float64), 1.0
    for _ in range(pieces):
        s = (r.abs().amax(2, keepdim=True) * (1 / 6)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        q = _e2m1(torch.where(s == 0, 0.0, r / s))
        total += (q * s).double() * f
        r = (r - q * s) * grow
        f /= grow
    return total.flatten(1) / up.double()


def one_fp16(v):
    up = 2.0 ** (14 - torch.floor(torch.log2(blocks_max(v, 256))))
    return (v * up).half().double() / up


def two_fp16(v):
    up = 2.0 ** (14 - torch.floor(torch.log2(blocks_max(v, 256))))
    hi = (v * up).float().half()
    lo = ((v * up).float() - hi.float()).half()
    return (hi.double() + lo.double()) / up
