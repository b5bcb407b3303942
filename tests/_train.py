"""Plain 64-bit forms of the calls that train through NVFP4 weights, written
from the formulas in include/nvfp4_lm_head.h, with error bounds that follow
each rounding of the kernels.

All tensors are on the GPU, where 64-bit products are quick enough."""
from __future__ import annotations

import math

import torch

from tests._operators import dequant, random_experts


def weight(N, K, seed, std=0.05):
    """(packed, scales, global f32[1]) with every code and scales over several
    binades, and W in 64 bits."""
    packed, scales, glob = random_experts(1, N, K, seed, std)
    q = packed[0].cuda(), scales[0].cuda(), glob[:1].cuda()
    return q, dequant(packed[0], scales[0], glob[0]).cuda()


def hidden(M, K, seed, outliers=2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    if outliers and K > outliers:
        x[:, torch.randint(0, K, (outliers,), generator=g)] *= 16.0
    return x.to(torch.bfloat16).cuda()


def sum_error(n):
    """Relative to the sum of magnitudes: the tensor cores add 16 products a
    step and drop bits below fp32, one unit in the last place a step at the
    most; a few more for parts that are joined and for scalings."""
    return (n / 16 + 24) * 2.0 ** -23


def product_error(x, W, n_part=None):
    """Of x W^T: the sums (in parts of n_part terms), and x in fp16 after a
    power of two, off by 2^-39 of the row's largest value."""
    mag = x.abs() @ W.abs().T
    K = W.shape[1]
    steps = min(K, n_part or K)
    return sum_error(steps) * mag + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * W.abs().sum(1)


def stored(value, tol, dtype):
    """The tolerance after rounding to dtype: half a step, eps / 2 of the
    value (bf16, with 8 significant bits: a step is 2^-7 of a power of two)."""
    half = torch.finfo(dtype).eps / 2
    return tol + half * (value.abs() + tol) + 2.0 ** -134  # subnormals of bf16


def within(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist(),
        (err / tol)[bad].max().item())


# -------------------------------------------------------------------- back
def back_error(d, W, d_error):
    """Of d W for d held with an error of d_error."""
    return d_error @ W.abs() + sum_error(d.shape[1]) * ((d.abs() + d_error) @ W.abs())


def back_reference(dy, W):
    """(dx, tolerance before its own rounding): bf16 gradients are exact in
    fp16 but for 2^-39 of the row's largest, fp32 ones are off by 2^-11 too."""
    d = dy.double()
    e = 2.0 ** -39 * d.abs().amax(1, keepdim=True).expand_as(d)
    if dy.dtype == torch.float32:
        e = e + 2.0 ** -11 * d.abs()
    return d @ W, back_error(d, W, e)


# --------------------------------------------------------------------- glu
def activation(g, name):
    """(act, act') in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def glu_reference(x, W, name):
    """(h, tolerance): |act'| < 1.13; the exponential, the division and the
    products take 2^-19 of the terms."""
    X, I = x.double(), W.shape[0] // 2
    gu, e = X @ W.T, product_error(X, W)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    act, _ = activation(g, name)
    tol = 1.13 * eg * (u.abs() + eu) + (act.abs() + 1.13 * eg) * eu + 2.0 ** -19 * (act * u).abs()
    return act * u, tol + 2.0 ** -126


def glu_grad_reference(dh, x, W, glob, name):
    """(dx, tolerance): |act''| < 1.2; dg and du are rounded to 11 bits, or by
    2^-36 of max|dh| sum|x| 2688 global where that is more."""
    X, D, I = x.double(), dh.double(), W.shape[0] // 2
    gu, e = X @ W.T, product_error(X, W)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    act, slope = activation(g, name)
    dg, du = D * u * slope, D * act
    eg_, eu_ = (D.abs() * (1.13 * eu + 1.2 * (u.abs() + eu) * eg) + 2.0 ** -18 * D.abs() * u.abs(),
                D.abs() * 1.13 * eg + 2.0 ** -18 * du.abs())
    floor = 2.0 ** -36 * D.abs().amax(1, keepdim=True) * X.abs().sum(1, keepdim=True) * 2688 * abs(float(glob))
    d = torch.cat((dg, du), 1)
    err = torch.cat((eg_, eu_), 1)
    err = err + 2.0 ** -11 * (d.abs() + err) + floor
    return d @ W, back_error(d, W, err)


# ----------------------------------------------------------- cross entropy
PART = 1792  # terms of a logit's sum that are added without a break, at the most


def entropy_reference(x, W, targets):
    """A dict of loss, lse, mean and what the gradient is made of, each with
    a tolerance `*_tol`."""
    X = x.double()
    N = W.shape[0]
    z, ez = X @ W.T, product_error(X, W, PART)
    # y = z / ln 2 is rounded twice, and 2^x is off by 2^-21 of itself
    ez = ez + 2.0 ** -22 * z.abs()
    has = (targets >= 0) & (targets < N)
    t = targets.clamp(0, N - 1)[:, None]
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    others = torch.where(has[:, None], p.scatter(1, t, 0.0), p)
    q = others.sum(1)  # 1 - p_t
    top = ez.amax(1)
    zt = z.gather(1, t)[:, 0]
    # log(1 + sum of the others over the target), with both in 64 bits
    loss = torch.where(has, torch.where(q < 0.5, -torch.log1p(-q), lse - zt), 0.0)
    r = {"loss": loss, "lse": lse, "p_t": 1 - q, "q": q}
    r["lse_tol"] = top + 2.0 ** -20 + 2.0 ** -21 * lse.abs()
    r["loss_tol"] = torch.where(has, q * 2 * top + 2.0 ** -19 * loss, 0.0) + 2.0 ** -140
    pW = others @ W.abs()
    r["mean"] = others @ W
    # a probability is stored in steps of 2^-39 of 2^r, r at most 8 above the
    # largest y but the target's, or 12 where that is more and y above -4
    y = torch.where(has[:, None], z.scatter(1, t, float("-inf")), z).amax(1) / math.log(2)
    r_at_most = torch.where(y >= -4.001, (y + 8).clamp(min=12.0), y + 8)
    step = 2.0 ** -39 * torch.exp2(r_at_most - lse / math.log(2))
    r["mean_tol"] = (2.0 ** -11 + 2 * top[:, None] + 2.0 ** -18 + sum_error(N)) * pW \
        + step[:, None] * W.abs().sum(0) \
        + 2.0 ** -125 * W.abs().sum(0)  # probabilities below fp32's smallest normal number, 2^-126
    r["has"], r["t"] = has, t[:, 0]
    return r


def entropy_grad_reference(r, W, a, b):
    """(dx, tolerance) for gradients a of loss and b of lse."""
    a = torch.where(r["has"], a.double(), 0.0)[:, None]
    b = b.double()[:, None]
    rows = torch.where(r["has"][:, None], W[r["t"]], 0.0)
    q = r["q"][:, None]
    dx = (a + b) * r["mean"] + (b * (1 - q) - a * q) * rows
    # q = 1 - exp(-loss): off by exp(-loss) of the loss's error, and 2^-21 of itself
    eq = (1 - q) * r["loss_tol"][:, None] + 2.0 ** -21 * q
    tol = (a + b).abs() * (r["mean_tol"] + 2.0 ** -22 * r["mean"].abs()) \
        + ((a.abs() + b.abs()) * eq + 2.0 ** -21 * (b * (1 - q) - a * q).abs() + 2.0 ** -22 * b.abs()) * rows.abs()
    return dx, tol
