"""Plain 64-bit forms of the router, the expert layer and the token log
probabilities, written from the formulas in include/nvfp4_lm_head.h, with
error bounds for the fp32 kernels."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def random_experts(E, N, K, seed, std=0.05):
    """NVFP4 weights [E, N, K] with random codes and block scales (every code,
    scales over several binades), on the CPU."""
    rng = np.random.default_rng(seed)
    packed = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
    s = np.exp(rng.normal(0.0, 0.6, (E, N, K // 16))) * 60.0
    scales = torch.from_numpy(s).clamp(max=448.0).to(torch.float8_e4m3fn)
    glob = torch.from_numpy((std / 200.0 * (0.5 + rng.random(E))).astype(np.float32))
    return packed, scales, glob


def dequant(packed, scales, glob):
    """[N, K/2], [N, K/16], scalar -> float64 [N, K]."""
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    return E2M1[codes] * scales.double().repeat_interleave(16, -1) * glob.double()


def moe_reference(x, ids, weights, w13, w2):
    """(out, tolerance of the fp32 output), both float64 [M, H].

    The bound follows each rounding of the kernel to first order: products
    are exact; an fp32 tensor-core sum of K terms in steps of 16, folded every
    256, is off by at most (K/16 + K/256 + 8) 2^-23 of the sum of magnitudes
    (one truncation a step); |silu'| <= 1.1; h is rounded to 11 bits, 2^-12
    of itself plus 2^-40 of its stage's largest; exp, the division and the
    scalings take 2^-20 of h; the combine adds k + 2 roundings."""
    M, H = x.shape
    I = w2[0].shape[2] * 2
    E = w2[0].shape[0]
    X = x.double()
    out = torch.zeros(M, H, dtype=torch.float64)
    tol = torch.zeros(M, H, dtype=torch.float64)
    rel = lambda K: (K / 16 + K / 256 + 8) * 2.0 ** -23  # noqa: E731
    k = ids.shape[1]
    for e in range(E):
        m, j = torch.nonzero(ids == e, as_tuple=True)
        if m.numel() == 0:
            continue
        A, B = dequant(*(t[e] for t in w13)), dequant(*(t[e] for t in w2))
        gu, mag = X[m] @ A.T, X[m].abs() @ A.abs().T
        g, u = gu[:, :I], gu[:, I:]
        silu = g / (1.0 + torch.exp(-g))
        h = silu * u
        dh = rel(H) * (1.1 * mag[:, :I] * u.abs() + silu.abs() * mag[:, I:]) \
            + (2.0 ** -12 + 2.0 ** -20) * h.abs() + 2.0 ** -40 * h.abs().amax(1, keepdim=True)
        w = weights[m, j].double()[:, None]
        y = w * (h @ B.T)
        ymag = w.abs() * (h.abs() @ B.abs().T)
        out.index_add_(0, m, y)
        tol.index_add_(0, m, w.abs() * (dh @ B.abs().T) + rel(I) * ymag + (k + 3) * 2.0 ** -23 * ymag)
    return out, tol


def bf16_half_ulp(v):
    a = v.abs().clamp(min=2.0 ** -126)
    return torch.pow(2.0, torch.floor(torch.log2(a)) - 8)


def logprobs_reference(logits, tokens, k, s):
    """float64 (logprobs, entropy, lse, ranks, top_ids, top_logprobs)."""
    raw = logits.double()
    M, N = raw.shape
    z = raw * s
    empty = torch.isneginf(z).all(1)
    top = torch.where(empty, 0.0, z.amax(1))
    e = torch.exp(z - top[:, None])
    lse = top + torch.log(e.sum(1))
    lp = torch.where(empty[:, None], float("-inf"), z - lse[:, None])
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    ent = torch.where(torch.isnan(lse), lse, ent)
    has = (tokens >= 0) & (tokens < N)
    t = tokens.clamp(0, N - 1)[:, None]
    chosen = torch.where(has, lp.gather(1, t)[:, 0], 0.0)
    ranks = torch.where(has, (raw > raw.gather(1, t)).sum(1) + 1, 0)
    key = torch.where(torch.isnan(raw), float("inf"), raw)
    ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
    return chosen, ent, lse, ranks, ids, lp.gather(1, ids)


def logprobs_grad_reference(logits, tokens, s, lse, entropy, a, b):
    """(float64 gradient, tolerance of an fp32 result)."""
    z = logits.double() * s
    M, N = z.shape
    lp = z - lse.double()[:, None]
    p = torch.exp(lp)
    has = (tokens >= 0) & (tokens < N)
    a = torch.where(has, a.double(), 0.0)[:, None]
    b = b.double()[:, None]
    hot = torch.zeros_like(z).scatter_(1, tokens.clamp(0, N - 1)[:, None], 1.0)
    live = p > 0
    lpf = torch.where(live, lp, 0.0)
    H = entropy.double()[:, None]
    g = s * (a * (hot - p) - b * p * torch.where(live, lpf + H, 0.0))
    # p: the argument is off by 2^-23 (|z| + |lse| + 2 |log p|), exp by 2^-22;
    # the factor by a few roundings of its terms
    arg = 2.0 ** -23 * (torch.where(live, z.abs(), 0.0) + lse.double().abs()[:, None] + 2 * lpf.abs())
    size = a.abs() + b.abs() * (lpf.abs() + H.abs())
    tol = s * p * size * (arg + 2.0 ** -20) + s * (a.abs() * hot) * 2.0 ** -22 + s * size * 2.0 ** -125
    empty = torch.isneginf(lse)[:, None]
    return torch.where(empty, 0.0, g), torch.where(empty, 0.0, tol)
