"""The operators around the products of this library, as measured cases.

What a mixture-of-experts decode step does between and after the NVFP4
products: the router's choice (``moe_route``), the whole expert layer for a
few tokens (``w4a16_moe``), and, behind the lm_head, the log probabilities of
given tokens with entropy, rank and top alternatives (``token_logprobs``) and
their gradient (``token_logprobs_backward``).

``run`` computes a case in plain torch operations in 32 bits, or, where
``own`` is true, by the library's calls; ``exact`` gives the same values from
the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding: the router of one token (latency)
        {"name": "route 1 token", "op": "route", "M": 1, "E": 128, "k": 8, "dtype": "bfloat16",
         "scoring": "softmax", "renorm": True},
        # a prompt's tokens routed at once, fp32 router logits, many experts
        {"name": "route prompt", "op": "route", "M": 16384, "E": 256, "k": 8, "dtype": "float32",
         "scoring": "sigmoid", "renorm": True},
        # one sequence decoding through the benchmark's expert layer (latency)
        {"name": "moe 1 token", "op": "moe", "M": 1, "E": 128, "k": 8, "H": 2048, "I": 768, "drop": 0.0},
        # a few sequences, wide experts whose sizes are not powers of two
        {"name": "moe 5 tokens 2880", "op": "moe", "M": 5, "E": 32, "k": 4, "H": 2880, "I": 2880, "drop": 0.0},
        # a decode batch: nearly every expert is read once (bandwidth)
        {"name": "moe 64 tokens", "op": "moe", "M": 64, "E": 128, "k": 8, "H": 2048, "I": 768, "drop": 0.0},
        # a large batch on one rank of two (half of the chosen experts live elsewhere), ragged inner size
        {"name": "moe 193 tokens of a shard", "op": "moe", "M": 193, "E": 64, "k": 8, "H": 2048, "I": 720,
         "drop": 0.5},
        # one sampled token's log probability and 20 alternatives (latency)
        {"name": "logprobs 1 row", "op": "logprobs", "M": 1, "N": 128256, "k": 20, "dtype": "float32",
         "pad": 0, "temp": 1.0},
        # a decode batch with a grammar's masks, logits of a padded vocabulary
        {"name": "logprobs 64 rows", "op": "logprobs", "M": 64, "N": 151936, "k": 8, "dtype": "float32",
         "pad": 64, "temp": 0.7},
        # scoring a few continuations: odd vocabulary, rows that start off a 16-byte boundary
        {"name": "logprobs odd vocabulary", "op": "logprobs", "M": 37, "N": 50257, "k": 5, "dtype": "bfloat16",
         "pad": 0, "temp": 1.0},
        # scoring a rollout for training: bf16 logits, no alternatives
        {"name": "logprobs rollout", "op": "logprobs", "M": 2048, "N": 128256, "k": 0, "dtype": "bfloat16",
         "pad": 0, "temp": 1.0},
        # the gradient of a short odd-sized batch, fp32
        {"name": "gradient odd vocabulary", "op": "grad", "M": 19, "N": 50257, "dtype": "float32", "pad": 0,
         "temp": 1.0},
        # the gradient of the rollout above
        {"name": "gradient rollout", "op": "grad", "M": 2048, "N": 128256, "dtype": "bfloat16", "pad": 0,
         "temp": 0.9},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, odd ones among them."""
    op = rng.choice(["route", "moe", "moe", "logprobs", "logprobs", "grad"])
    if op == "route":
        E = rng.randint(8, 256)
        return {"op": op, "M": _log_int(rng, 1, 16384), "E": E, "k": rng.randint(1, 8),
                "dtype": rng.choice(["bfloat16", "float32"]), "scoring": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.7}
    if op == "moe":
        while True:
            k = rng.randint(1, 8)
            E = rng.randint(max(8, k), 128)
            H, I = 64 * _log_int(rng, 8, 64), 16 * _log_int(rng, 16, 180)
            if 128 * 2048 * 768 >= E * H * I and 3072 not in (H, I, 2 * I):
                break
        return {"op": op, "M": _log_int(rng, 1, 256), "E": E, "k": k, "H": H, "I": I,
                "drop": rng.choice([0.0, 0.0, 0.25, 0.5])}
    while True:
        N = _log_int(rng, 1000, 262144)
        M = _log_int(rng, 1, 2048)
        dtype = rng.choice(["bfloat16", "float32"])
        if M * N * (4 if dtype == "float32" else 2) <= 2048 * 128256 * 2 and N != 3072:
            break
    case = {"op": op, "M": M, "N": N, "dtype": dtype, "pad": rng.choice([0, 0, 1, 64]),
            "temp": rng.choice([1.0, 1.0, 0.6, 1.3])}
    if op == "logprobs":
        case["k"] = rng.choice([0, 1, rng.randint(2, 20), rng.randint(21, 128)])
    return case


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _code_table():
    """Packed byte (two E2M1 codes) of each 16-bit random value, distributed
    as the codes of normal weights whose block maximum maps to 6."""
    edges = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    cdf = [math.erf(e / (3.2 * math.sqrt(2.0))) for e in edges]
    one = torch.tensor([sum(((r & 127) + 0.5) / 128 > c for c in cdf) | ((r >> 7) << 3)
                        for r in range(256)], dtype=torch.int64)
    one[one == 8] = 0  # a zero code carries no sign
    r = torch.arange(65536)
    return (one[r & 255] | (one[r >> 8] << 4)).to(torch.uint8).to(DEV)


def _experts(E, N, K, std, gen):
    """NVFP4 weights [E, N, K] as the quantizer leaves them: codes, block
    scales, one global scale per expert."""
    table = _code_table()
    packed = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // 16, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 26) // (N * K // 2))
    for e in range(0, E, step):
        n = min(step, E - e)
        r = torch.randint(0, 65536, (n, N, K // 2), device=DEV, generator=gen, dtype=torch.int32)
        packed[e:e + n] = table[r]
        s = 150.0 * torch.exp(0.22 * torch.randn(n, N, K // 16, device=DEV, generator=gen))
        scales[e:e + n] = s.clamp(max=448.0).to(torch.float8_e4m3fn)
    glob = std * 5.2 / 2688.0 * (0.8 + 0.4 * torch.rand(E, device=DEV, generator=gen))
    return packed, scales, glob


def _logits(case, gen):
    """Logits as an lm_head gives them: a broad bulk, a few likely tokens,
    some rows with half of the vocabulary masked, rows of a padded buffer."""
    M, N = case["M"], case["N"]
    dtype = getattr(torch, case["dtype"])
    buf = torch.empty(M, N + case["pad"], dtype=dtype, device=DEV)
    top = torch.randint(0, N, (M, 8), device=DEV, generator=gen)
    up = 4.0 + 8.0 * torch.rand(M, 8, device=DEV, generator=gen)
    masked = torch.rand(M, 1, device=DEV, generator=gen) < 0.2
    step = max(1, (1 << 27) // N)
    for m in range(0, M, step):
        x = 2.0 * torch.randn(min(step, M - m), buf.shape[1], device=DEV, generator=gen)
        if M > 8:
            hide = torch.rand(x.shape, device=DEV, generator=gen) < 0.5
            x.masked_fill_(hide & masked[m:m + step], float("-inf"))
        x.scatter_(1, top[m:m + step], up[m:m + step])
        buf[m:m + step] = x
    ids = torch.where(torch.rand(M, device=DEV, generator=gen) < 0.7, top[:, 0],
                      torch.randint(0, N, (M,), device=DEV, generator=gen))
    if M > 8:  # padding positions of a batch have no token
        ids = torch.where(torch.rand(M, device=DEV, generator=gen) < 0.05, -torch.ones_like(ids), ids)
    return buf[:, :N], ids


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case)
    if case["op"] == "route":
        dtype = getattr(torch, case["dtype"])
        st["logits"] = (1.5 * torch.randn(case["M"], case["E"], device=DEV, generator=gen)).to(dtype)
    elif case["op"] == "moe":
        M, E, k, H, I = (case[c] for c in ("M", "E", "k", "H", "I"))
        x = torch.randn(M, H, device=DEV, generator=gen)
        x[:, torch.randint(0, H, (4,), device=DEV, generator=gen)] *= 8.0  # outlier channels
        st["x"] = x.to(torch.bfloat16)
        st["w13"] = _experts(E, 2 * I, H, 0.02, gen)
        st["w2"] = _experts(E, H, I, 0.02, gen)
        r = torch.randn(M, E, device=DEV, generator=gen) + 0.5 * torch.randn(E, device=DEV, generator=gen)
        w, ids = torch.softmax(r, -1).topk(k, -1)
        st["weights"] = w / w.sum(-1, keepdim=True)
        gone = torch.rand(M, k, device=DEV, generator=gen) < case["drop"]  # experts of another rank
        st["ids"] = torch.where(gone, -torch.ones_like(ids), ids).to(torch.int32)
    else:
        st["logits"], st["tokens"] = _logits(case, gen)
        if case["op"] == "grad":
            M = case["M"]
            lse, ent = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
            step = max(1, (1 << 27) // case["N"])
            for m in range(0, M, step):
                z = st["logits"][m:m + step].float() / case["temp"]
                lse[m:m + step] = torch.logsumexp(z, -1)
                lp = z - lse[m:m + step, None]
                ent[m:m + step] = -(lp.exp() * lp.clamp(min=-1e4)).sum(-1)
            st["lse"], st["entropy"] = lse, ent
            # advantages of a policy gradient, and an entropy bonus
            st["g_lp"] = torch.randn(M, device=DEV, generator=gen) / M
            st["g_ent"] = torch.full((M,), 0.01 / M, device=DEV)
    return st


# ------------------------------------------------------------------- plain
def _dequant(packed, scales):
    """[..., N, K/2] codes and [..., N, K/16] block scales -> fp32 [..., N, K]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=DEV)
    pairs = torch.stack((lut[torch.arange(256, device=DEV) & 15], lut[torch.arange(256, device=DEV) >> 4]), -1)
    w = pairs[packed.int()].flatten(-2)
    return (w.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_route(st):
    x, k = st["logits"].float(), st["k"]
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :k]
    if st["scoring"] == "softmax":
        e = torch.exp(x - x.max(-1, keepdim=True).values)
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    w = s.gather(1, ids)
    if st["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w}


def _plain_moe(st):
    x, ids, I, E = st["x"].float(), st["ids"].long(), st["I"], st["E"]
    M, k = ids.shape
    here = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    (p13, s13, g13), (p2, s2, g2) = st["w13"], st["w2"]
    if M * k < E:  # the chosen experts' weights, one copy for each pair
        flat = at.flatten()
        gu = torch.einsum("pnk,pk->pn", _dequant(p13[flat], s13[flat]), x.repeat_interleave(k, 0))
        gu = (gu * g13[flat, None]).unflatten(0, (M, k))
        h = gu[..., :I] / (1.0 + torch.exp(-gu[..., :I])) * gu[..., I:]
        y = torch.einsum("pnk,pk->pn", _dequant(p2[flat], s2[flat]), h.flatten(0, 1)).unflatten(0, (M, k))
    else:  # every expert on every token, then the chosen ones
        gu = torch.einsum("enk,mk->emn", _dequant(p13, s13), x) * g13[:, None, None]
        h = gu[..., :I] / (1.0 + torch.exp(-gu[..., :I])) * gu[..., I:]
        y = torch.einsum("enk,emk->emn", _dequant(p2, s2), h)
        y = y[at, torch.arange(M, device=DEV)[:, None]]
    y = torch.where(here[..., None], y * (st["weights"] * g2[at])[..., None], 0.0)
    return {"out": y.sum(1).to(torch.bfloat16)}


def _plain_logprobs(st):
    raw, t, k = st["logits"].float(), st["tokens"], st["k"]
    M, N = raw.shape
    z = raw * (1.0 / st["temp"])
    top = z.max(-1, keepdim=True).values
    empty = torch.isneginf(top)
    top = torch.where(empty, 0.0, top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    logp = torch.where(empty, float("-inf"), z - lse)
    p = torch.where(empty, 0.0, e / total)
    ent = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    has = (t >= 0) & (t < N)
    tc = t.clamp(0, N - 1)[:, None]
    lp = torch.where(has, logp.gather(1, tc)[:, 0], 0.0)
    rank = torch.where(has, (raw > raw.gather(1, tc)).sum(-1) + 1, 0)
    # order key: value, then the lower index
    bits = torch.where(raw == 0, 0.0, raw).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 31) - torch.arange(N, device=DEV)
    top_ids = key.topk(k, -1).indices if k else torch.empty(M, 0, dtype=torch.int64, device=DEV)
    return {"logprobs": lp, "entropy": ent, "lse": lse[:, 0], "ranks": rank, "top_ids": top_ids,
            "top_logprobs": logp.gather(1, top_ids)}


def _plain_grad(st):
    raw, t = st["logits"], st["tokens"]
    M, N = raw.shape
    s = 1.0 / st["temp"]
    logp = raw.float() * s - st["lse"][:, None]
    p = torch.exp(logp)
    has = (t >= 0) & (t < N)
    a = torch.where(has, st["g_lp"], 0.0)
    d = -p * (a[:, None] + st["g_ent"][:, None] * torch.where(p > 0, logp + st["entropy"][:, None], 0.0))
    d.scatter_add_(1, t.clamp(0, N - 1)[:, None], a[:, None])
    return {"grad": (d * s).to(raw.dtype)}


# --------------------------------------------------------------------- run
def run(st):
    if not own:
        return {"route": _plain_route, "moe": _plain_moe, "logprobs": _plain_logprobs, "grad": _plain_grad}[st["op"]](st)
    import nvfp4_weight_only_rows_gb300 as nv

    if st["op"] == "route":
        ids, w = nv.moe_route(st["logits"], st["k"], scoring=st["scoring"], renormalize=st["renorm"])
        return {"ids": ids, "weights": w}
    if st["op"] == "moe":
        return {"out": nv.w4a16_moe(st["x"], st["ids"], st["weights"], *st["w13"], *st["w2"])}
    if st["op"] == "logprobs":
        lp, ent, lse, ranks, top_ids, top_lp = nv.token_logprobs(st["logits"], st["tokens"], st["k"],
                                                                 inv_temperature=1.0 / st["temp"])
        return {"logprobs": lp, "entropy": ent, "lse": lse, "ranks": ranks, "top_ids": top_ids,
                "top_logprobs": top_lp}
    return {"grad": nv.token_logprobs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"], st["g_lp"],
                                               st["g_ent"], inv_temperature=1.0 / st["temp"])}


def work(case):
    if case["op"] == "route":
        M, E, k = case["M"], case["E"], case["k"]
        return {"bytes": M * (E * (4 if case["dtype"] == "float32" else 2) + 8 * k), "flops": 5 * M * E}
    if case["op"] == "moe":
        M, E, k, H, I = (case[c] for c in ("M", "E", "k", "H", "I"))
        pairs = M * k * (1.0 - case["drop"])
        active = E * (1.0 - (1.0 - k * (1.0 - case["drop"]) / E) ** M)  # expected under even routing
        return {"bytes": active * 3 * H * I * 9 / 16 + 4 * M * H + 8 * M * k, "flops": 6 * pairs * H * I}
    size = 4 if case["dtype"] == "float32" else 2
    M, N = case["M"], case["N"]
    if case["op"] == "logprobs":
        return {"bytes": M * (N * size + 28 + 12 * case["k"]), "flops": 6 * M * N}
    return {"bytes": M * (2 * N * size + 24), "flops": 8 * M * N}


# ------------------------------------------------------------------- exact
def _exact_weights(packed, scales, glob):
    """One expert's weights [N, K] in 64 bits, from the format's definition:
    sign bit, two exponent bits with bias 1, one mantissa bit."""
    c = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.pow(2.0, (exp - 1).double()))
    w = torch.where(c >= 8, -mag, mag) * glob.double()
    return w * scales.double().repeat_interleave(16, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        x = st["logits"].double()
        # the k largest of distinct keys: the value, then the lower index
        ids = torch.argsort(-x, dim=-1, stable=True)[:, :case["k"]]
        s = torch.softmax(x, -1) if case["scoring"] == "softmax" else torch.sigmoid(x)
        w = torch.gather(s, 1, ids)
        return {"ids": None, "weights": w / w.sum(-1, keepdim=True) if case["renorm"] else w}
    if case["op"] == "moe":
        x, I = st["x"].double(), case["I"]
        out = torch.zeros(case["M"], case["H"], dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            m, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            if m.numel() == 0:
                continue
            a = x[m] @ _exact_weights(*(t[e] for t in st["w13"])).T
            h = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
            y = h @ _exact_weights(*(t[e] for t in st["w2"])).T
            out.index_add_(0, m, y * st["weights"][m, j].double()[:, None])
        return {"out": out}
    M, N = case["M"], case["N"]
    s, t = 1.0 / case["temp"], st["tokens"]
    has, tc = (t >= 0) & (t < N), t.clamp(0, N - 1)[:, None]
    parts, step = [], max(1, (1 << 26) // N)
    for m in range(0, M, step):
        rows = slice(m, m + step)
        z = st["logits"][rows].double() * s
        if case["op"] == "logprobs":
            lp = torch.log_softmax(z, -1)
            ent = torch.special.entr(lp.exp()).sum(-1)
            top = torch.sort(lp, dim=-1, descending=True).values[:, :case["k"]]
            parts.append((torch.where(has[rows], lp.gather(1, tc[rows])[:, 0], 0.0), ent, torch.logsumexp(z, -1), top))
        else:
            lp = z - st["lse"][rows, None].double()
            p = lp.exp()
            a, b = torch.where(has, st["g_lp"], 0.0)[rows, None].double(), st["g_ent"][rows, None].double()
            pull = torch.zeros_like(z).scatter_(1, tc[rows], 1.0) - p
            bonus = torch.special.entr(p) - p * st["entropy"][rows, None].double()
            parts.append((s * (a * pull + b * bonus),))
    if case["op"] == "grad":
        return {"grad": torch.cat([q[0] for q in parts])}
    lp, ent, lse, top = (torch.cat([q[i] for q in parts]) for i in range(4))
    return {"logprobs": lp, "entropy": ent, "lse": lse, "ranks": None, "top_ids": None, "top_logprobs": top}
