"""Training through frozen NVFP4 weights, as measured cases.

Three operators on the packed weights that ``nvfp4_quantize_rows`` leaves:
the softmax cross entropy over the vocabulary of an lm_head without its
logits (``w4a16_cross_entropy``) and its gradient in the hidden states
(``w4a16_cross_entropy_backward``), the gated feed-forward block with its
gradient (``w4a16_glu``, ``w4a16_glu_backward``), and the product back through
a packed weight (``w4a16_lm_head_backward``).

``run`` computes a case in plain torch operations in 32 bits, or, where
``own`` is true, by the library's calls; ``exact`` gives the same values from
the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROWS = 1 << 26  # weight values made or dequantized at a time


# ------------------------------------------------------------------ cases
def listed():
    return [
        # scoring one more token of one sequence: the whole head read for it (latency, bandwidth)
        {"name": "loss 1 token", "op": "loss", "M": 1, "N": 128256, "K": 4096, "z": 0.0},
        # evaluation of a text: losses only
        {"name": "loss 2048 tokens", "op": "loss", "M": 2048, "N": 128256, "K": 4096, "z": 0.0},
        # a short odd-sized batch of a small model, rows that no 256 divides, with a penalty on lse
        {"name": "training odd vocabulary", "op": "train", "M": 37, "N": 50257, "K": 1040, "z": 1e-4},
        # a micro-batch of a middle-sized model
        {"name": "training 600 tokens", "op": "train", "M": 600, "N": 32000, "K": 2880, "z": 0.0},
        # a training step's loss and gradient over the benchmark's head
        {"name": "training 2048 tokens", "op": "train", "M": 2048, "N": 128256, "K": 4096, "z": 1e-4},
        # one token decoding through a dense layer (latency, bandwidth)
        {"name": "glu 1 token", "op": "glu", "M": 1, "K": 4096, "I": 14336, "act": "silu"},
        # a prompt or a training batch through the same layer
        {"name": "glu 2048 tokens", "op": "glu", "M": 2048, "K": 4096, "I": 14336, "act": "silu"},
        # the gradient of a few packed sequences, sizes that are not powers of two
        {"name": "glu gradient 203 tokens", "op": "glu_grad", "M": 203, "K": 2880, "I": 2880, "act": "gelu_tanh"},
        # the gradient of a training batch
        {"name": "glu gradient 2048 tokens", "op": "glu_grad", "M": 2048, "K": 4096, "I": 14336, "act": "silu"},
        # back through a down projection: a few tokens
        {"name": "back 8 tokens", "op": "back", "M": 8, "N": 4096, "K": 14336, "dtype": "bfloat16"},
        # gradients of an odd number of logits, fp32
        {"name": "back odd rows", "op": "back", "M": 77, "N": 4099, "K": 1008, "dtype": "float32"},
        # a training batch back through a down projection
        {"name": "back 2048 tokens", "op": "back", "M": 2048, "N": 4096, "K": 14336, "dtype": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, odd ones among them."""
    op = rng.choice(["loss", "train", "train", "glu", "glu_grad", "back"])
    M = _log_int(rng, 1, 2048)
    K = 16 * _log_int(rng, 16, 320)
    if op in ("loss", "train"):
        N = _log_int(rng, 1000, 151936)
        while M * N * K > 2048 * 128256 * 4096:
            N = _log_int(rng, 1000, 151936)
        return {"op": op, "M": M, "N": N, "K": K, "z": rng.choice([0.0, 1e-4]) if op == "train" else 0.0}
    if op == "back":
        return {"op": op, "M": M, "N": _log_int(rng, 100, 16384), "K": 16 * _log_int(rng, 16, 896),
                "dtype": rng.choice(["bfloat16", "float32"])}
    return {"op": op, "M": M, "K": K, "I": _log_int(rng, 200, 14336), "act": rng.choice(["silu", "gelu_tanh"])}


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


def _weight(N, K, std, gen):
    """An NVFP4 weight [N, K] as the quantizer leaves it: codes, block scales, global scale."""
    table = _code_table()
    packed = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(N, K // 16, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, ROWS // K)
    for n in range(0, N, step):
        m = min(step, N - n)
        packed[n:n + m] = table[torch.randint(0, 65536, (m, K // 2), device=DEV, generator=gen, dtype=torch.int32)]
        s = 150.0 * torch.exp(0.22 * torch.randn(m, K // 16, device=DEV, generator=gen))
        scales[n:n + m] = s.clamp(max=448.0).to(torch.float8_e4m3fn)
    glob = torch.full((1,), std * 5.2 / 2688.0, device=DEV)
    return packed, scales, glob


def _hidden(M, K, gen):
    """Normalised hidden states with a few outlier channels."""
    x = torch.randn(M, K, device=DEV, generator=gen)
    x[:, torch.randint(0, K, (4,), device=DEV, generator=gen)] *= 8.0
    return x


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case)
    M, K = case["M"], case["K"]
    if case["op"] in ("loss", "train"):
        N = case["N"]
        st["w"] = packed, scales, glob = _weight(N, K, 1.3 / math.sqrt(K), gen)
        t = torch.randint(0, N, (M,), device=DEV, generator=gen)
        # the model knows most targets: their rows lie in the hidden state, log probabilities from about -10 to 0
        rows = _dequant(packed[t], scales[t]) * glob
        pull = 22.0 * torch.rand(M, 1, device=DEV, generator=gen) * (torch.rand(M, 1, device=DEV, generator=gen) < 0.8)
        x = torch.randn(M, K, device=DEV, generator=gen) + pull * rows / (rows * rows).sum(-1, keepdim=True)
        st["x"] = x.to(torch.bfloat16)
        if M > 8:  # positions of a prompt or of padding have no target
            t = torch.where(torch.rand(M, device=DEV, generator=gen) < 0.1, torch.full_like(t, -100), t)
        st["targets"] = t
        st["g"] = torch.where(t >= 0, 1.0 / max(1, M), 0.0)
    elif case["op"] in ("glu", "glu_grad"):
        st["w"] = _weight(2 * case["I"], K, 1.0 / math.sqrt(K), gen)
        st["x"] = _hidden(M, K, gen).to(torch.bfloat16)
        if case["op"] == "glu_grad":
            st["dh"] = (1e-4 * torch.randn(M, case["I"], device=DEV, generator=gen)).to(torch.bfloat16)
    else:
        st["w"] = _weight(case["N"], K, 0.02, gen)
        size = torch.exp(torch.randn(M, 1, device=DEV, generator=gen))  # tokens weigh differently
        dy = 1e-4 * size * torch.randn(M, case["N"], device=DEV, generator=gen)
        st["dy"] = dy.to(getattr(torch, case["dtype"]))
    return st


# ------------------------------------------------------------------- plain
def _dequant(packed, scales):
    """[N, K/2] codes and [N, K/16] block scales -> fp32 [N, K], without the global scale."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=DEV)
    pairs = torch.stack((lut[torch.arange(256, device=DEV) & 15], lut[torch.arange(256, device=DEV) >> 4]), -1)
    w = pairs[packed.int()].flatten(-2)
    return (w.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _pieces(packed, scales):
    """(first row, fp32 rows) of the weight, piece by piece."""
    N, step = packed.shape[0], max(1, ROWS // (2 * packed.shape[1]))
    for n in range(0, N, step):
        yield n, _dequant(packed[n:n + step], scales[n:n + step])


def _plain_product(x, w):
    packed, scales, glob = w
    return torch.cat([x @ rows.T for _, rows in _pieces(packed, scales)], 1) * glob


def _plain_back(dy, w):
    packed, scales, glob = w
    dx = torch.zeros(dy.shape[0], packed.shape[1] * 2, device=DEV)
    for n, rows in _pieces(packed, scales):
        dx += dy[:, n:n + rows.shape[0]] @ rows
    return (dx * glob).to(torch.bfloat16)


def _plain_entropy(st):
    N, t, a = st["N"], st["targets"], st["g"]
    z = _plain_product(st["x"].float(), st["w"])
    has = (t >= 0) & (t < N)
    tc = t.clamp(0, N - 1)[:, None]
    top = z.max(-1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    out = {"loss": torch.where(has, lse - z.gather(1, tc)[:, 0], 0.0), "lse": lse}
    if st["op"] == "train":
        del z
        b = 2.0 * st["z"] * lse * a
        p = e.div_(total)
        # p - 1 of the target by the sum of the others where it is near 1
        others = p.scatter(1, tc, 0.0).sum(-1)
        pt = p.gather(1, tc)[:, 0]
        d = p.mul_((torch.where(has, a, 0.0) + b)[:, None])
        d.scatter_(1, tc, torch.where(has, b * pt - a * others, b * pt)[:, None])
        out["dx"] = _plain_back(d, st["w"])
    return out


def _plain_act(g, name):
    """(activation, its derivative)."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    v = c * (g + 0.044715 * g * g * g)
    s = 1.0 / (1.0 + torch.exp(-2.0 * v))  # (1 + tanh v) / 2
    return g * s, s + g * s * (1.0 - s) * 2.0 * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_glu(st):
    I = st["I"]
    gu = _plain_product(st["x"].float(), st["w"])
    g, u = gu[:, :I], gu[:, I:]
    a, da = _plain_act(g, st["act"])
    if st["op"] == "glu":
        return {"h": (a * u).to(torch.bfloat16)}
    dh = st["dh"].float()
    return {"dx": _plain_back(torch.cat((dh * u * da, dh * a), 1), st["w"])}


# --------------------------------------------------------------------- run
def run(st):
    op = st["op"]
    if not own:
        if op in ("loss", "train"):
            return _plain_entropy(st)
        return {"dx": _plain_back(st["dy"].float(), st["w"])} if op == "back" else _plain_glu(st)
    import nvfp4_weight_only_rows_gb300 as nv

    if op == "loss":
        loss, lse = nv.w4a16_cross_entropy(st["x"], *st["w"], st["targets"])
        return {"loss": loss, "lse": lse}
    if op == "train":
        loss, lse, mean = nv.w4a16_cross_entropy(st["x"], *st["w"], st["targets"], with_mean=True)
        b = 2.0 * st["z"] * lse * st["g"] if st["z"] else None
        return {"loss": loss, "lse": lse,
                "dx": nv.w4a16_cross_entropy_backward(mean, *st["w"], st["targets"], loss, st["g"], b)}
    if op == "glu":
        return {"h": nv.w4a16_glu(st["x"], *st["w"], activation=st["act"])}
    if op == "glu_grad":
        return {"dx": nv.w4a16_glu_backward(st["dh"], st["x"], *st["w"], activation=st["act"])}
    return {"dx": nv.w4a16_lm_head_backward(st["dy"], *st["w"])}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] in ("loss", "train"):
        N, train = case["N"], case["op"] == "train"
        return {"bytes": N * K * 9 / 16 + M * (2 * K + 16) + (M * (2 * K + 4) if train else 0),
                "flops": (4 if train else 2) * M * N * K}
    if case["op"] == "back":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["N"] * K * 9 / 16 + M * case["N"] * size + 2 * M * K, "flops": 2 * M * case["N"] * K}
    I, grad = case["I"], case["op"] == "glu_grad"
    return {"bytes": 2 * I * K * 9 / 16 + 2 * M * (K + I) + (2 * M * K if grad else 0),
            "flops": (8 if grad else 4) * M * I * K}


# ------------------------------------------------------------------- exact
def _exact_weights(packed, scales, glob):
    """Weights [N, K] in 64 bits, from the format's definition: sign bit, two
    exponent bits with bias 1, one mantissa bit."""
    c = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.pow(2.0, (exp - 1).double()))
    w = torch.where(c >= 8, -mag, mag) * glob.double()
    return w * scales.double().repeat_interleave(16, dim=-1)


def _exact_rows(w, step):
    packed, scales, glob = w
    for n in range(0, packed.shape[0], step):
        yield slice(n, min(n + step, packed.shape[0])), _exact_weights(packed[n:n + step], scales[n:n + step], glob)


def exact(case, seed):
    if work(case)["flops"] > 1e13:  # too long in 64 bits
        return None
    st = prepare(case, seed)
    M, K, w = case["M"], case["K"], st["w"]
    step = max(1, (1 << 25) // K)
    if case["op"] == "back":
        dx = torch.zeros(M, K, dtype=torch.float64, device=DEV)
        for rows, W in _exact_rows(w, step):
            dx.addmm_(st["dy"][:, rows].double(), W)
        return {"dx": dx}
    x = st["x"].double()
    z = torch.empty(M, w[0].shape[0], dtype=torch.float64, device=DEV)
    for rows, W in _exact_rows(w, step):
        z[:, rows] = x @ W.T
    if case["op"] in ("loss", "train"):
        t, N = st["targets"], case["N"]
        has, tc = (t >= 0) & (t < N), t.clamp(0, N - 1)[:, None]
        lse = torch.logsumexp(z, -1)
        out = {"loss": torch.where(has, lse - z.gather(1, tc)[:, 0], 0.0), "lse": lse}
        if case["op"] == "loss":
            return out
        a = torch.where(has, st["g"], 0.0).double()
        d = (a + 2.0 * case["z"] * lse * st["g"].double())[:, None] * (z - lse[:, None]).exp()
        d.scatter_add_(1, tc, -a[:, None])
        out["dx"] = torch.zeros(M, K, dtype=torch.float64, device=DEV)
        for rows, W in _exact_rows(w, step):
            out["dx"].addmm_(d[:, rows], W)
        return out
    I, F = case["I"], torch.nn.functional
    with torch.enable_grad():
        g = z[:, :I].clone().requires_grad_(True)
        act = F.silu(g) if case["act"] == "silu" else F.gelu(g, approximate="tanh")
        if case["op"] == "glu":
            return {"h": act.detach() * z[:, I:]}
        dh = st["dh"].double()
        (dg,) = torch.autograd.grad(act, g, dh * z[:, I:])
    d = torch.cat((dg, dh * act.detach()), 1)
    dx = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for rows, W in _exact_rows(w, step):
        dx.addmm_(d[:, rows], W)
    return {"dx": dx}
