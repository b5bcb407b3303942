"""One decode step of a mixture-of-experts model's tail, and its gradient.

    python examples/moe_rollout_step.py [--tokens 4] [--steps 3]

The weights are random.  What runs, in the order a rollout engine runs it:

1. the bf16 expert and lm_head weights are quantized online
   (``nvfp4_quantize_rows``);
2. each step routes the hidden states (``moe_route``), runs the expert layer
   (``w4a16_moe``), the lm_head (``w4a16_lm_head``) and scores the token it
   picked with its entropy and alternatives (``token_logprobs``), all in one
   CUDA graph that is replayed as the hidden states change;
3. a policy-gradient step turns advantages and an entropy bonus into the
   gradient of the logits (``token_logprobs_backward``) and of the hidden
   states.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import nvfp4_weight_only_rows_gb300 as nv


def quantize_experts(W: torch.Tensor):
    """bf16 [E, N, K] -> (packed [E, N, K/2], scales [E, N, K/16], global [E])."""
    E, N, K = W.shape
    packed = torch.empty(E, N, K // 2, dtype=torch.uint8, device=W.device)
    scales = torch.empty(E, N, K // 16, dtype=torch.float8_e4m3fn, device=W.device)
    glob = torch.empty(E, dtype=torch.float32, device=W.device)
    for e in range(E):
        nv.nvfp4_quantize_rows(W[e], packed[e], scales[e], glob[e:e + 1])
    return packed, scales, glob


class MoeTail:
    """Router, experts and lm_head of one model, with the buffers of a step."""

    def __init__(self, tokens=4, hidden=1024, inner=512, experts=32, top_k=4, vocab=32000,
                 alternatives=5, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device=device, generator=g) * 0.03).to(torch.bfloat16)

        self.top_k, self.alternatives = top_k, alternatives
        self.router = weight(experts, hidden)
        self.w13 = quantize_experts(weight(experts, 2 * inner, hidden))
        self.w2 = quantize_experts(weight(experts, hidden, inner))
        self.head = weight(vocab, hidden)
        self.head_q = nv.nvfp4_quantize_rows(self.head)
        self.x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=device)
        self.workspace = torch.empty(nv.w4a16_moe_workspace_bytes(tokens, top_k, hidden, inner),
                                     dtype=torch.uint8, device=device)
        self.graph = None

    def _forward(self):
        ids, weights = nv.moe_route(self.x @ self.router.T, self.top_k)
        y = nv.w4a16_moe(self.x, ids, weights, *self.w13, *self.w2, workspace=self.workspace)
        h = self.x + y
        logits = nv.w4a16_lm_head(h, *self.head_q)
        token = logits.argmax(-1)  # a sampler stands here
        return h, logits, token, nv.token_logprobs(logits, token, self.alternatives)

    def step(self, x: torch.Tensor):
        """(hidden states, logits, tokens, log probabilities) of hidden states x."""
        self.x.copy_(x)
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._forward()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self._forward()
        self.graph.replay()
        return self.out

    def gradient(self, logits, token, scores, advantages, entropy_bonus=0.01):
        """Gradients of mean(advantage * log p + bonus * entropy) with respect
        to the logits and to the hidden states behind the lm_head."""
        _, entropy, lse, *_ = scores
        M = logits.shape[0]
        dlogits = nv.token_logprobs_backward(logits, token, lse, entropy, advantages / M,
                                             torch.full_like(lse, entropy_bonus / M))
        return dlogits, dlogits.to(torch.bfloat16) @ self.head


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args(argv)
    tail = MoeTail(tokens=a.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(a.steps):
        x = torch.randn(tail.x.shape, device="cuda", generator=g).to(torch.bfloat16)
        h, logits, token, scores = tail.step(x)
        lp, entropy, _, rank, top_ids, top_lp = scores
        print(f"step {i}: token {token.tolist()} log p {[round(v, 3) for v in lp.tolist()]} "
              f"entropy {[round(v, 3) for v in entropy.tolist()]}")
    advantages = torch.randn(a.tokens, device="cuda", generator=g)
    dlogits, dh = tail.gradient(logits, token, scores, advantages)
    print(f"gradient: logits {tuple(dlogits.shape)} norm {dlogits.norm():.4f}, "
          f"hidden {tuple(dh.shape)} norm {dh.float().norm():.4f}")
    return {"x": x, "h": h, "logits": logits, "token": token, "scores": scores,
            "advantages": advantages, "dlogits": dlogits, "tail": tail}


if __name__ == "__main__":
    main()
