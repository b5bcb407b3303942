"""examples/moe_rollout_step.py end to end against plain 64-bit forms."""
import importlib.util
import os

import pytest
import torch

from tests._operators import logprobs_grad_reference, logprobs_reference, moe_reference
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 4, 48])
def test_rollout_step(tokens):
    import __graft_entry__

    __graft_entry__.build()
    path = os.path.join(ROOT, "examples", "moe_rollout_step.py")
    spec = importlib.util.spec_from_file_location("moe_rollout_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(["--tokens", str(tokens), "--steps", "2"])
    tail = r["tail"]
    import nvfp4_weight_only_rows_gb300 as nv

    # the layer the captured step ran, on the routing of the same logits
    ids, w = nv.moe_route(r["x"] @ tail.router.T, tail.top_k)
    cpu = lambda ts: tuple(t.cpu() for t in ts)  # noqa: E731
    ref, tol = moe_reference(r["x"].cpu(), ids.cpu(), w.cpu(), cpu(tail.w13), cpu(tail.w2))
    # y and h = x + y are each rounded to bf16: 2^-9 of themselves at most
    want = r["x"].double().cpu() + ref
    bound = tol + 2.0 ** -9 * (ref.abs() + tol) + 2.0 ** -8 * (want.abs() + ref.abs())
    assert bool(((r["h"].double().cpu() - want).abs() <= bound).all())
    logits, token = r["logits"].cpu(), r["token"].cpu()
    assert torch.equal(token, logits.argmax(-1))
    lp, ent, lse, ranks, top_ids, top_lp = (t.cpu() for t in r["scores"])
    wlp, went, wlse, wranks, wids, wtop = logprobs_reference(logits, token, tail.alternatives, 1.0)
    assert torch.equal(ranks, wranks) and torch.equal(top_ids, wids)
    for got, ref in ((lp, wlp), (ent, went), (lse, wlse), (top_lp, wtop)):
        assert bool(((got.double() - ref).abs() <= 1e-4 * (1 + ref.abs())).all())
    M = tokens
    g, gt = logprobs_grad_reference(logits, token, 1.0, lse, ent, r["advantages"].cpu() / M,
                                    torch.full((M,), 0.01 / M))
    assert bool(((r["dlogits"].double().cpu() - g).abs() <= gt).all())
