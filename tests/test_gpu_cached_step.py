"""The example's step: the cache calls, verification and the answer's log probabilities together."""

import math
import os
import sys

import pytest
import torch

import kvref
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_step():
    import cached_step
    import verify_draft_prep_gb300 as sd

    B, K = 5, 3
    step = cached_step.Step(B=B, K=K, V=700, heads=2, groups=4, dim=64, H=64, ctx=(1, 300), seed=3)
    rows = step.randn(B * K, step.V)
    drafts = torch.empty(B, K, **step.i32)
    sd.sd_draft_sample(rows, drafts, seed=1, err=step.err)
    before = [t.clone() for t in step.draft_cache.all()]
    r = step.run(drafts, rows)
    torch.cuda.synchronize()
    assert int(step.err) == 0
    # every verify slot attends to what the cache holds up to its position
    cache = step.target_cache
    for b in range(B):
        T = int(step.pos0[b]) + K + 1
        k = kvref.held(cache.k, cache.k_scale, step.table[b], T)
        v = kvref.held(cache.v, cache.v_scale, step.table[b], T)
        rows_b = slice(b * (K + 1), (b + 1) * (K + 1))
        o, _, tol, _ = kvref.attend_ref(r["q"][rows_b].double(), k, v, 64 ** -0.5, True)
        assert torch.all((r["attended"][rows_b].double() - o).abs() <= tol)
        # and the last K+1 of those tokens are the ones just written
        new = r["k"][rows_b].double()
        assert float((k[-(K + 1):] - new).norm() / new.norm()) < 0.05
    # the answer's log probabilities are its rows' log softmax
    lp = torch.log_softmax(r["logits"].double(), -1).view(B, K + 1, -1)
    t = r["out_tokens"].long()
    live = t >= 0
    assert torch.equal(live.sum(1), r["accepted"].long() + 1)
    want = lp.gather(2, t.clamp(min=0)[..., None])[..., 0]
    assert torch.all((r["logprob"].double() - want)[live].abs() < 2.0 ** -16)
    assert torch.all(r["logprob"][~live] == 0) and torch.all(r["top_ids"][~live] == -1)
    assert torch.all(r["top_logprobs"][~live] == -math.inf)
    # the drafter's cache changed in the pages of its slots alone
    pages = torch.unique(r["draft_slots"][r["draft_slots"] >= 0] // cached_step.BLOCK).long()
    same = torch.ones(step.draft_cache.k.shape[0], dtype=torch.bool, device="cuda")
    same[pages] = False
    for a, b in zip(before, step.draft_cache.all()):
        assert torch.equal(a.view(torch.uint8)[same], b.view(torch.uint8)[same])
        assert not torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.isfinite(r["drafted"].float()).all()
