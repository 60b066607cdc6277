"""The example's drafter: every position that its rows attend to was written."""

import os
import sys

import pytest
import torch

import kvref
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_drafter_attends_to_what_was_written():
    import cached_step
    import verify_draft_prep_gb300 as sd

    B, K = 6, 4
    step = cached_step.Step(B=B, K=K, V=500, heads=2, groups=4, dim=64, H=64, ctx=(1, 200), seed=11)
    # the context's positions, 0 to pos0 of each request, hold values and scales
    for b in range(B):
        n = int(step.pos0[b]) + 1
        page, off = step.table[b, (n - 1) // cached_step.BLOCK].long(), (n - 1) % cached_step.BLOCK
        for x, s in ((step.draft_cache.k, step.draft_cache.k_scale),
                     (step.draft_cache.v, step.draft_cache.v_scale)):
            assert torch.all(s[page] > 0)
            assert torch.all(x[page, off].float().abs().amax(-1) > 0), (b, n - 1)
    rows = step.randn(B * K, step.V)
    drafts = torch.empty(B, K, **step.i32)
    sd.sd_draft_sample(rows, drafts, seed=2, err=step.err)
    r = step.run(drafts, rows)
    torch.cuda.synchronize()
    assert int(step.err) == 0
    W, cache = step.W, step.draft_cache
    slots = r["draft_slots"].view(B, W)
    for b in range(B):
        live = int((slots[b] >= 0).sum())  # the first a_r + K of its row
        assert live == int(r["accepted"][b]) + K and bool((slots[b, :live] >= 0).all())
        first = int(step.pos0[b]) + 1
        k = kvref.held(cache.k, cache.k_scale, step.table[b], first + live)
        v = kvref.held(cache.v, cache.v_scale, step.table[b], first + live)
        mine = slice(b * W, b * W + live)
        o, _, tol, _ = kvref.attend_ref(r["draft_q"][mine].double(), k, v, 64 ** -0.5, True)
        assert torch.all((r["drafted"][mine].double() - o).abs() <= tol)
