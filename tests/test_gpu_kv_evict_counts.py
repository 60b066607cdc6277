"""sd_kv_evict at the largest budgets and lengths that it accepts: places are counted up to 2^31 - 1024 by
clusters whose step is up to 4096."""

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
MOST = 2 ** 31 - 1024
GUARD = 1 << 20  # ints before and behind the places


def places():
    """[1, 1, MOST] ints within a larger array, all of it -9."""
    whole = torch.full((GUARD + MOST + GUARD,), -9, dtype=torch.int32, device=DEV)
    return whole, whole[GUARD:GUARD + MOST].view(1, 1, MOST)


def check_places(whole, n):
    """The places are 0..n-1 and -1 behind, and nothing around them is touched."""
    assert torch.all(whole[:GUARD] == -9) and torch.all(whole[GUARD + MOST:] == -9)
    step = 1 << 28
    for a in range(0, MOST, step):
        b = min(MOST, a + step)
        got = whole[GUARD + a:GUARD + b]
        m = max(0, min(b, n) - a)
        assert torch.equal(got[:m], torch.arange(a, a + m, dtype=torch.int32, device=DEV))
        assert torch.all(got[m:] == -1)


def cache(nb, bs):
    k, v = (torch.zeros(nb, bs, 1, 16, dtype=torch.uint8, device=DEV).view(kvref.E4M3) for _ in range(2))
    ks, vs = (torch.ones(nb, 1, device=DEV) for _ in range(2))
    return k, v, ks, vs, torch.zeros(nb, 1, bs, device=DEV)


@pytest.mark.parametrize("blocks", [64, 200, 400, 1024])  # clusters of 1, 2, 4 and 8
def test_largest_budget(blocks):
    whole, kept = places()
    table = torch.full((1, blocks), -1, dtype=torch.int32, device=DEV)
    table[0, :3] = torch.tensor([2, 0, 1], dtype=torch.int32)
    ctx, lens = (torch.full((1,), 40, dtype=torch.int32, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sd.sd_kv_evict(*cache(3, 16), table, ctx, kept, lens, err=err)
    assert int(lens) == 40 and int(err) == 0
    check_places(whole, 40)


def test_largest_length():
    """A table of 2^31 places without a page: every place stays, and nothing is moved."""
    whole, kept = places()
    table = torch.full((1, 1 << 24), -1, dtype=torch.int32, device=DEV)
    to = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
    ctx = torch.full((1,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = cache(1, 128)
    sd.sd_kv_evict(*c, table, ctx, kept, lens, to_table=to)
    assert int(lens) == MOST
    check_places(whole, MOST)
    assert int(c[0].view(torch.uint8).sum()) == 0 and int(c[4].sum()) == 0
