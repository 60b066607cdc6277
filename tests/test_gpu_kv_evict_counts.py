"""sd_kv_evict where it counts far: the largest budgets and lengths that it accepts (places up to 2^31 - 1024,
by clusters whose step is up to 4096), and moves within a request's own pages that take several rounds."""

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd
from test_gpu_kv_evict import bits, make, run

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


@pytest.mark.parametrize("H,D,bs,n,budget", [(2, 128, 16, 9000, 3500), (1, 128, 128, 7000, 3000), (3, 96, 32, 6000, 4111),
                                             (2, 64, 16, 9000, 5000)])
def test_rounds_of_a_move_in_place(H, D, bs, n, budget):
    """More places than a cluster takes at a time (1024, or 2048 of heads of up to 64): what stays is where
    a move into fresh pages puts it, and where a sort of the weights says."""
    sink, recent = 5, 300
    c = make([n], H, D, bs, budget, seed=n, fresh=True)
    was = {f: c[f].clone() for f in ("k", "v", "ks", "vs", "w")}
    kept, lens = run(c, budget, sink, recent)
    mine = {**{f: was[f].clone() for f in was}, "table": c["table"], "to": None, "ctx": c["ctx"]}
    kept2, lens2 = run(mine, budget, sink, recent)
    assert torch.equal(kept, kept2) and int(lens) == int(lens2) == budget
    t, j = torch.arange(n, device=DEV), torch.arange(budget, device=DEV)
    page = c["table"][0].long()
    fresh, own = c["to"][0].long()[j // bs], page[j // bs]
    for h in range(H):
        w = was["w"][page[t // bs], h, t % bs]
        mid = torch.sort(w[sink:n - recent], descending=True, stable=True).indices[:budget - sink - recent]
        want = torch.cat([t[:sink], torch.sort(mid + sink).values, t[n - recent:]])
        assert torch.equal(kept[0, h].long(), want)
        src = page[want // bs]
        assert torch.equal(mine["w"][own, h, j % bs], was["w"][src, h, want % bs])
        for x, s in (("k", "ks"), ("v", "vs")):
            assert torch.equal(mine[s][own, h], c[s][fresh, h])
            got, same = (bits(y[x])[p, j % bs, h] for y, p in ((mine, own), (c, fresh)))
            assert torch.equal(got, same)
            # powers of two: a value is what it was but for what became subnormal
            step = mine[s][own, h].double() * 2.0 ** -10
            a = got.view(kvref.E4M3).double() * mine[s][own, h].double()[:, None]
            b = bits(was[x])[src, want % bs, h].view(kvref.E4M3).double() * was[s][src, h].double()[:, None]
            assert torch.all((a - b).abs() <= step[:, None])
    # pages behind the kept ones, and pages of no request, stay as they are
    rest = torch.ones(mine["k"].shape[0], dtype=torch.bool, device=DEV)
    rest[own] = False
    for f in was:
        assert torch.equal(bits(mine[f])[rest], bits(was[f])[rest])
