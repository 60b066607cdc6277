"""NaN in the cache reaches the query tokens that see it and nothing else: every other row has the same
bits as without it, in every kernel and where several CTAs share a request."""

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"

# units of 32, 64, 128 and 256 rows: query tokens and query heads of a KV head
FORMS = [(5, 6), (9, 7), (17, 7), (60, 7)]


class Call:
    def __init__(self, n, T, G, D, bs, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.n, self.T, self.G, self.bs = n, T, G, bs
        nb, self.table = kvref.make_table([T], bs, g, DEV)
        self.cache = list(kvref.make_cache(nb, bs, 2, D, g, DEV))
        self.q = torch.randn(n, 2 * G, D, generator=g, device=DEV).bfloat16()
        self.cu = kvref.prefix([n], DEV)
        self.lens = torch.full((1,), T, dtype=torch.int32, device=DEV)

    def run(self, causal=True):
        out = torch.zeros_like(self.q)
        lse = torch.zeros(self.q.shape[:2], device=DEV)
        sd.sd_kv_attend(self.q, *self.cache, self.table, self.lens, self.cu, out, lse=lse,
                        max_q=self.n, causal=causal)
        return out, lse

    def at(self, t):
        return int(self.table[0, t // self.bs]), t % self.bs


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D,bs", [(64, 16), (80, 8), (128, 16), (128, 128), (112, 32)])
@pytest.mark.parametrize("T", [70, 1100, 9000])
def test_reaches_only_the_rows_that_see_it(n, G, D, bs, T):
    c = Call(n, T, G, D, bs, seed=D + T)
    want, want_lse = c.run()
    # seen by all, by the last two rows, by the last alone; the first token, a tile's last and first
    for t in sorted({0, min(127, T - n), (T - n) // 2, T - n, T - 2, T - 1}):
        page, off = c.at(t)
        first = max(0, t - (T - n))
        for side in (0, 1):
            d = (5 * t + 3) % D
            raw = c.cache[side].view(torch.uint8)
            keep = int(raw[page, off, 1, d])
            raw[page, off, 1, d] = 0xFF if t % 2 else 0x7F
            out, lse = c.run()
            raw[page, off, 1, d] = keep
            hit = torch.zeros_like(out, dtype=torch.bool)
            if side == 1:
                hit[first:, G:, d] = True
            else:
                hit[first:, G:] = True
            assert torch.equal(torch.isnan(out), hit), (t, side)
            assert torch.equal(out[~hit], want[~hit]), (t, side)
            rows = hit.all(-1)
            assert torch.equal(torch.isnan(lse), rows), (t, side)
            assert torch.equal(lse[~rows], want_lse[~rows]), (t, side)


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D,bs", [(64, 16), (80, 64), (128, 16), (96, 128)])
@pytest.mark.parametrize("T", [70, 1100, 9001])
@pytest.mark.parametrize("causal", [True, False])
def test_beyond_the_context(n, G, D, bs, T, causal):
    """Bytes behind the last token and in pages of others, scales of others."""
    c = Call(n, T, G, D, bs, seed=D + T + 1)
    want, want_lse = c.run(causal)
    used = c.table[0, :-(-T // bs)].long()
    other = torch.ones(c.cache[0].shape[0], dtype=torch.bool, device=DEV)
    other[used] = False
    for i in range(2):
        raw = c.cache[i].view(torch.uint8)
        raw[other] = 0x7F
        if T % bs:
            raw[used[-1], T % bs:] = 0xFF
        c.cache[i + 2][other] = float("nan")
    out, lse = c.run(causal)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_do_not_depend_on_one_another(n, G, D):
    """A row's bits are the same whatever the queries of the others are."""
    c = Call(n, 3000, G, D, 16, seed=D)
    want, want_lse = c.run()
    mine = torch.zeros(n, 2 * G, dtype=torch.bool, device=DEV)
    mine[n // 2, 1] = mine[0, G] = mine[n - 1, 2 * G - 1] = True
    for size in (0.0, 0.1, 20.0, float("nan")):
        keep = c.q.clone()
        c.q[~mine] = keep[~mine] * size
        out, lse = c.run()
        c.q.copy_(keep)
        assert torch.equal(out[mine], want[mine]) and torch.equal(lse[mine], want_lse[mine])
