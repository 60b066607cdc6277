"""The sums that sd_truncate and sd_sample decide by, against whole numbers: draws and top-p cuts whose goal
lies as near to a border between two entries as an error of 2^-40 of the sum allows.

The numbers u and top_p are fp32, so a border is near one only by chance; rows of thousands of entries
have some. A host search in exact arithmetic finds them."""

import bisect
import math
from decimal import Decimal, getcontext

import pytest
import torch

import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
ONE = 1 << 160  # units of the host's sums
NEAR = 2.0 ** -34  # borders within this of an fp32 number (of the sum), but not within 2^-40


def weights(row, logits, T):
    """The order of a row's entries and their weights in that order, as whole numbers of 1 / ONE (of the
    largest, for logits, to 2^-100 of it). Every value occurs; the row is on the CPU."""
    x = row.double()
    x, order = torch.sort(x, descending=True, stable=True)
    values, counts = torch.unique_consecutive(x, return_counts=True)
    if logits:
        getcontext().prec = 60
        top, t = Decimal(float(values[0])), Decimal(T)
        each = [int(((Decimal(v) - top) / t).exp() * ONE) for v in values.tolist()]
    else:
        each = [int(Decimal(v) * ONE) for v in values.tolist()]
    out = []
    for w, c in zip(each, counts.tolist()):
        out += [w] * c
    return order.tolist(), out


def floats_beside(a, b):
    """The fp32 numbers at or below and above a / b (0 < a < b), as Python floats."""
    x = float(torch.tensor(a / b, dtype=torch.float32))
    up = float(torch.nextafter(torch.tensor(x), torch.tensor(2.0)))
    down = float(torch.nextafter(torch.tensor(x), torch.tensor(-1.0)))
    return [v for v in (down, x, up) if 0 < v < 1]


def near_borders(w, most):
    """(gap, number, how many sums lie at or below number * total) for numbers that lie near a border,
    the nearest first."""
    sums, run = [], 0
    for x in w:
        run += x
        sums.append(run)
    # most borders are far from every fp32 number: look at them in fp64 first (2^-52 of the sum)
    r = torch.tensor([s / run for s in sums], dtype=torch.float64)
    gap = (r - r.float().double()).abs()
    numbers = set()
    for j in torch.nonzero((gap < 2 * NEAR) & (r < 1) & (r > 0))[:, 0].tolist():
        numbers.update(floats_beside(sums[j], run))
    found = []
    for v in numbers:
        n, d = v.as_integer_ratio()
        below = bisect.bisect_right(sums, n * run // d)
        beside = [abs(s * d - n * run) for s in sums[max(0, below - 1):below + 1]]
        gap = min(beside) / (d * run)
        if 2.0 ** -40 <= gap <= NEAR:
            found.append((gap, v, below))
    return sorted(found)[:most]


def check(row, logits, T, least):
    """Every near border of the row, as a draw's number and as a top-p."""
    order, w = weights(row.cpu(), logits, T)
    near = near_borders(w, 128)
    assert len(near) >= least, len(near)
    if not near:
        return
    B, V = len(near), row.shape[0]
    rows = row.to(DEV).expand(B, V).contiguous()
    i32 = dict(dtype=torch.int32, device=DEV)
    u = torch.tensor([v for _, v, _ in near], dtype=torch.float32, device=DEV)
    temperature = torch.full((B,), T, device=DEV)
    tokens, kept = torch.empty(B, 1, **i32), torch.empty(B, 1, **i32)
    sd.sd_sample(rows, u.view(B, 1), tokens, temperature=temperature)
    wrong = [(i, g) for i, ((g, _, n), t) in enumerate(zip(near, tokens[:, 0].tolist())) if t != order[n]]
    assert not wrong, [(i, math.log2(g)) for i, g in wrong]
    probs = torch.empty(B, V, device=DEV)
    sd.sd_truncate(rows, probs, kept, temperature=temperature, top_p=u)
    # those before which less than top_p of the sum lies: the first, and one for every sum below
    wrong = [(i, g) for i, ((g, _, n), k) in enumerate(zip(near, kept[:, 0].tolist())) if k != n + 1]
    assert not wrong, [(i, math.log2(g)) for i, g in wrong]
    assert torch.equal((probs > 0).sum(1).int(), kept[:, 0])


def every_value(low, high, top):
    """A row of `top` and one entry of every bf16 value of magnitude 2^low to 2^high."""
    bits = torch.arange((127 + low) << 7, (127 + high) << 7)
    bits = torch.cat([bits, bits + 0x8000]).to(torch.int32) << 16
    x = torch.cat([torch.tensor([top]), bits.view(torch.float32)])
    g = torch.Generator()
    g.manual_seed(low + 100)
    return x[torch.randperm(x.numel(), generator=g)].bfloat16()


@pytest.mark.parametrize("low,high,T", [(-15, -2, 0.1), (-15, 2, 0.3), (-40, -2, 0.07), (-126, 1, 0.4)])
def test_a_bin_for_every_value(low, high, T):
    """Thousands of bins of one entry each, at ten temperatures: from 2^-15 on the quick kernel has them,
    below the one with a bin for every value."""
    row = every_value(low, high, 1.0 if high < 0 else 2.0 ** high)
    for i in range(10):
        check(row, True, float(torch.tensor(T * (1 + i / 16))), 1)


@pytest.mark.parametrize("seed,spread,T", [(0, 4.0, 0.5), (8, 4.0, 0.5), (10, 4.0, 0.5), (1, 4.0, 1.0),
                                           (2, 2.0, 0.7)])
def test_vocabularies(seed, spread, T):
    g = torch.Generator()
    g.manual_seed(seed)
    check((torch.randn(201088, generator=g) * spread).bfloat16(), True, float(torch.tensor(T)), 1)


@pytest.mark.parametrize("seed,V,spread,times", [(4, 201088, 2.0, 1.0), (5, 30000, 4.0, 1.0),
                                                 (6, 201088, 4.0, 2.0 ** -9), (7, 1500, 1.0, 1.0)])
def test_probabilities(seed, V, spread, times):
    """Rows that add up to one, and (by `times`) one that needs the kernel with a bin for every value."""
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.softmax(torch.randn(V, generator=g, dtype=torch.float64) * spread, 0) * times
    check(p.float(), False, 1.0, 0 if V < 10000 else 1)


@pytest.mark.parametrize("seed", [8, 9])
def test_rows_that_a_warp_sorts(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    for i in range(30):
        x = torch.randn(500, generator=g) * 3
        check(x.bfloat16(), True, float(torch.tensor(0.4 + i / 20)), 0)
        check(torch.softmax(x, 0), False, 1.0, 0)
