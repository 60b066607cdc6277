"""The kernel with a bin for every value, which does the rows that the quick one marks, with 4 and 8 CTAs a
row: its counters are two 16-bit counts a word, of at most 65528 entries each."""

import math

import pytest
import torch

import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
VOCABULARIES = [262112, 262113, sd.SD_CUT_MAX_V]


def call(rows, u, **s):
    n, V = rows.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, kept, kept2 = (torch.empty(n, 1, **i32) for _ in range(3))
    probs, prob = torch.empty(n, V, device=DEV), torch.empty(n, 1, device=DEV)
    err = torch.zeros(1, **i32)
    sd.sd_sample(rows, u, tokens, prob=prob, kept=kept, err=err, **s)
    sd.sd_truncate(rows, probs, kept2, err=err, **s)
    assert torch.equal(kept, kept2) and int(err) == 0
    return tokens[:, 0].tolist(), kept[:, 0].tolist(), probs, prob[:, 0]


# Subnormal bf16 logits are too small for e^l to be anything but 1 to 2^-125: entries of one value or of two
# weigh the same, but larger ones come first.
@pytest.mark.parametrize("V", VOCABULARIES)
@pytest.mark.parametrize("bits", [0x0003, 0x8005])
def test_one_value(V, bits):
    """A part of a row all in one counter: places are indices."""
    rows = torch.full((8, V), bits - (bits & 0x8000) * 2, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    top_k = [0, 1, V, V - 1, 65537, 100000, 0, 0]
    top_p = [1, 1, 1, 1, 1, 1, 0.5, 0.25]
    u = [0.0, 0.9, 1.0 - 2.0 ** -24, 0.75, 0.5, 0.999, 0.5, 0.125]
    f = lambda x: torch.tensor(x, dtype=torch.float32, device=DEV)  # noqa: E731
    tokens, kept, probs, prob = call(rows, f(u).view(8, 1), top_p=f(top_p),
                                     top_k=torch.tensor(top_k, dtype=torch.int32, device=DEV))
    for i in range(8):
        n = min(V, top_k[i]) if top_k[i] else V
        n = math.ceil(top_p[i] * n)  # (halves and quarters: exact)
        w = float(torch.tensor(u[i])) * n
        assert kept[i] == n and tokens[i] == min(n - 1, math.floor(w)), i
        assert torch.all(probs[i, :n] > 0) and torch.all(probs[i, n:] == 0)
        assert abs(float(prob[i]) * n - 1) <= 2.0 ** -22
        assert torch.all((probs[i, :n].double() * n - 1).abs() <= 2.0 ** -22)


@pytest.mark.parametrize("V", VOCABULARIES)
def test_two_values_of_one_word(V):
    """Neighbouring values, whose counts share a word, in every mixture: a count that ran over would show in
    the other's."""
    low, high = 0x0004, 0x0005  # bins stand in pairs of an odd value and the even one below it
    g = torch.Generator()
    g.manual_seed(V)
    rows, u, top_k = [], [], []
    for share in (0.5, 0.0001, 0.9999, 1.0 - 1.0 / V, 1.0 / V, 0.25):
        first = torch.rand(V, generator=g) < share
        first[17], first[V - 5] = True, False
        rows.append(torch.where(first, high, low).to(torch.int16))
        u.append(float(torch.rand(1, generator=g)))
        top_k.append(0)
        rows.append(rows[-1])
        u.append(float(torch.rand(1, generator=g)))
        top_k.append(int(first.sum()) + int(torch.randint(-20, 20, (1,), generator=g)))
    bits = torch.stack(rows)
    top_k = [min(V, max(1, k)) if k else 0 for k in top_k]
    number = torch.tensor(u, dtype=torch.float32)
    tokens, kept, probs, _ = call(bits.to(DEV).view(torch.bfloat16), number.to(DEV).view(-1, 1),
                                  top_k=torch.tensor(top_k, dtype=torch.int32, device=DEV))
    for i, row in enumerate(bits):
        order = torch.sort(row, descending=True, stable=True).indices
        n = top_k[i] or V
        assert kept[i] == n, i
        assert tokens[i] == int(order[min(n - 1, math.floor(float(number[i]) * n))]), i
        at = torch.nonzero(probs[i].cpu() > 0)[:, 0]
        assert torch.equal(at, torch.sort(order[:n]).values), i
