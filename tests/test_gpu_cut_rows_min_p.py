"""Min-p thresholds of any size against logarithms in 50 digits: a logit l stays where
(l - l_max) / T >= ln min_p, however small min_p is and however finely the logits lie around the border."""

from decimal import Decimal, getcontext

import pytest
import torch

import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
SIZES = [4, 52, 300, 512, 700, 5000, 70000]


def stay(row, T, min_p):
    """How many entries of a row (float64) stay."""
    getcontext().prec = 50
    top = Decimal(float(row.max()))
    least = top + Decimal(T) * Decimal(min_p).ln()
    # (the border in fp64, and the few values within its rounding by themselves)
    near = float(least)
    band = abs(near) * 2.0 ** -50 + 2.0 ** -1000
    n = int((row > near + band).sum())
    return n + sum(Decimal(v) >= least for v in row[(row - near).abs() <= band].tolist())


def check(rows, T, min_p):
    n, V = rows.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, kept, kept2 = (torch.empty(n, 1, **i32) for _ in range(3))
    probs = torch.empty(n, V, device=DEV)
    s = dict(temperature=torch.tensor(T, dtype=torch.float32, device=DEV),
             min_p=torch.tensor(min_p, dtype=torch.float32, device=DEV))
    sd.sd_sample(rows.to(DEV), torch.full((n, 1), 0.5, device=DEV), tokens, kept=kept, **s)
    sd.sd_truncate(rows.to(DEV), probs, kept2, **s)
    assert torch.equal(kept, kept2)
    x = rows.double()
    for i in range(n):
        want = stay(x[i], float(s["temperature"][i]), float(s["min_p"][i]))
        assert int(kept[i]) == want, (i, int(kept[i]), want, T[i], min_p[i])


@pytest.mark.parametrize("V", SIZES)
def test_far_below_the_largest(V):
    g = torch.Generator()
    g.manual_seed(V)
    min_p = [0.3, 1e-3, 2.0 ** -15, 2.0 ** -17, 1e-6, 1e-9, 1e-12, 1e-15, 2.0 ** -61, 2.0 ** -62, 2.0 ** -63, 1e-20,
             1e-30, 1e-37, 1e-42, 2.0 ** -149]
    for spread in (0.5, 5.0, 20.0, 80.0):
        rows = (torch.randn(len(min_p), V, generator=g) * spread).bfloat16()
        T = (0.3 + 1.2 * torch.rand(len(min_p), generator=g)).tolist()
        check(rows, T, min_p)


@pytest.mark.parametrize("V", SIZES)
def test_borders_among_values_that_lie_close(V):
    """The border near zero, where bf16 values lie closely: the largest logit is as far as ln min_p says."""
    g = torch.Generator()
    g.manual_seed(V + 1)
    for top in (4.0, 12.0, 20.0, 32.0, 40.0):
        T, min_p, rows = [], [], []
        for i in range(8):
            T.append(float(torch.tensor(0.5 + 0.25 * i)))
            p = float(torch.exp(torch.tensor(-top / T[-1], dtype=torch.float64)).float())
            min_p.append(p)
            border = float(Decimal(top) + Decimal(T[-1]) * Decimal(p).ln())
            x = border * (1 + torch.randn(V, generator=g, dtype=torch.float64) * 2.0 ** -(i + 2))
            x[0] = top
            rows.append(x)
        check(torch.stack(rows).bfloat16(), T, min_p)
