"""The probabilities that sd_truncate and sd_sample write, as near to 64 bits as each is made.

One made from probabilities, and a drawn token's: its weight and the sum are off by 2^-40 together, and one
rounding to fp32 is 2^-24: 2^-24 (1 + 2^-12). One made from logits: the distance d from the largest logit is
rounded by 2^-24 d, which is 2^-24 d / T of the exponential, with d / T = -ln of the share of the largest;
the exponential is off by two places (CUDA's bound for exp2f, 4 x 2^-24), and its factor, their product
and the quotient are rounded: 7 x 2^-24, and 2^-35 for the factor's square."""

import pytest
import torch

import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
ONCE = 2.0 ** -24 * (1 + 2.0 ** -12)
LOGITS = 7 * 2.0 ** -24 + 2.0 ** -34


def check(rows, s, u):
    n, V = rows.shape
    logits = rows.dtype == torch.bfloat16
    dev = {k: v.to(DEV) for k, v in s.items()}
    i32 = dict(dtype=torch.int32, device=DEV)
    probs, prob = torch.empty(n, V, device=DEV), torch.empty(n, 1, device=DEV)
    kept, tokens = torch.empty(n, 1, **i32), torch.empty(n, 1, **i32)
    sd.sd_truncate(rows, probs, kept, **dev)
    sd.sd_sample(rows, u, tokens, prob=prob, **dev)
    x = rows.double().cpu()
    get = lambda f, i, none: float(s[f][i]) if f in s else none  # noqa: E731
    for i in range(n):
        order, p, m = stepref.cut_ref(x[i], logits, get("temperature", i, 1.0), int(get("top_k", i, 0)),
                                      get("top_p", i, 1.0), get("min_p", i, 0.0))
        assert int(kept[i]) == m
        want = torch.zeros_like(p)
        want[order] = p
        off = (probs[i].double().cpu() - want).abs()
        nats = -torch.log((want / want.max()).clamp(min=1e-300))
        # (numbers below 2^-126 have fewer places)
        bad = off > want * (LOGITS + 2.0 ** -24 * nats if logits else ONCE) + 2.0 ** -148 * (want < 2.0 ** -125)
        assert not torch.any(bad), (i, float((off / want.clamp(min=1e-300)).max() * 2.0 ** 24))
        mine = float(want[int(tokens[i])])
        assert abs(float(prob[i]) - mine) <= mine * ONCE, i


def rows_of(n, V, kind, spread, seed, times=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(n, V, generator=g, dtype=torch.float64) * spread
    x = torch.softmax(x, -1).float() * times if kind == "probs" else (x * times).bfloat16()
    return x.to(DEV), torch.rand(n, 1, generator=g).to(DEV)


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V", [1, 100, 512, 1100, 5000, 201088])
def test_all_kept(kind, V):
    for seed, spread in enumerate((0.5, 2.0, 6.0)):
        rows, u = rows_of(6, V, kind, spread, seed)
        T = torch.tensor([0.3, 0.7, 1.0, 1.7, 5.0, 60.0]) if kind == "logits" else torch.ones(6)
        check(rows, dict(temperature=T), u)


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V", [100, 1100, 5000, 201088])
def test_cut(kind, V):
    rows, u = rows_of(12, V, kind, 2.5, 5)
    check(rows, dict(top_k=torch.tensor([0, 1, 2, 40, 90, 0] * 2).int(), min_p=torch.tensor([0.0] * 6 + [0.02] * 6),
                     top_p=torch.tensor([0.9, 1.0, 1.0, 0.8, 1.0, 0.4] * 2)), u)


@pytest.mark.parametrize("V", [600, 20000])
@pytest.mark.parametrize("kind,times", [("logits", 2.0 ** -14), ("logits", 2.0 ** 16), ("probs", 2.0 ** -9),
                                        ("probs", 2.0 ** -100)])
def test_rows_with_a_bin_for_every_value(V, kind, times):
    """Small and large logits, rows that do not add up to a half."""
    rows, u = rows_of(5, V, kind, 2.0, 6, times)
    T = torch.tensor([0.5, 1.0, 2.0, 4.0, 8.0]) * (times if kind == "logits" else 1.0)
    check(rows, dict(temperature=T, top_p=torch.tensor([1.0, 0.9, 1.0, 0.5, 0.999])), u)
