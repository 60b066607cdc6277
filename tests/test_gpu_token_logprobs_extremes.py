"""sd_token_logprobs at temperatures and logits far from the ordinary: the definition in 64 bits."""

import math

import pytest
import torch

import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOWEST = torch.finfo(torch.bfloat16).min


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def check(rows, tokens, T, n_top=3):
    """rows [n, V] bf16, tokens [n], one request a row at temperature T (a number or [n])."""
    n, V = rows.shape
    temp = torch.full((n,), T, device=DEV) if isinstance(T, float) else T
    got = dict(logprob=torch.full((n, 1), 7.0, device=DEV), entropy=torch.full((n, 1), 7.0, device=DEV),
               rank=torch.zeros(n, 1, dtype=torch.int32, device=DEV),
               top_ids=torch.zeros(n, 1, n_top, dtype=torch.int32, device=DEV),
               top_logprobs=torch.full((n, 1, n_top), 7.0, device=DEV),
               err=torch.zeros(1, dtype=torch.int32, device=DEV))
    sd.sd_token_logprobs(rows, tokens.to(torch.int32)[:, None].contiguous(), temperature=temp, **got)
    assert int(got["err"]) == 0
    x = rows.double()
    d = (x - x.amax(-1, keepdim=True)) / temp.double()[:, None]  # 0 at the largest, -inf stays
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    lp = d - torch.log(z)
    p = e / z
    ent = torch.log(z[:, 0]) - torch.where(e > 0, p * d, torch.zeros_like(d)).sum(-1)
    # a difference of logits, its quotient by T and the sum with ln z are rounded to fp32 each, an
    # exponential is off by a few steps of its argument and of itself, sums as half steps of their terms
    sums = (V / 512 + 64) * 2.0 ** -24
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n_top]
    assert torch.equal(got["top_ids"][:, 0].long(), order)
    for have, at in ((got["logprob"], tokens.long()[:, None]), (got["top_logprobs"][:, 0], order)):
        want = lp.gather(1, at)
        fits = want >= -torch.finfo(torch.float32).max
        assert torch.all(have.double()[~fits] == -math.inf)
        off = (have.double() - want)[fits].abs()
        assert torch.all(off <= (want.abs() * 2.0 ** -22 + sums)[fits]), float(off.max())
    off = (got["entropy"][:, 0].double() - ent).abs()
    assert torch.all(off <= (1 + ent) * (sums + 2.0 ** -21)), (off, ent)
    i = torch.arange(V, device=DEV)[None]
    xt = x.gather(1, tokens.long()[:, None])
    assert torch.equal(got["rank"][:, 0].long(),
                       1 + ((x > xt) | ((x == xt) & (i < tokens.long()[:, None]))).sum(-1))


SIZES = [(3, 1000), (5, 201088), (400, 5003), (40, 131072)]


@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("T", [1e-30, 1e-20, 1e-10, 1e-9, 4e-9, 1e-5, 0.01, 1.0, 100.0, 1e8, 1e20, 1e30])
def test_any_temperature(n, V, T):
    """V is no multiple of what a warp loads at once: the entries past the row's end are -inf. The
    largest logit several times, at equal distances and alone."""
    g = gen(V)
    rows = (3 * torch.randn(n, V, generator=g, device=DEV)).bfloat16()
    rows[0, ::97] = rows[0].max()
    rows[1, ::3] = -math.inf
    rows[2, 7] = 50.0
    tokens = torch.randint(0, V, (n,), generator=g, device=DEV)
    tokens[:3] = rows[:3].argmax(-1)
    check(rows, tokens, T)
    check(-rows[:1] * 1e-3, tokens[:1], T)


@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("T", [1e-9, 0.7, 1.0, 1e9])
def test_rows_with_the_lowest_number(n, V, T):
    """finfo.min as a mask: beside ordinary logits, beside -inf, alone, and next to other such numbers."""
    g = gen(V + 1)
    rows = torch.randn(n, V, generator=g, device=DEV).bfloat16()
    rows[0, 1::2] = LOWEST
    rows[1] = LOWEST
    rows[2] = -math.inf
    rows[2, 5::7] = LOWEST
    if n > 4:
        rows[3] = LOWEST
        rows[3, V // 2] = -3.3e38
        rows[4] = -math.inf
        rows[4, ::5] = LOWEST
        rows[4, V - 1] = -2.9e38
    tokens = torch.randint(0, V, (n,), generator=g, device=DEV)
    tokens[0], tokens[2] = 1, 5
    check(rows, tokens, T)


@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("size", [1e4, 1e10, 1e25, 1e37])
def test_large_logits(n, V, size):
    """All far from 0, on either side: only differences count."""
    g = gen(V + 2)
    x = torch.randn(n, V, generator=g, device=DEV)
    for rows in (x * size, size - x.abs() * size / 64, -size - x.abs() * size / 64):
        rows = rows.bfloat16()
        tokens = rows.argmax(-1)
        for T in (1e-3, 1.0, min(size / 8, 1e30)):
            check(rows, tokens, T)


def test_one_nan_stays_a_nan():
    """Among lowest numbers, -inf and ordinary logits, before and after them in the row."""
    V = 3000
    for fill in (LOWEST, -math.inf, 1.0):
        for at in (0, 1400, V - 1):
            rows = torch.full((2, V), fill, device=DEV).bfloat16()
            rows[0, at] = math.nan
            rows[0, 700] = 2.0
            rows[1, at] = math.nan
            lp, h = (torch.zeros(2, 1, device=DEV) for _ in range(2))
            for T in (1e-10, 1.0):
                sd.sd_token_logprobs(rows, torch.full((2, 1), 700, dtype=torch.int32, device=DEV), lp,
                                     entropy=h, temperature=torch.full((2,), T, device=DEV))
                assert torch.isnan(lp).all() and torch.isnan(h).all()
