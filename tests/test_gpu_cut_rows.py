"""sd_truncate and sd_sample against a sort in 64 bits: what is kept and what is drawn are equal."""

import math

import pytest
import torch

import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"


def settings(B, seed, **fixed):
    g = torch.Generator()
    g.manual_seed(seed)
    s = dict(temperature=0.4 + torch.rand(B, generator=g), top_k=torch.randint(1, 60, (B,), generator=g).int(),
             top_p=0.3 + 0.69 * torch.rand(B, generator=g), min_p=0.2 * torch.rand(B, generator=g))
    r = torch.arange(B)
    s["temperature"][r % 5 == 3] = 0
    s["top_k"][r % 3 != 0] = 0
    s["top_p"][r % 4 == 1] = 1
    s["min_p"][r % 2 == 0] = 0
    s.update(fixed)
    return s


def run(rows, B, J, s, u=None, err=None, pad=0, stream=None):
    dev = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    V = rows.shape[1]
    i32 = dict(dtype=torch.int32, device=DEV)
    wide = torch.full((B * J, V + pad), -5.0, device=DEV)
    kept, kept2, tokens = (torch.full((B, J), -9, **i32) for _ in range(3))
    prob = torch.full((B, J), -9.0, device=DEV)
    sd.sd_truncate(rows, wide[:, :V], kept, err=err, stream=stream, **dev)
    u = torch.rand(B, J, device=DEV) if u is None else u
    sd.sd_sample(rows, u, tokens, prob=prob, kept=kept2, err=err, stream=stream, **dev)
    torch.cuda.synchronize()
    assert torch.equal(kept, kept2)
    assert not pad or torch.all(wide[:, V:] == -5.0)
    return wide[:, :V], kept, tokens, prob, u


def check(rows, B, J, s, u=None, want_err=0, pad=0):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    probs, kept, tokens, prob, u = run(rows, B, J, s, u, err, pad)
    logits = rows.dtype == torch.bfloat16
    x, probs, prob = rows.double().cpu(), probs.double().cpu(), prob.double().cpu()
    get = lambda f, r, none: none if s[f] is None else float(s[f][r])  # noqa: E731
    for i in range(B * J):
        r, j = divmod(i, J)
        order, p, n = stepref.cut_ref(x[i], logits, get("temperature", r, 1.0), int(get("top_k", r, 0)),
                                      get("top_p", r, 1.0), get("min_p", r, 0.0))
        assert int(kept[r, j]) == n, (i, int(kept[r, j]), n)
        want = torch.zeros_like(p)
        want[order] = p
        # an exponential's argument in fp32, its value to 2^-21, the quotient
        tol = want * (2.0 ** -20 + 2.0 ** -22 * -torch.log(want.clamp(min=1e-300) / want.max().clamp(min=1e-300)))
        assert torch.all((probs[i] - want).abs() <= tol + 2.0 ** -149), i
        assert torch.equal(probs[i] > 0, want > 2.0 ** -126) or n == 0 or want[want > 0].min() < 2.0 ** -120
        t, pt = stepref.draw_ref(order, p, n, float(u[r, j]))
        assert int(tokens[r, j]) == t, (i, int(tokens[r, j]), t)
        assert abs(float(prob[r, j]) - pt) <= 2.0 ** -22 * pt
    assert int(err) == want_err


def rows_of(n, V, kind, seed, spread=2.0, ld=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, V, generator=g, device=DEV) * spread
    x = torch.softmax(x, -1) if kind == "probs" else x.bfloat16()
    if ld:
        wide = torch.zeros(n, ld, dtype=x.dtype, device=DEV)
        wide[:, :V] = x
        x = wide[:, :V]
    return x


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 100, 1000, 1024, 5003])
def test_sizes(kind, V):
    check(rows_of(24, V, kind, V), 12, 2, settings(12, V))


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V", [255, 256, 257, 511, 512, 513, 4097])
def test_sizes_where_kernels_change(kind, V):
    """Rows that a warp sorts, and those that a CTA or several count."""
    check(rows_of(24, V, kind, V, spread=4.0), 12, 2, settings(12, V + 1))
    check(rows_of(3, V, kind, V, ld=V + 5), 3, 1, settings(3, V + 2), pad=1)


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V", [300, 3000])
def test_many_rows(kind, V):
    """More rows than fit on the GPU at a time: tokens, counts and sums of all of them."""
    n = 3000
    rows, s = rows_of(n, V, kind, 19), settings(n, 19)
    probs, kept, tokens, prob, u = run(rows, n, 1, s)
    for i in range(0, n, 37):
        get = lambda f: float(s[f][i])  # noqa: E731
        order, p, m = stepref.cut_ref(rows[i].double().cpu(), kind == "logits", get("temperature"),
                                      int(s["top_k"][i]), get("top_p"), get("min_p"))
        assert int(kept[i]) == m and int(tokens[i]) == stepref.draw_ref(order, p, m, float(u[i]))[0]
    assert torch.equal((probs > 0).sum(1).int(), kept[:, 0])
    assert torch.all((probs.double().sum(1) - 1).abs() < 2.0 ** -18)
    assert torch.all((probs.gather(1, tokens.long()) - prob).abs() <= prob * 2.0 ** -18)


@pytest.mark.parametrize("V", [1500, 201088])
def test_grammar_masks(V):
    """Nearly every entry -inf or the type's lowest number: fewer numbers than top_k, draws and counts
    among what is left, with and without another cut."""
    low = torch.finfo(torch.bfloat16).min
    x = rows_of(8, V, "logits", 20)
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    hide = torch.rand(8, V, generator=g, device=DEV) < 0.99
    hide[:, 7] = False
    x[:4] = x[:4].masked_fill(hide[:4], -math.inf)
    x[4:] = x[4:].masked_fill(hide[4:], low)
    s = dict(temperature=torch.full((8,), 0.9), top_k=torch.tensor([0, 50, 0, 5000] * 2).int(),
             top_p=torch.tensor([1.0, 1.0, 0.8, 1.0] * 2), min_p=None)
    check(x, 8, 1, s)


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("V,ld", [(8193, 8193), (20000, 20001), (32768, 32776), (50001, 50004),
                                  (201088, 201088), (262113, 262120)])
def test_large(kind, V, ld):
    check(rows_of(10, V, kind, V, ld=ld), 10, 1, settings(10, V), pad=3)


@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_largest(kind):
    check(rows_of(2, sd.SD_CUT_MAX_V, kind, 5, spread=0.3), 2, 1,
          settings(2, 5, top_p=torch.tensor([0.97, 1.0]), top_k=torch.tensor([0, 300000]).int()))


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("spread", [0.01, 0.3, 8.0, 60.0])
def test_flat_and_peaked(kind, spread):
    check(rows_of(30, 4000, kind, 7, spread=spread), 30, 1, settings(30, 7))


@pytest.mark.parametrize("kind", ["probs", "logits"])
@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
def test_each_alone(kind, name):
    s = dict(temperature=None, top_k=None, top_p=None, min_p=None)
    s[name] = {"temperature": torch.tensor([0.0, 0.1, 1.0, 7.0, -1.0, math.nan]),
               "top_k": torch.tensor([-1, 0, 1, 2, 299, 10 ** 6]).int(),
               "top_p": torch.tensor([-0.5, 0.0, 1e-6, 0.5, 0.999999, 1.5]),
               "min_p": torch.tensor([-1.0, 0.0, 1e-30, 0.3, 1.0, 2.0])}[name]
    check(rows_of(12, 300, kind, 8), 6, 2, s)
    check(rows_of(12, 300, kind, 8), 6, 2, dict.fromkeys(s))


@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_ties(kind):
    """Equal entries go by index: a few values, one value, and a cut or a draw within a run of ties."""
    V = 3000
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    x = torch.randint(0, 4, (16, V), generator=g, device=DEV).float()
    x[0] = 2.0
    x[1] = -3.0
    rows = x.bfloat16() if kind == "logits" else (x + 1 + 4 * (x < 0)) / 4096
    s = settings(16, 9, top_k=torch.tensor([1, 2999, 3000, 700, 0, 5, 0, 0] * 2).int(),
                 top_p=torch.tensor([1.0, 1.0, 0.5, 0.25] * 4), min_p=torch.zeros(16))
    s["temperature"][:2] = 1.0
    check(rows, 16, 1, s)


@pytest.mark.parametrize("u", [0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan])
def test_given_numbers_at_the_edges(u):
    """Four equal entries: the running sums are quarters exactly. Numbers outside [0, 1) are taken
    within it."""
    rows = torch.full((1, 4), 0.25, device=DEV)
    for x in (rows, torch.zeros(1, 4, device=DEV).bfloat16()):
        got = run(x, 1, 1, dict(temperature=None, top_k=None, top_p=None, min_p=None),
                  u=torch.full((1, 1), u, device=DEV))
        v = 0.0 if u != u else u
        assert int(got[2]) == min(3, max(0, int(v * 4)))
        assert float(got[3]) == 0.25
    cut = run(rows, 1, 1, dict(temperature=None, top_k=None, top_p=torch.tensor([0.5]), min_p=None))
    assert int(cut[1]) == 2  # less than half lies before the first two alone


def test_masks():
    """-inf, the type's lowest number, +inf and NaN among logits; rows of one value; rows of nothing."""
    V, ninf, low = 700, -math.inf, torch.finfo(torch.bfloat16).min
    x = rows_of(12, V, "logits", 10)
    x[0, ::2] = ninf
    x[1, 1:] = ninf
    x[2, 5:] = low
    x[3] = low
    x[4, 3] = x[4, 9] = math.inf
    x[5, ::3] = math.nan
    x[6, :] = 0.0
    x[6, 100:300] = -0.0
    x[7, :-1] = ninf
    x[8] = x[8] * 1e-38  # subnormal
    x[9] = x[9] * 1e37
    for seed in range(3):
        s = settings(12, seed)
        if seed == 2:
            s = dict(temperature=None, top_k=None, top_p=None, min_p=None)
        check(x, 12, 1, s)
    x[10] = ninf
    x[11] = math.nan
    check(x, 12, 1, settings(12, 4), want_err=sd.SD_ERR_ZERO_ROW)


def test_odd_probabilities():
    """Zeros, numbers below 2^-126, rows that do not add up to 1, numbers that are none."""
    V = 700
    x = rows_of(10, V, "probs", 11)
    x[0, ::2] = 0.0
    x[1, 1:] = 0.0
    x[2] *= 1e-38
    x[3] *= 1e-42
    x[4] *= 900.0  # some above 1
    x[5, ::5] = math.nan
    x[6, ::7] = -0.5
    x[7, 3] = math.inf
    x[8, :300] = 2.0 ** -149
    s = settings(10, 11)
    s["min_p"][:] = 0
    check(x, 10, 1, s)
    x[9] = 0.0
    check(x, 10, 1, s, want_err=sd.SD_ERR_ZERO_ROW)


@pytest.mark.parametrize("T", [2.0 ** -120, 1e-20, 1e-3, 1e4, 1e30, 3e38])
def test_temperatures(T):
    s = dict(temperature=torch.full((6,), T), top_k=torch.tensor([0, 5] * 3).int(),
             top_p=torch.tensor([1.0, 1.0, 0.7, 0.7, 0.2, 1.0]), min_p=None)
    check(rows_of(6, 500, "logits", 12), 6, 1, s)


def test_same_upper_halves():
    """Probabilities that share their upper 16 bits: a row within one bin, and runs of equal ones."""
    V = 6000
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    low = torch.randint(0, 65536, (8, V), generator=g, device=DEV).int()
    low[4:] &= 0x303
    low[6:, :] = low[6:, :1]
    x = (low + (0x3900 << 16)).view(torch.float32)
    check(x, 8, 1, settings(8, 13, top_k=torch.tensor([0, 1, 3000, 0] * 2).int()))


def test_draws_follow_the_cut_distribution():
    """Frequencies of 200000 draws: each within 5 standard deviations of its probability."""
    V, n = 50, 200000
    row = rows_of(1, V, "logits", 14, spread=1.0)
    rows = row.expand(n, V).contiguous()
    f = lambda v: torch.full((n,), v, device=DEV)  # noqa: E731
    tokens = torch.empty(n, 1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(15)
    u = torch.rand(n, 1, generator=g, device=DEV)
    sd.sd_sample(rows, u, tokens, top_p=f(0.9), min_p=f(0.02))
    order, p, k = stepref.cut_ref(row[0].double().cpu(), True, 1.0, 0, float(torch.tensor(0.9)),
                                  float(torch.tensor(0.02)))
    want = torch.zeros(V, dtype=torch.float64)
    want[order] = p
    got = torch.bincount(tokens.view(-1).long().cpu(), minlength=V).double() / n
    assert torch.all(got[want == 0] == 0)
    assert torch.all((got - want).abs() <= 5 * torch.sqrt(want / n))


def test_graphs_and_streams():
    rows = rows_of(12, 9000, "logits", 16)
    s = settings(6, 16)
    want = run(rows, 6, 2, s)
    dev = {k: v.to(DEV) for k, v in s.items()}
    probs, kept, tokens = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(want[2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.sd_truncate(rows, probs, kept, **dev)
        sd.sd_sample(rows, want[4], tokens, **dev)
    for _ in range(2):
        probs.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(probs, want[0]) and torch.equal(kept, want[1]) and torch.equal(tokens, want[2])
    got = run(rows, 6, 2, s, u=want[4], stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_cut_rows_verify(kind):
    """Target and draft rows cut by the same settings go through verification: what is accepted or
    drawn again is always among the target's kept entries, and drafts outside are rejected."""
    B, K, V = 40, 3, 500
    s = settings(B, 17, temperature=torch.full((B,), 0.8))
    dev = {k: v.to(DEV) for k, v in s.items()}
    i32 = dict(dtype=torch.int32, device=DEV)
    target, draft = rows_of(B * (K + 1), V, kind, 18), rows_of(B * K, V, kind, 18)
    p, q = torch.empty(B * (K + 1), V, device=DEV), torch.empty(B * K, V, device=DEV)
    sd.sd_truncate(target, p, torch.empty(B, K + 1, **i32), **dev)
    sd.sd_truncate(draft, q, torch.empty(B, K, **i32), **dev)
    drafts, out, acc = torch.empty(B, K, **i32), torch.empty(B, K + 1, **i32), torch.empty(B, **i32)
    err = torch.zeros(1, **i32)
    sd.sd_sample(draft, torch.rand(B, K, device=DEV), drafts, err=err, **dev)
    assert torch.all(q.view(B, K, V).gather(2, drafts.long()[..., None]) > 0)
    sd.sd_verify(p, q, drafts, out, acc, seed=3, err=err)
    live = out >= 0
    at = p.view(B, K + 1, V).gather(2, out.clamp(min=0).long()[..., None])[..., 0]
    assert torch.all(at[live] > 0) and int(err) == 0
