"""sd_token_logprobs against the definition in 64 bits; ids and ranks exactly."""

import math

import pytest
import torch

import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def call(rows, tokens, n_top, temperature=None, **kw):
    B, J = tokens.shape
    out = dict(logprob=torch.full((B, J), 7.0, device=DEV),
               entropy=torch.full((B, J), 7.0, device=DEV),
               rank=torch.full((B, J), 7, dtype=torch.int32, device=DEV),
               top_ids=torch.full((B, J, n_top), 7, dtype=torch.int32, device=DEV),
               top_logprobs=torch.full((B, J, n_top), 7.0, device=DEV),
               err=torch.zeros(1, dtype=torch.int32, device=DEV))
    sd.sd_token_logprobs(rows, tokens, temperature=temperature, **out, **kw)
    torch.cuda.synchronize()
    return out


def check(rows, tokens, n_top, temperature=None, want_err=0):
    got = call(rows, tokens, n_top, temperature)
    assert int(got["err"]) == want_err
    B, J = tokens.shape
    V = rows.shape[1]
    x = rows.double()
    if rows.dtype == torch.float32:
        lp, p, size = torch.log(x), x, torch.zeros(B * J, 1, device=DEV)
    else:
        T = torch.ones(B, device=DEV) if temperature is None else temperature
        T = torch.where(T > 0, T, torch.ones_like(T)).double().repeat_interleave(J)[:, None]
        lp = torch.log_softmax(x / T, -1)
        p = torch.exp(lp)
        size = 0.0
    ent = -torch.special.xlogy(p, p).sum(-1)
    t = tokens.view(-1).long()
    ok = (t >= 0) & (t < V)
    at = t.clamp(0, V - 1)[:, None]
    # each exponential is off by a few fp32 steps of its argument and of itself, a thread's sum of
    # V / 512 terms by as many half steps, then a tree's
    sums = (V / 512 + 64) * 2.0 ** -24
    tol = lp.abs().clamp(max=1e30) * 2.0 ** -22 + sums
    want = lp.gather(1, at)[:, 0]
    flat = got["logprob"].double().view(-1)
    fin = ok & torch.isfinite(want)
    assert torch.all((flat - want)[fin].abs() <= tol.gather(1, at)[:, 0][fin])
    assert torch.equal(flat[ok & ~fin], want[ok & ~fin])
    live = t >= 0
    tol_h = (1 + ent) * sums + 2.0 ** -21 * (1 + ent)
    assert torch.all((got["entropy"].double().view(-1) - ent)[live].abs() <= tol_h[live])
    xt = x.gather(1, at)
    i = torch.arange(V, device=DEV)[None]
    rank = 1 + ((x > xt) | ((x == xt) & (i < at))).sum(-1)
    assert torch.equal(got["rank"].view(-1)[ok].long(), rank[ok])
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n_top]
    ids = got["top_ids"].view(B * J, n_top).long()
    assert torch.equal(ids[live], order[live])
    a, b = got["top_logprobs"].double().view(B * J, n_top)[live], lp.gather(1, order)[live]
    fin = torch.isfinite(b)
    assert torch.equal(a[~fin], b[~fin])
    assert torch.all((a - b)[fin].abs() <= tol.gather(1, order)[live][fin])
    dead = t == -1
    for k, v in (("logprob", 0.0), ("entropy", 0.0), ("rank", 0)):
        assert torch.all(got[k].view(-1)[dead] == v)
    assert torch.all(ids[dead] == -1)
    assert torch.all(got["top_logprobs"].view(B * J, n_top)[dead] == -math.inf)
    out = t >= V
    assert torch.all(got["logprob"].view(-1)[out] == -math.inf)
    assert torch.all(got["rank"].view(-1)[out] == 0)


@pytest.mark.parametrize("V", [1, 2, 31, 255, 257, 1024, 8191, 32000, 151936, 201088])
@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_sizes(V, kind):
    g = gen(V)
    B, J = 3, 5
    rows = (2 * torch.randn(B * J, V, generator=g, device=DEV)).bfloat16()
    if kind == "probs":
        rows = torch.softmax(rows.float(), -1)
    tokens = torch.randint(0, V, (B, J), generator=g, device=DEV, dtype=torch.int32)
    tokens[1, 3:] = -1
    temp = torch.tensor([0.7, 0.0, 1.9], device=DEV)
    for n_top in (0, 1, 5, 20, 32):
        if n_top <= V:
            check(rows, tokens, n_top, temp)


@pytest.mark.parametrize("rows_n", [1, 40, 400])
def test_cluster_sizes(rows_n):
    """One row is shared by many CTAs, 400 rows have one each."""
    g = gen(rows_n)
    V = 50257
    rows = torch.randn(rows_n, V, generator=g, device=DEV).bfloat16()
    tokens = torch.randint(0, V, (rows_n, 1), generator=g, device=DEV, dtype=torch.int32)
    check(rows, tokens, 9)


@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_ties_and_flat_rows(kind):
    """A constant row, two values, a sorted row and one whose best lie together."""
    V = 20011
    i = torch.arange(V, device=DEV)
    x = torch.stack([torch.zeros(V, device=DEV), (i % 3 == 2).float(), i / 4096.0, -i / 4096.0,
                     ((i >= 5000) & (i < 5040)).float() * 9 - 0.0, -(i % 7 == 3).float() * 0.0])
    rows = x.bfloat16()
    if kind == "probs":
        rows = torch.softmax(x, -1)
    tokens = torch.tensor([[0], [3], [V - 1], [5], [5020], [19999]], dtype=torch.int32, device=DEV)
    check(rows, tokens, 32)


@pytest.mark.parametrize("off", [1, 3])
def test_unaligned_rows(off):
    g = gen(off)
    V, n = 4999, 6
    flat = torch.randn(n * (V + 7) + off, generator=g, device=DEV).bfloat16()
    rows = flat[off:].view(n, V + 7)[:, :V]
    tokens = torch.randint(0, V, (2, 3), generator=g, device=DEV, dtype=torch.int32)
    check(rows, tokens, 4)


def test_infinities():
    """-inf counts as probability 0, in the row and as the token; +inf or NaN make the row NaN."""
    g = gen(8)
    V = 3000
    rows = torch.randn(4, V, generator=g, device=DEV).bfloat16()
    rows[0, ::2] = -math.inf
    rows[1, :] = -math.inf
    rows[1, 77] = 3.0
    tokens = torch.tensor([[2, 77]], dtype=torch.int32, device=DEV)
    check(rows[:2], tokens, 1)
    rows[2, 9] = math.inf
    rows[3, 9] = math.nan
    got = call(rows[2:], torch.tensor([[5, 6]], dtype=torch.int32, device=DEV), 3)
    assert torch.all(torch.isnan(got["logprob"])) and torch.all(torch.isnan(got["entropy"]))


def test_certain_rows():
    """Nearly all of the probability on one entry: the logarithm near 1, an entropy near 0."""
    V = 1000
    p = torch.full((4, V), 1e-9, device=DEV)
    p[torch.arange(4), torch.tensor([0, 5, 500, 999])] = torch.tensor(
        [1 - 1e-6, 1 - 1e-5, 0.999, 0.6], device=DEV)
    check(p, torch.tensor([[0, 5], [500, 999]], dtype=torch.int32, device=DEV), 2)
    l = torch.zeros(2, V, device=DEV)
    l[0, 3], l[1, 7] = 25.0, 90.0
    check(l.bfloat16(), torch.tensor([[3], [7]], dtype=torch.int32, device=DEV), 2)


def test_tokens_out_of_range():
    rows = torch.randn(4, 100, generator=gen(3), device=DEV).bfloat16()
    tokens = torch.tensor([[100, 2 ** 31 - 1, 3, -1]], dtype=torch.int32, device=DEV)
    check(rows, tokens, 3, want_err=sd.SD_ERR_TOKEN_RANGE)
    got = call(rows[:1], torch.tensor([[-5]], dtype=torch.int32, device=DEV), 2)
    assert int(got["err"]) == sd.SD_ERR_TOKEN_RANGE and float(got["logprob"]) == 0.0


def test_optional_outputs_stream_and_graph():
    g = gen(4)
    rows = torch.randn(6, 9000, generator=g, device=DEV).bfloat16()
    tokens = torch.randint(0, 9000, (2, 3), generator=g, device=DEV, dtype=torch.int32)
    want = call(rows, tokens, 3)["logprob"]
    lp = torch.zeros(2, 3, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sd.sd_token_logprobs(rows, tokens, lp, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(lp, want)
    lp.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_token_logprobs(rows, tokens, lp)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lp, want)


@pytest.mark.parametrize("V,rows_n", [(1000, 3), (8192, 5), (32000, 5), (32000, 1300), (201088, 3),
                                      (201088, 1300)])
@pytest.mark.parametrize("n_top", [1, 20, 32])
def test_rows_of_few_entries(V, rows_n, n_top):
    """Rows cut to their largest entries, as sampling leaves them: fewer than n_top positive
    probabilities, and logits of -inf everywhere else."""
    g = gen(V + n_top)
    for kind in ("probs", "logits"):
        x = 2 * torch.randn(rows_n, V, generator=g, device=DEV)
        keep = torch.randint(1, 40, (rows_n, 1), generator=g, device=DEV)
        kth = x.sort(-1, descending=True).values.gather(1, keep)
        x = torch.where(x >= kth, x, torch.full_like(x, -math.inf))
        rows = torch.softmax(x, -1) if kind == "probs" else x.bfloat16()
        check(rows, rows.argmax(-1).to(torch.int32)[:, None], n_top)


@pytest.mark.parametrize("V", [8192, 32000, 201088])
@pytest.mark.parametrize("kind", ["probs", "logits"])
def test_best_entries_in_one_place(V, kind):
    """The largest entries all where one thread reads, in one block, or in order along the row."""
    g = gen(V)
    x = torch.randn(6, V, generator=g, device=DEV)
    i = torch.arange(V, device=DEV)
    x[0] += 20.0 * ((i % 256) < 8)          # a lane of every warp
    x[1] += 20.0 * ((i % 1024) < 4)
    x[2] += 20.0 * ((i >= 1000) & (i < 1700))
    x[3] = 8.0 * i / V
    x[4] = -8.0 * i / V
    x[5] += 20.0 * ((i % 4096) >= 4088)
    rows = torch.softmax(x, -1) if kind == "probs" else x.bfloat16()
    check(rows, torch.full((6, 1), 1001, dtype=torch.int32, device=DEV), 32)
