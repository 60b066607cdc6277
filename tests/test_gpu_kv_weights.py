"""sd_kv_weights against its formula in 64 bits."""

import math

import pytest
import torch

import kvref
import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(lens, n_q, Hq, H, D, bs, seed=0, spread=0.5, layout="token"):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    nb, table = kvref.make_table(lens, bs, g, DEV)
    k, _, ks, _ = kvref.make_cache(nb, bs, H, D, g, DEV, layout=layout, spread=spread)
    n = sum(n_q)
    q = torch.randn(n, Hq, D, generator=g, device=DEV).bfloat16()
    cu = kvref.prefix(n_q, DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    before = torch.rand(nb, H, bs, generator=g, device=DEV)
    return dict(q=q, k=k, ks=ks, table=table, cu=cu, ctx=ctx, before=before, lens=lens, n_q=n_q)


def lse_of(c, sm, causal=True):
    """The log sums of all heads, in fp32, and the keys of every request in 64 bits."""
    n, Hq, D = c["q"].shape
    H = c["k"].shape[2]
    lse = torch.full((n, Hq), -math.inf, device=DEV)
    at = 0
    for r, (T, m) in enumerate(zip(c["lens"], c["n_q"])):
        if T and m:
            k = kvref.held(c["k"], c["ks"], c["table"][r], T)
            _, l, _, _ = kvref.attend_ref(c["q"][at:at + m].double(), k, k, sm, causal)
            lse[at:at + m] = l.float()
        at += m
    return lse


def check(c, out, lse, sm, causal=True, live=None, decay=1.0, before=True, untouched=-3.0):
    at, bs = 0, c["k"].shape[1]
    want_mask = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    for r, (T, m) in enumerate(zip(c["lens"], c["n_q"])):
        if T:
            k = kvref.held(c["k"], c["ks"], c["table"][r], T)
            t = torch.arange(T, device=DEV)
            page = c["table"][r].long()[t // bs]
            old = c["before"][page, :, t % bs].double() if before else None
            w, tol = stepref.weights_ref(c["q"][at:at + m].double(), lse[at:at + m].double(), k, sm,
                                         causal, m if live is None else live[r], decay, old)
            got = out[page, :, t % bs].double()
            assert torch.all((got - w).abs() <= tol), (r, float(((got - w).abs() - tol).max()))
            want_mask[page, :, t % bs] = True
        at += m
    assert torch.all(out[~want_mask] == untouched)


def call(c, out, lse, err=None, **kw):
    sd.sd_kv_weights(c["q"], lse, c["k"], c["ks"], c["table"], c["ctx"], c["cu"], out, err=err, **kw)


@pytest.mark.parametrize("Hq,H,D,bs", [(8, 2, 64, 16), (4, 4, 128, 8), (7, 1, 32, 32), (16, 2, 80, 64),
                                       (6, 2, 96, 128), (64, 8, 64, 16), (1, 1, 16, 16)])
@pytest.mark.parametrize("lens,n_q", [
    ([37], [5]), ([1], [1]), ([0, 3, 130], [0, 3, 2]), ([129, 500, 64, 257], [6, 1, 17, 9])])
def test_shapes(Hq, H, D, bs, lens, n_q):
    c = make(lens, n_q, Hq, H, D, bs, seed=D + bs)
    sm = D ** -0.5
    lse = lse_of(c, sm)
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, out, lse, err, before=c["before"], decay=0.75)
    check(c, out, lse, sm, decay=0.75)
    again = torch.full_like(out, -3.0)
    call(c, again, lse, before=c["before"], decay=0.75, max_q=1)
    assert torch.equal(out, again)
    # without numbers of before; every row's weights add up to 1
    out.fill_(-3.0)
    call(c, out, lse, err, max_q=max(n_q))
    check(c, out, lse, sm, before=False)
    assert int(err) == 0
    total = out[out != -3.0].double().sum()
    assert abs(float(total) - sum(n_q) * Hq) <= 1e-4 * max(1, sum(n_q) * Hq)


def test_in_place_and_not_causal():
    c = make([70, 200], [3, 4], 8, 4, 64, 16, seed=5)
    lse = lse_of(c, 0.2, causal=False)
    out = c["before"].clone()
    call(c, out, lse, before=out, decay=0.5, sm_scale=0.2, causal=False)
    was = torch.full_like(out, -3.0)
    call(c, was, lse, before=c["before"], decay=0.5, sm_scale=0.2, causal=False)
    check(c, was, lse, 0.2, causal=False, decay=0.5)
    assert torch.equal(out[was != -3.0], was[was != -3.0])
    assert torch.equal(out[was == -3.0], c["before"][was == -3.0])


@pytest.mark.parametrize("live", [[0, 0], [6, 1], [1, 4]])
def test_live(live):
    c = make([300, 41], [6, 4], 16, 2, 64, 16, seed=6)
    lse = lse_of(c, 0.125)
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, out, lse, err, before=c["before"], live=torch.tensor(live, dtype=torch.int32, device=DEV))
    check(c, out, lse, 0.125, live=live)
    assert int(err) == 0
    # counts beyond the tokens are clamped, and said so
    more = torch.full_like(out, -3.0)
    call(c, more, lse, err, before=c["before"], live=torch.tensor([9, -2], dtype=torch.int32, device=DEV))
    check(c, more, lse, 0.125, live=[6, 0])
    assert int(err) == sd.SD_ERR_KV_RANGE


@pytest.mark.parametrize("n_q,G,D", [(300, 4, 64), (200, 8, 128), (513, 1, 128)])
def test_prompts(n_q, G, D):
    c = make([n_q, n_q + 77], [n_q, n_q], 2 * G, 2, D, 16, seed=n_q, layout="head")
    lse = lse_of(c, D ** -0.5)
    out = torch.full_like(c["before"], -3.0)
    call(c, out, lse, before=c["before"], max_q=n_q)
    check(c, out, lse, D ** -0.5)


def test_what_rows_do_not_see_has_no_effect():
    """NaN in K and in rows that do not count, in the tokens behind a row, and behind the context."""
    c = make([100], [4], 4, 2, 64, 16, seed=9)
    lse = lse_of(c, 0.125)
    out = torch.full_like(c["before"], -3.0)
    call(c, out, lse, live=torch.tensor([2], dtype=torch.int32, device=DEV))
    raw = c["k"].view(torch.uint8)
    t = torch.arange(98, 112, device=DEV)  # tokens 98 and 99 are seen by rows 2 and 3 alone
    raw[c["table"][0].long()[t // 16], t % 16] = 0x7f
    c["q"][2:] = float("nan")
    lse[2:] = float("nan")
    dirty = torch.full_like(out, -3.0)
    call(c, dirty, lse, live=torch.tensor([2], dtype=torch.int32, device=DEV))
    assert torch.equal(out, dirty)
    assert torch.all(dirty[c["table"][0].long()[t[:2] // 16], :, t[:2] % 16] == 0)


def test_pages():
    """A page of scale 0 holds zeros whatever its bytes; a table entry out of range leaves its tokens
    out, with the bit."""
    c = make([90], [2], 4, 2, 64, 16, seed=10)
    page = c["table"][0].long()
    c["ks"][page[1]] = 0.0
    lse = torch.zeros(2, 4, device=DEV)
    raw = c["k"].view(torch.uint8)
    raw[page[1]] = 0x7f
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, out, lse, err)
    assert torch.all(out[page[1]] == 4.0)  # two rows of two heads, each e^(0 - 0)
    assert int(err) == 0
    c["table"][0, 2], c["table"][0, 3] = -1, c["k"].shape[0]
    part = torch.full_like(out, -3.0)
    call(c, part, lse, err)
    assert int(err) == sd.SD_ERR_KV_RANGE
    assert torch.all(part[page[2:4]] == -3.0)
    keep = torch.ones(out.shape[0], dtype=torch.bool, device=DEV)
    keep[page[2:4]] = False
    assert torch.equal(out[keep], part[keep])


def test_lengths_out_of_range():
    c = make([90, 30], [2, 2], 4, 2, 64, 16, seed=11)
    lse = lse_of(c, 0.125)
    want, out = torch.full_like(c["before"], -3.0), torch.full_like(c["before"], -3.0)
    call(c, want, lse)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    c["ctx"][1] = -5
    call(c, out, lse, err)
    assert int(err) == sd.SD_ERR_KV_RANGE
    first = c["table"][0].long()
    assert torch.equal(out[first], want[first])
    second = c["table"][1, :2].long()
    assert torch.all(out[second] == -3.0)


def test_no_queries_keep_and_decay():
    """A request without query tokens in this call keeps its numbers times the decay."""
    c = make([50, 40], [0, 2], 4, 2, 64, 16, seed=12)
    lse = lse_of(c, 0.125)
    out = torch.full_like(c["before"], -3.0)
    call(c, out, lse, before=c["before"], decay=0.25)
    t = torch.arange(50, device=DEV)
    page = c["table"][0].long()[t // 16]
    assert torch.equal(out[page, :, t % 16], c["before"][page, :, t % 16] * 0.25)
    check(c, out, lse, 0.125, decay=0.25)


def test_peaked_rows():
    """One token that takes nearly all of the weight, and lse of any size."""
    c = make([400], [3], 4, 2, 64, 16, seed=13, spread=2.0)
    c["q"] *= 6
    lse = lse_of(c, 0.125)
    out = torch.full_like(c["before"], -3.0)
    call(c, out, lse)
    check(c, out, lse, 0.125, before=False)


def test_graphs_and_streams():
    c = make([130, 260], [6, 6], 16, 2, 64, 16, seed=14)
    lse = lse_of(c, 0.125)
    want, out = torch.full_like(c["before"], -3.0), torch.full_like(c["before"], -3.0)
    call(c, want, lse, before=c["before"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, out, lse, before=c["before"])
    for _ in range(2):
        out.fill_(-3.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        outs.append(torch.full_like(want, -3.0))
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        call(c, o, lse, before=c["before"], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_after_attend():
    """The lse that sd_kv_attend writes: every row's weights add up to 1."""
    B, n_q, Hq, H, D, bs = 3, 6, 32, 4, 64, 16
    lens = [400, 61, 1000]
    c = make(lens, [n_q] * B, Hq, H, D, bs, seed=15)
    out, lse = torch.empty_like(c["q"]), torch.empty(B * n_q, Hq, device=DEV)
    sd.sd_kv_attend(c["q"], c["k"], c["k"], c["ks"], c["ks"], c["table"], c["ctx"], c["cu"], out,
                    lse=lse, max_q=n_q)
    w = torch.zeros_like(c["before"])
    call(c, w, lse, max_q=n_q)
    for r, T in enumerate(lens):
        t = torch.arange(T, device=DEV)
        got = w[c["table"][r].long()[t // bs], :, t % bs].double().sum(0)
        assert torch.all((got - n_q * Hq // H).abs() < 1e-4 * n_q * Hq / H)


@pytest.mark.parametrize("max_q", [1, 40, 600])
def test_any_number_expected(max_q):
    """max_q only chooses the kernel: many chunks of rows in the one for few, few in the one for many."""
    c = make([600, 333], [500, 3], 8, 2, 64, 16, seed=16)
    lse = lse_of(c, 0.125)
    out = torch.full_like(c["before"], -3.0)
    call(c, out, lse, before=c["before"], max_q=max_q)
    check(c, out, lse, 0.125)


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 128), (96, 8)])
def test_long_contexts(D, bs):
    """Many units a CTA, among them those of neighbours that have none or one."""
    c = make([20000, 0, 1, 7001], [4, 0, 1, 6], 16, 8, D, bs, seed=17)
    lse = lse_of(c, D ** -0.5)
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, out, lse, err, before=c["before"], max_q=6)
    check(c, out, lse, D ** -0.5)
    assert int(err) == 0


def test_many_requests():
    """More requests than threads find their places."""
    g = torch.Generator()
    g.manual_seed(18)
    lens = torch.randint(0, 60, (1500,), generator=g).tolist()
    n_q = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 4, (1500,), generator=g))]
    c = make(lens, n_q, 4, 1, 32, 8, seed=18)
    lse = torch.zeros(sum(n_q), 4, device=DEV)
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, out, lse, err, before=c["before"], max_q=3, sm_scale=2.0 ** -6)
    check(c, out, lse, 2.0 ** -6)
    assert int(err) == 0


@pytest.mark.parametrize("D,G", [(64, 8), (128, 4), (80, 7)])
@pytest.mark.parametrize("causal", [True, False])
def test_the_kernel_for_prompts(D, G, causal):
    """Prompts in earnest and, by what is expected, single tokens and requests without any."""
    c = make([700, 0, 1200, 31, 130], [700, 0, 650, 1, 0], 2 * G, 2, D, 16, seed=D)
    lse = lse_of(c, D ** -0.5, causal=causal)
    out, err = torch.full_like(c["before"], -3.0), torch.zeros(1, dtype=torch.int32, device=DEV)
    live = [700, 0, 301, 1, 0]
    call(c, out, lse, err, before=c["before"], max_q=1 << 20, causal=causal, decay=0.5,
         live=torch.tensor(live, dtype=torch.int32, device=DEV))
    check(c, out, lse, D ** -0.5, causal=causal, decay=0.5, live=live)
    assert int(err) == 0
