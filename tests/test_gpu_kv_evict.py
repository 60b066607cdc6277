"""sd_kv_evict against its definition, token by token: everything is equal."""

import pytest
import torch

import kvref
import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(lens, H, D, bs, budget, seed=0, layout="token", fresh=True, ties=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(lens)
    counts = list(lens) + ([min(n, budget) for n in lens] if fresh else [])
    nb, table = kvref.make_table(counts, bs, g, DEV)
    k, v, ks, vs = kvref.make_cache(nb, bs, H, D, g, DEV, layout=layout, spread=2.5)
    w = torch.rand(nb, H, bs, generator=g, device=DEV)
    if ties:
        w = (w * 3).floor()
    to = None
    if fresh:
        to = table[B:, :max(1, -(-budget // bs))].contiguous()
    return dict(k=k, v=v, ks=ks, vs=vs, w=w, table=table[:B].contiguous(), to=to,
                ctx=torch.tensor(lens, dtype=torch.int32, device=DEV))


def run(c, budget, sink=0, recent=0, err=None, **kw):
    B, H = c["ctx"].shape[0], c["k"].shape[2]
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    sd.sd_kv_evict(c["k"], c["v"], c["ks"], c["vs"], c["w"], c["table"], c["ctx"], kept, lens,
                   to_table=c["to"], sink=sink, recent=recent, err=err, **kw)
    return kept, lens


def bits(x):
    return x.view(torch.uint8)


def check(c, budget, sink=0, recent=0, want_err=0):
    val = lambda x: bits(x).view(kvref.E4M3).double().cpu()  # noqa: E731
    want = stepref.evict_ref((val(c["k"]), val(c["v"])), (c["ks"].double().cpu(), c["vs"].double().cpu()),
                             c["w"].double().cpu(), c["table"].tolist(),
                             None if c["to"] is None else c["to"].tolist(), c["ctx"].tolist(), budget,
                             sink, recent)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, lens = run(c, budget, sink, recent, err)
    assert torch.equal(kept.cpu(), want[3]) and torch.equal(lens.cpu(), want[4])
    assert torch.equal(c["ks"].double().cpu(), want[1][0]) and torch.equal(c["vs"].double().cpu(), want[1][1])
    for got, x in ((c["k"], want[0][0]), (c["v"], want[0][1])):
        assert torch.equal(val(got).nan_to_num(500.0), x.nan_to_num(500.0))
    assert torch.equal(c["w"].double().cpu().nan_to_num(-7.0), want[2].nan_to_num(-7.0))
    assert int(err) == want_err


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("H,D,bs", [(2, 64, 16), (1, 128, 8), (3, 80, 32), (2, 16, 64), (1, 96, 128)])
@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([100, 7, 0, 33], 24, 2, 5), ([1, 2, 3], 1, 0, 0), ([1, 2, 3], 1, 1, 0), ([50], 50, 4, 4),
    ([51], 50, 4, 4), ([130, 64], 64, 0, 64), ([129], 128, 128, 0), ([257, 300], 200, 3, 17)])
def test_shapes(H, D, bs, lens, budget, sink, recent, fresh):
    check(make(lens, H, D, bs, budget, seed=budget + D, fresh=fresh), budget, sink, recent)


@pytest.mark.parametrize("fresh", [True, False])
def test_ties_go_to_the_earlier(fresh):
    check(make([300, 200], 2, 32, 16, 90, seed=1, fresh=fresh, ties=True), 90, 4, 10)
    c = make([300, 200], 2, 32, 16, 90, seed=1, fresh=fresh)
    c["w"].zero_()
    c["w"][::2] = -0.0
    check(c, 90, 4, 10)


@pytest.mark.parametrize("fresh", [True, False])
def test_odd_weights(fresh):
    """NaN before all, infinities, negative and subnormal numbers."""
    c = make([200], 2, 32, 16, 40, seed=2, fresh=fresh)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    some = torch.rand(c["w"].shape, generator=g, device=DEV)
    c["w"][some < 0.05] = float("nan")
    c["w"][(some >= 0.05) & (some < 0.1)] = float("inf")
    c["w"][(some >= 0.1) & (some < 0.3)] *= -1
    c["w"][(some >= 0.3) & (some < 0.5)] *= 1e-40
    check(c, 40, 1, 2)


@pytest.mark.parametrize("fresh", [True, False])
def test_scales(fresh):
    """Sources far apart in scale, pages of scale 0 with any bytes, NaN among the values."""
    c = make([150, 90], 2, 64, 16, 60, seed=4, fresh=fresh)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    e = torch.randint(-30, 10, c["ks"].shape, generator=g, device=DEV).double()
    c["ks"].copy_((2.0 ** e).float())
    c["ks"][c["table"][0, 1]] = 0.0
    c["vs"][c["table"][1, 0]] = 0.0
    bits(c["k"])[c["table"][0, 1].long(), 3] = 0x7f
    bits(c["v"])[c["table"][0, 2].long(), 5, 0, 7] = 0xff
    check(c, 60, 2, 8)


@pytest.mark.parametrize("fresh", [True, False])
def test_long(fresh):
    """More tokens than one round of the move and than shared memory holds keys for."""
    H, D, bs, n, budget = 1, 16, 128, 60000, 5000
    c = make([n], H, D, bs, budget, seed=6, fresh=fresh)
    was = {f: c[f].clone() for f in ("k", "v", "ks", "vs", "w")}
    kept, lens = run(c, budget, 4, 100)
    t = torch.arange(n, device=DEV)
    w = was["w"][c["table"][0].long()[t // bs], 0, t % bs]
    mid = torch.sort(w[4:n - 100], descending=True, stable=True).indices[:budget - 104] + 4
    want = torch.cat([t[:4], torch.sort(mid).values, t[n - 100:]])
    assert torch.equal(kept[0, 0].long(), want) and int(lens[0]) == budget
    dest = (c["table"] if c["to"] is None else c["to"])[0].long()
    j = torch.arange(budget, device=DEV)
    src, dst = c["table"][0].long()[want // bs], dest[j // bs]
    assert torch.equal(c["w"][dst, 0, j % bs], was["w"][src, 0, want % bs])
    for x, s in (("k", "ks"), ("v", "vs")):
        big = torch.zeros(c["ks"].shape[0], device=DEV).index_reduce_(0, dst, was[s][src, 0], "amax")
        assert torch.equal(c[s][dst, 0], big[dst])
        y = bits(was[x])[src, want % bs, 0].view(kvref.E4M3).float() * (was[s][src, 0] / big[dst])[:, None]
        assert torch.equal(bits(c[x])[dst, j % bs, 0].view(kvref.E4M3).float(), y.to(kvref.E4M3).float())


@pytest.mark.parametrize("fresh", [True, False])
def test_head_major_cache(fresh):
    check(make([100, 200], 3, 48, 16, 70, seed=7, layout="head", fresh=fresh), 70, 3, 9)


def test_bad_pages():
    """A source without a page counts as weight 0 and zeros, a place without one is not written."""
    c = make([150], 2, 32, 16, 60, seed=8)
    c["table"][0, 2] = -1
    c["table"][0, 4] = c["k"].shape[0]
    c["to"][0, 1] = -1
    check(c, 60, 40, 8, want_err=sd.SD_ERR_KV_RANGE)
    c = make([150, 20], 2, 32, 16, 60, seed=9)
    c["ctx"][0] = 10 ** 6  # beyond the table: its places alone
    c["ctx"][1] = -4
    c["table"] = c["table"][:, :9].contiguous()
    check(c, 60, 2, 8, want_err=sd.SD_ERR_KV_RANGE)


def test_twice_gives_the_same():
    """Into fresh pages the sources stay: a second call finds and writes the same."""
    c = make([100, 60], 2, 64, 16, 40, seed=10)
    first = run(c, 40, 2, 4)
    was = {f: bits(c[f]).clone() for f in ("k", "v", "ks", "vs", "w")}
    second = run(c, 40, 2, 4)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    assert all(torch.equal(bits(c[f]), was[f]) for f in was)


def test_graph_and_stream():
    c = make([100, 60], 2, 64, 16, 40, seed=11)
    kept, lens = run(c, 40, 2, 4)
    was = bits(c["k"]).clone()
    torch.cuda.synchronize()
    out, out_lens = torch.empty_like(kept), torch.empty_like(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.sd_kv_evict(c["k"], c["v"], c["ks"], c["vs"], c["w"], c["table"], c["ctx"], out, out_lens,
                       to_table=c["to"], sink=2, recent=4)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, kept) and torch.equal(out_lens, lens) and torch.equal(bits(c["k"]), was)
    s = torch.cuda.Stream()
    again, again_lens = run(c, 40, 2, 4, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, kept) and torch.equal(again_lens, lens)


def test_attention_goes_on_over_what_stayed():
    """sd_kv_attend over the cut cache sees the tokens that stayed, each head its own."""
    H, G, D, bs, budget = 2, 2, 64, 16, 48
    c = make([200, 30], H, D, bs, budget, seed=12)
    vals = {}
    for r, n in enumerate([200, 30]):
        vals[r] = [kvref.held(c[x], c[s], c["table"][r], n) for x, s in (("k", "ks"), ("v", "vs"))]
    kept, lens = run(c, budget, 2, 6)
    q = torch.randn(2, H * G, D, device=DEV).bfloat16()
    out = torch.empty_like(q)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    sd.sd_kv_attend(q, c["k"], c["v"], c["ks"], c["vs"], c["to"], lens, cu, out, causal=False)
    for r in range(2):
        n = int(lens[r])
        k, v = (torch.stack([x[kept[r, h, :n].long(), h] for h in range(H)], 1) for x in vals[r])
        # (values moved to a larger scale may have lost what became subnormal: 2^-10 of the scale each)
        page = c["to"][r, :-(-n // bs)].long()
        kk = kvref.held(c["k"], c["ks"], c["to"][r], n)
        vv = kvref.held(c["v"], c["vs"], c["to"][r], n)
        for x, y, s in ((k, kk, c["ks"]), (v, vv, c["vs"])):
            lim = s[page].repeat_interleave(bs, 0)[:n].double() * 2.0 ** -10
            assert torch.all((x - y).abs() <= lim[..., None])
        o, _, tol, _ = kvref.attend_ref(q[r:r + 1].double(), kk, vv, D ** -0.5, False)
        assert torch.all((out[r:r + 1].double() - o).abs() <= tol)


@pytest.mark.parametrize("lens,H,bs", [([5000, 4097], 32, 16), ([9000, 100, 3000], 16, 32), ([430000], 1, 128),
                                       ([60000] * 2, 80, 128)])
def test_choice_of_long_requests(lens, H, bs):
    """One CTA a request and head, clusters of several, keys that fit shared memory and keys that do not:
    the tokens that stay are those of a sort."""
    budget, sink, recent, D = 777, 3, 50, 16
    c = make(lens, H, D, bs, budget, seed=13, ties=True)
    c["w"] += torch.rand(c["w"].shape, device=DEV).mul(64).floor() / 64
    was = c["w"].clone()
    kept, out = run(c, budget, sink, recent)
    for r, n in enumerate(lens):
        assert int(out[r]) == min(n, budget)
        t = torch.arange(n, device=DEV)
        w = was[c["table"][r].long()[t // bs], :, t % bs]  # [n, H]
        if n <= budget:
            assert torch.all(kept[r, :, :n] == t) and torch.all(kept[r, :, n:] == -1)
            continue
        mid = torch.sort(w[sink:n - recent], dim=0, descending=True, stable=True).indices
        mid = torch.sort(mid[:budget - sink - recent] + sink, dim=0).values
        want = torch.cat([t[:sink, None].expand(-1, H), mid, t[n - recent:, None].expand(-1, H)]).T
        assert torch.equal(kept[r].long(), want)
        # and their weights stand where they went
        j = torch.arange(budget, device=DEV)
        for h in (0, H - 1):
            assert torch.equal(c["w"][c["to"][r].long()[j // bs], h, j % bs], w[want[h], h])
