"""sd_kv_attend against the formula in 64 bits, request by request."""

import math

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Case:
    """Requests with n_q[r] new tokens and ctx[r] cached ones (the new ones included)."""

    def __init__(self, n_q, ctx, Hq, Hkv, D, bs, seed=0, layout="token", size=1.0):
        g = gen(seed)
        self.n_q, self.ctx, self.Hq, self.D = n_q, ctx, Hq, D
        nb, self.table = kvref.make_table(ctx, bs, g, DEV)
        self.cache = list(kvref.make_cache(nb, bs, Hkv, D, g, DEV, layout))
        n = sum(n_q)
        self.q = (size * torch.randn(n, Hq, D, generator=g, device=DEV)).bfloat16()
        self.cu = kvref.prefix(n_q, DEV)
        self.lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)

    def run(self, causal=True, max_q=None, out=None, lse=None, **kw):
        n = self.q.shape[0]
        self.out = torch.full((n, self.Hq, self.D), 7.0, device=DEV).bfloat16() if out is None else out
        self.lse = torch.full((n, self.Hq), 7.0, device=DEV) if lse is None else lse
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sd.sd_kv_attend(self.q, *self.cache, self.table, self.lens, self.cu, self.out,
                        lse=self.lse, max_q=max(self.n_q + [1]) if max_q is None else max_q,
                        causal=causal, err=err, **kw)
        torch.cuda.synchronize()
        return int(err)

    def check(self, causal=True, hide=None, only=None):
        at = 0
        for r, n in enumerate(self.n_q):
            if only is not None and r not in only:
                at += n
                continue
            T = self.ctx[r]
            k = kvref.held(self.cache[0], self.cache[2], self.table[r], T)
            v = kvref.held(self.cache[1], self.cache[3], self.table[r], T)
            o, l, tol, tol_l = kvref.attend_ref(self.q[at:at + n].double(), k, v, self.D ** -0.5,
                                                causal, None if hide is None else hide[r])
            got, lse = self.out[at:at + n].double(), self.lse[at:at + n].double()
            at += n
            none = torch.isinf(l)
            assert torch.all(got[none] == 0), r
            assert torch.equal(lse[none], l[none]), r
            assert torch.all((got - o).abs() <= tol), (r, float(((got - o).abs() / (tol + 1e-30)).max()))
            assert torch.all((lse - l)[~none].abs() <= tol_l[~none]), r


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (7, 1, 80), (64, 8, 64),
                                      (32, 8, 128), (3, 3, 16), (40, 2, 96), (128, 1, 64), (6, 2, 32),
                                      (4, 1, 48), (16, 2, 112)])
@pytest.mark.parametrize("n_q,ctx", [([5], [42]), ([1], [1]), ([1, 6, 3], [700, 6, 129]),
                                     ([17, 9], [128, 1300])])
def test_head_layouts(Hq, Hkv, D, n_q, ctx):
    c = Case(n_q, ctx, Hq, Hkv, D, 16, seed=Hq + D)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_page_sizes(bs, layout):
    c = Case([4, 2, 8], [3 * bs + 1, bs, 11 * bs - 1], 8, 2, 64, bs, seed=bs, layout=layout)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("ctx", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 5000, 20011])
@pytest.mark.parametrize("n_q", [1, 8])
def test_lengths(ctx, n_q):
    n = min(n_q, ctx)
    c = Case([n], [ctx], 8, 1, 128, 16, seed=ctx)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("n_q,ctx", [([130], [130]), ([300], [1000]), ([257, 1, 64], [257, 500, 64]),
                                     ([1000], [1003]), ([33, 700], [90, 700])])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (8, 1, 128), (5, 5, 80)])
def test_prompts(n_q, ctx, Hq, Hkv, D):
    c = Case(n_q, ctx, Hq, Hkv, D, 16, seed=sum(n_q) + D)
    assert c.run() == 0
    c.check()
    assert c.run(causal=False) == 0
    c.check(causal=False)
    assert c.run(max_q=1) == 0  # the expected number only chooses a kernel
    c.check()


def test_many_uneven_requests():
    g = torch.Generator().manual_seed(3)
    B = 230
    ctx = [int(x) for x in torch.exp(torch.rand(B, generator=g) * 7.5).long()]
    n_q = [min(int(x), c) for x, c in zip(torch.randint(0, 10, (B,), generator=g), ctx)]
    ctx[5], n_q[5] = 9000, 1
    ctx[6], n_q[6] = 0, 0
    c = Case(n_q, ctx, 8, 2, 64, 16, seed=3)
    assert c.run() == 0
    c.check()
    assert c.run(max_q=1000) == 0
    c.check()


def test_rows_that_see_nothing():
    """No tokens in the cache, and more query tokens than tokens in the cache."""
    c = Case([2, 5, 3], [0, 2, 3], 4, 2, 64, 16, seed=4)
    assert c.run() == 0
    c.check()
    assert torch.all(c.out[:2] == 0) and torch.all(c.lse[:2] == -math.inf)
    assert torch.all(c.out[2:5] == 0) and torch.all(c.lse[2:5] == -math.inf)


@pytest.mark.parametrize("size", [0.0, 0.02, 30.0])
def test_flat_and_peaked_scores(size):
    c = Case([6, 200], [900, 1500], 8, 2, 64, 16, seed=5, size=size)
    assert c.run() == 0
    c.check()


def test_scales_far_apart():
    """Pages whose scales differ by many powers of two, in K and in V."""
    c = Case([6], [1000], 4, 2, 64, 16, seed=6)
    g = gen(1)
    for i, spread in ((2, 3), (3, 12)):
        k = torch.randint(-spread, spread, c.cache[i].shape, generator=g, device=DEV)
        c.cache[i] *= torch.ldexp(torch.ones_like(c.cache[i]), k)
    assert c.run() == 0
    c.check()


def test_zero_scales_and_plain_ones():
    c = Case([3], [300], 4, 2, 64, 16, seed=7)
    c.cache[2][::2] = 0.0
    c.cache[3][::3] = 0.0
    c.cache[2][1::2] *= 0.77
    c.cache[3][1::3] *= 1.31
    assert c.run() == 0
    c.check()
    c.cache[3].zero_()
    assert c.run() == 0
    c.check()
    assert torch.all(c.out == 0)


@pytest.mark.parametrize("n_q,ctx", [([6], [70]), ([1], [129]), ([200], [333]), ([8], [8])])
@pytest.mark.parametrize("bs", [8, 64])
def test_nan_where_nothing_is_seen(n_q, ctx, bs):
    """Bytes beyond the context, pages of others and scales of others may hold anything."""
    c = Case(n_q, ctx, 8, 2, 64, bs, seed=8)
    used = c.table[0, :-(-ctx[0] // bs)].long()
    for i in range(2):
        raw = c.cache[i].view(torch.uint8)
        other = torch.ones(raw.shape[0], dtype=torch.bool, device=DEV)
        other[used] = False
        raw[other] = 0x7F
        if ctx[0] % bs:
            raw[used[-1], ctx[0] % bs:] = 0xFF
        c.cache[i + 2][other] = math.nan
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("n_q,t", [(6, 67), (6, 69), (200, 100), (200, 199), (300, 20)])
def test_nan_reaches_only_the_rows_that_see_it(n_q, t):
    """A NaN in token t's V (one dimension) or K (the whole row's scores)."""
    ctx = 70 if n_q == 6 else n_q
    first = t - (ctx - n_q)  # the first query token that sees token t
    for side in (1, 0):
        c = Case([n_q], [ctx], 4, 2, 64, 16, seed=9)
        page, off = int(c.table[0, t // 16]), t % 16
        c.cache[side].view(torch.uint8)[page, off, 1, 5] = 0x7F
        assert c.run() == 0
        got, lse = c.out, c.lse
        hit = torch.zeros_like(got, dtype=torch.bool)
        if side == 1:
            hit[max(first, 0):, 2:, 5] = True
        else:
            hit[max(first, 0):, 2:] = True
        assert torch.equal(torch.isnan(got), hit)
        if side == 1:
            assert not torch.isnan(lse).any()
        # the others as without it
        c.cache[side].view(torch.uint8)[page, off, 1, 5] = 0
        o = got.clone()
        assert c.run() == 0
        if side == 1:
            assert torch.all((o == c.out)[~hit])


def test_infinite_and_nan_queries():
    c = Case([4, 3], [50, 200], 4, 2, 64, 16, seed=10)
    c.q[1, 2, 7] = math.nan
    c.q[5, 0, 1] = math.inf
    assert c.run() == 0
    bad = torch.zeros(7, 4, dtype=torch.bool, device=DEV)
    bad[1, 2] = bad[5, 0] = True
    assert torch.equal(torch.isnan(c.out).any(-1), bad)
    keep = c.out.clone()
    c.q[1, 2, 7] = c.q[5, 0, 1] = 0.5
    assert c.run() == 0
    assert torch.equal(keep[~bad], c.out[~bad])


def test_holes_in_the_table():
    """Entries outside the cache: their tokens are left out, and the call says so."""
    c = Case([5, 2, 40], [200, 90, 400], 4, 2, 64, 16, seed=11)
    hide = [torch.zeros(n, dtype=torch.bool, device=DEV) for n in c.ctx]
    keep = c.table.clone()
    for r, i, bad in ((0, 3, -1), (0, 12, 10 ** 6), (2, 0, -5), (2, 9, c.cache[0].shape[0])):
        c.table[r, i] = bad
        hide[r][i * 16:(i + 1) * 16] = True
    assert c.run() == sd.SD_ERR_KV_RANGE
    c.table = keep
    c.check(hide=hide)


def test_lengths_out_of_range():
    """A context longer than its table is cut, a negative one is empty, prefixes are clamped."""
    c = Case([3, 2, 2], [160, 32, 100], 4, 2, 64, 16, seed=12)
    c.lens[1] = -4
    assert c.run() == sd.SD_ERR_KV_RANGE
    assert torch.all(c.out[3:5] == 0)
    c.lens[1] = 32
    c.table = c.table[:, :10].contiguous()
    c.lens[0] = 170  # 160 are covered; the new tokens stand at 167, 168 and 169
    assert c.run() == sd.SD_ERR_KV_RANGE
    assert c.run(causal=False) == sd.SD_ERR_KV_RANGE
    c.check(causal=False)
    c.lens[0] = 160
    c.cu[3] = 1000
    assert c.run() == sd.SD_ERR_KV_RANGE
    c.check()


def test_strided_queries_and_outputs():
    g = gen(13)
    c = Case([5, 9], [77, 500], 8, 2, 64, 16, seed=13)
    n = c.q.shape[0]
    qkv = torch.randn(n, 12, 64, generator=g, device=DEV).bfloat16()
    qkv[:, 2:10] = c.q
    c.q = qkv[:, 2:10]
    wide = torch.full((n, 10, 72), 7.0, device=DEV).bfloat16()
    assert c.run(out=wide[:, 1:9, :64]) == 0
    c.check()
    assert torch.all(wide[:, 0] == 7) and torch.all(wide[:, 9] == 7) and torch.all(wide[..., 64:] == 7)


def test_rows_of_no_request_are_not_written():
    c = Case([4, 4], [60, 60], 4, 2, 64, 16, seed=14)
    c.cu = torch.tensor([2, 5, 7], dtype=torch.int32, device=DEV)
    assert c.run() == 0
    for i in (0, 1, 7):
        assert torch.all(c.out[i] == 7.0) and torch.all(c.lse[i] == 7.0)
    assert not torch.any(c.lse[2:7] == 7.0)


def test_no_lse_and_workspace_contents():
    """The result does not depend on what the scratch held, nor on asking for lse."""
    c = Case([6] * 3, [3000, 40, 900], 8, 2, 128, 16, seed=15)
    assert c.run() == 0
    want, lse = c.out.clone(), c.lse.clone()
    need = max(16, sd.sd_kv_attend_workspace_bytes(128))
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        assert c.run(workspace_buf=ws) == 0
        assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
    out = torch.zeros_like(want)
    sd.sd_kv_attend(c.q, *c.cache, c.table, c.lens, c.cu, out, max_q=6)
    assert torch.equal(out, want)


def test_offsets_beyond_32_bits():
    """Pages 2^31 and more elements apart."""
    bs, H, D = 16, 1, 64
    c = Case([3], [40], 4, H, D, bs, seed=16)
    assert c.run() == 0
    want = c.out.clone()
    nb = c.cache[0].shape[0]
    stride = 2 ** 31 + 2 ** 20
    room = torch.zeros(2, (nb - 1) * stride + bs * H * D, dtype=torch.uint8, device=DEV)
    for i in range(2):
        far = torch.as_strided(room[i], (nb, bs, H, D), (stride, H * D, D, 1))
        far.copy_(c.cache[i].view(torch.uint8))
        c.cache[i] = far
    assert c.run() == 0
    assert torch.equal(c.out, want)


def test_on_another_stream_in_a_graph_and_again():
    c = Case([6, 1, 150], [2000, 300, 150], 8, 2, 64, 16, seed=17)
    assert c.run() == 0
    want = c.out.clone()
    assert c.run() == 0
    assert torch.equal(c.out, want)  # the same bits every time
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert c.run(stream=side) == 0
    assert torch.equal(c.out, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_kv_attend(c.q, *c.cache, c.table, c.lens, c.cu, out, max_q=150)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # new lengths in the same graph
    c.lens.copy_(torch.tensor([500, 299, 150], dtype=torch.int32, device=DEV))
    c.ctx = [500, 299, 150]
    graph.replay()
    torch.cuda.synchronize()
    c.out = out
    assert c.run(max_q=150) == 0
    assert torch.equal(c.out, out)
    c.check()


def test_write_then_attend_matches_attention_on_what_was_written():
    """A step: its tokens are quantised into the cache and attended to by their own call."""
    g = gen(18)
    c = Case([4, 7], [100, 45], 8, 2, 64, 16, seed=18)
    n = sum(c.n_q)
    k = torch.randn(n, 2, 64, generator=g, device=DEV).bfloat16()
    slots = []
    for r in range(2):
        for i in range(c.n_q[r]):
            p = c.ctx[r] - c.n_q[r] + i
            slots.append(int(c.table[r, p // 16]) * 16 + p % 16)
    sd.sd_kv_write(k, 2 * k, torch.tensor(slots, dtype=torch.int32, device=DEV), *c.cache)
    assert c.run() == 0
    c.check()
    got = kvref.held(c.cache[0], c.cache[2], c.table[0], 100)[-4:]
    assert float((got - k[:4].double()).norm() / k[:4].double().norm()) < 0.04


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 64, 8)])
def test_a_large_cache_seen_for_the_first_time(D, Hq, Hkv):
    """Pages all over gigabytes of memory that the GPU has not touched lately arrive late and in
    any order: every stage of K and V is waited for in its own phase, whichever stream runs
    ahead. Every kernel of this head size, units of a part of a request and of whole ones, rows that
    do not fill a warp."""
    g = torch.Generator().manual_seed(8)
    B, n = 96, 28 if D == 128 else 14
    ctx = [int(x) for x in torch.randint(n, 16000, (B,), generator=g)]
    c = Case([n] * B, ctx, Hq, Hkv, D, 16, seed=8)
    for rows in (32, 64, 128, 256):
        assert c.run(max_q=max(1, rows * Hkv // Hq)) == 0
        c.check(only=(0, 31, 64, 95))
