"""sd_kv_attend on rows with dominant tokens: what thousands of small weights add up to.

The tolerance counts each weight's own rounding. In units in which the largest weight of the row so far
is 2^10 or more and the largest of each tile of 128 tokens 2^-2 or more, a weight is off by 2^-8 of itself
(half a step of 8 significant bits) or by 2^-10 (half of the second term's finest step), but by no
more than 2^-3 of itself (half a step of the first term's 3 significant bits) and 2^-17 (half of its finest
step). Away from a dominant token's tile the bound is relative to sum p |v|, however many tokens there
are. Sums are fp32: a row's L takes a term for each 8 tokens, its accumulator one for each 32."""

import math

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"
TILE = 128


def reference(q, k, v, first):
    """One KV head in 64 bits: q [n, G, D] (token i sees k[:first + i + 1]), k, v [T, D]. Returns out,
    lse and their tolerances."""
    n, G, D = q.shape
    T = k.shape[0]
    sm = D ** -0.5
    x = (q @ k.T) * sm
    seen = torch.arange(T, device=q.device)[None] <= first + torch.arange(n, device=q.device)[:, None]
    x = torch.where(seen[:, None], x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    tiles = torch.nn.functional.pad(p, (0, -T % TILE)).view(n, G, -1, TILE)
    near = tiles.amax(-1, keepdim=True)
    far = near.cummax(-2).values
    unit = torch.minimum(2.0 ** -10 * far, 4 * near).expand_as(tiles).reshape(n, G, -1)[..., :T]
    off = torch.maximum(2.0 ** -8 * p, torch.minimum(2.0 ** -3 * p + 2.0 ** -17 * unit,
                                                     2.0 ** -10 * unit))
    # q to 2^-18 of its largest, products and sums of a score in fp32
    ds = (2.0 ** -18 * q.abs().amax(-1)[..., None] * k.abs().sum(1)
          + (D + 8) * 2.0 ** -24 * (q.abs() @ k.abs().T)) * sm
    ds = torch.where(seen[:, None], ds, torch.zeros_like(ds)).amax(-1)
    fp32 = 2.0 ** -20 + (T / 4) * 2.0 ** -24
    out, a = p @ v, p @ v.abs()
    tol = 2.0 ** -8 * out.abs() + off @ v.abs() + (2 * ds + fp32)[..., None] * a
    return out, lse, tol, ds + fp32 + 2.0 ** -22 * lse.abs()


class Peaked:
    """Requests of n new tokens at the end of T, with tokens `at` that every query prefers to the
    others by `gap` (in natural units, over the others' mean), their V `sink_v` times the others'. The
    others' scores spread by `spread`. alone: the other tokens of their tiles have V 0."""

    def __init__(self, n, T, Hq, Hkv, D, at, gap, spread, sink_v, seed, B=1, alone=False):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        bs, H = 16, Hkv
        nb, self.table = kvref.make_table([T] * B, bs, g, DEV, extra=1)
        self.n, self.T, self.Hq, self.Hkv, self.D, self.B = n, T, Hq, Hkv, D, B
        # dimension 0 tells the dominant tokens from the others
        self.q = torch.randn(B * n, Hq, D, generator=g, device=DEV)
        self.q[..., 0] = 8.0
        self.q = self.q.bfloat16()
        raw = []
        for side in range(2):
            x = torch.randn(B, T, H, D, generator=g, device=DEV)
            x = x * spread if side == 0 else x + 0.5
            if side == 1:
                x[:, at] *= sink_v
                if alone:
                    for t in at:
                        x[:, t // TILE * TILE:t // TILE * TILE + TILE] = 0.0
            if side == 0:
                x[:, at] = 0.0
                x[..., 0] = 0.0
                for i, t in enumerate(at):
                    x[:, t, :, 0] = gap * D ** 0.5 / 8.0
            raw.append(x)
        self.cache = []
        for x in raw:
            scale = 2.0 ** (math.ceil(math.log2(float(x.abs().max()) / 448)))
            pages = torch.zeros(nb, bs, H, D, device=DEV)
            for b in range(B):
                for i in range(-(-T // bs)):
                    part = x[b, i * bs:(i + 1) * bs]
                    pages[int(self.table[b, i]), :part.shape[0]] = part
            self.cache.append((pages / scale).to(kvref.E4M3))
            self.cache.append(torch.full((nb, H), scale, device=DEV))
        self.cache = [self.cache[0], self.cache[2], self.cache[1], self.cache[3]]
        self.cu = kvref.prefix([n] * B, DEV)
        self.lens = torch.full((B,), T, dtype=torch.int32, device=DEV)

    def check(self, max_q=None):
        out = torch.full((self.B * self.n, self.Hq, self.D), 7.0, device=DEV).bfloat16()
        lse = torch.full((self.B * self.n, self.Hq), 7.0, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sd.sd_kv_attend(self.q, *self.cache, self.table, self.lens, self.cu, out, lse=lse,
                        max_q=self.n if max_q is None else max_q, err=err)
        assert int(err) == 0
        G = self.Hq // self.Hkv
        for b in range(self.B):
            k = kvref.held(self.cache[0], self.cache[2], self.table[b], self.T)
            v = kvref.held(self.cache[1], self.cache[3], self.table[b], self.T)
            rows = slice(b * self.n, (b + 1) * self.n)
            for h in range(self.Hkv):
                heads = slice(h * G, (h + 1) * G)
                o, l, tol, tol_l = reference(self.q[rows, heads].double(), k[:, h], v[:, h],
                                             self.T - self.n)
                d = (out[rows, heads].double() - o).abs()
                assert torch.all(d <= tol), float((d / (tol + 1e-300)).max())
                assert torch.all((lse[rows, heads].double() - l).abs() <= tol_l)
        return out, lse


# units of 32, 64, 128 and 256 rows: a step's slots, a drafter's rows, a chunk of a prompt
FORMS = [(4, 4), (8, 6), (16, 7), (50, 8)]  # query tokens, query heads of a KV head


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [300, 8192, 32000])
@pytest.mark.parametrize("gap", [7.0, 10.0, 12.0, 14.0])
def test_one_dominant_token(n, G, D, T, gap):
    """The others alike or spread, the dominant one first, in the middle or among the last."""
    for spread, at in ((0.0, 0), (0.0, T // 2 + 5), (1.5, 1), (1.5, T - n - 1)):
        Peaked(n, T, G, 1, D, [at], gap, spread, 0.01, seed=T + n).check()


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D", [64, 80, 128])
def test_several_dominant_tokens(n, G, D):
    """References that fall behind each of them and rise to the next, over several requests and heads."""
    at = [0, 40, 700, 701, 1500, 2600]
    c = Peaked(n, 3000, 2 * G, 2, D, at, 13.0, 1.0, 0.02, seed=n, B=3)
    out, lse = c.check()
    again, l = c.check()
    assert torch.equal(out, again) and torch.equal(lse, l)
    c.check(max_q=1)  # every unit 32 rows


@pytest.mark.parametrize("gap", [30.0, 40.0])
@pytest.mark.parametrize("n,G", FORMS)
def test_far_apart(n, G, gap):
    """Weights 43 and 57 binades below the dominant ones, whose tiles have V 0: the others are all of
    the answer, to the same relative bound."""
    for D in (64, 128):
        Peaked(n, 2000, G, 1, D, [3, 1200], gap, 0.5, 0.0, seed=5, alone=True).check()


@pytest.mark.parametrize("n,G", FORMS)
def test_beyond_any_range(n, G):
    """A dominant token 288 binades above the others: they count as nothing, nothing overflows."""
    for D in (64, 128):
        c = Peaked(n, 2000, G, 1, D, [900], 200.0, 0.5, 1.0, seed=6)
        c.check()
