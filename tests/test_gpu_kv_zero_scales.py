"""A page whose scale is 0 holds zeros, whatever its bytes: only scales need to be zeroed memory."""

import math

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = kvref.E4M3


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def bytes_of_any_kind(shape, g):
    """Among them NaN of both signs and the largest values."""
    raw = torch.randint(0, 256, shape, generator=g, device=DEV).to(torch.uint8)
    raw.view(-1)[::7] = 0x7F
    raw.view(-1)[3::7] = 0xFF
    return raw


@pytest.mark.parametrize("D", [16, 64, 80, 128])
def test_read(D):
    g = gen(D)
    nb, table = kvref.make_table([100], 16, g, DEV)
    cache = list(kvref.make_cache(nb, 16, 2, D, g, DEV))
    want = [c.clone() for c in cache]
    for i in range(2):
        cache[i] = bytes_of_any_kind(cache[i].shape, g).view(E4M3)
        cache[i].view(torch.uint8)[1::2] = want[i].view(torch.uint8)[1::2]
        cache[i + 2][::2] = 0.0
        want[i].view(torch.uint8)[::2] = 0
    out = [torch.full((100, 2, D), 7.0, device=DEV).bfloat16() for _ in range(4)]
    sd.sd_kv_read(*cache, table, kvref.prefix([100], DEV), *out[:2])
    sd.sd_kv_read(*want, table, kvref.prefix([100], DEV), *out[2:])
    for i in range(2):
        assert torch.all(out[i] == out[i + 2])


@pytest.mark.parametrize("D,bs", [(64, 16), (80, 32), (128, 8), (16, 128)])
def test_write_into_the_middle(D, bs):
    """The page's other slots hold zeros afterwards."""
    g = gen(D + bs)
    shape = (3, bs, 2, D)
    cache = [bytes_of_any_kind(shape, g).view(E4M3) for _ in range(2)]
    scales = [torch.zeros(3, 2, device=DEV) for _ in range(2)]
    k = torch.randn(2, 2, D, generator=g, device=DEV).bfloat16()
    slots = torch.tensor([bs + 3, 2 * bs + bs - 1], dtype=torch.int32, device=DEV)
    before = [c.clone() for c in cache]
    sd.sd_kv_write(k, 3 * k, slots, *cache, *scales)
    zero = [torch.zeros(shape, device=DEV).to(E4M3) for _ in range(2)]
    zs = [torch.zeros(3, 2, device=DEV) for _ in range(2)]
    sd.sd_kv_write(k, 3 * k, slots, *zero, *zs)
    for i in range(2):
        assert torch.equal(scales[i], zs[i])
        assert torch.all(cache[i].float()[1:] == zero[i].float()[1:])
        assert torch.equal(cache[i][0].view(torch.uint8), before[i][0].view(torch.uint8))


# units of 32, 64, 128 and 256 rows
@pytest.mark.parametrize("n,G", [(4, 4), (8, 6), (16, 7), (50, 8)])
@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("sides", [(0,), (1,), (0, 1)])
def test_attend(n, G, D, sides):
    """Every bit as with bytes of 0; NaN queries stay NaN."""
    g = gen(D + n)
    T, bs = 1000, 16
    nb, table = kvref.make_table([T, T], bs, g, DEV)
    cache = list(kvref.make_cache(nb, bs, 1, D, g, DEV))
    clean = [c.clone() for c in cache]
    none = torch.zeros(nb, dtype=torch.bool, device=DEV)
    none[::3] = True
    none[table[1, :-(-T // bs)].long()] = True  # all of one request
    for i in sides:
        raw = bytes_of_any_kind(cache[i].shape, g)
        cache[i].view(torch.uint8)[none] = raw[none]
        clean[i].view(torch.uint8)[none] = 0
        cache[i + 2][none] = 0.0
        clean[i + 2][none] = 0.0
    q = torch.randn(2 * n, G, D, generator=g, device=DEV).bfloat16()
    q[1, 0, 3] = math.nan
    q[n + 2, 1, 0] = math.inf
    cu = kvref.prefix([n, n], DEV)
    lens = torch.full((2,), T, dtype=torch.int32, device=DEV)
    got = []
    for c in (cache, clean):
        out, lse = torch.zeros_like(q), torch.zeros(2 * n, G, device=DEV)
        sd.sd_kv_attend(q, *c, table, lens, cu, out, lse=lse, max_q=n)
        got.append((out, lse))
    bad = torch.zeros(2 * n, G, dtype=torch.bool, device=DEV)
    bad[1, 0] = bad[n + 2, 1] = True
    for a, b in zip(*got):
        assert torch.equal(torch.isnan(a).view(2 * n, G, -1).any(-1), bad)
        assert torch.equal(a[~bad], b[~bad])
