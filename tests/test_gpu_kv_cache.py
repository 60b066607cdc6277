"""The paged 8-bit cache: sd_kv_write and sd_kv_read against the definition in 64 bits, exactly."""

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def same(got, want):
    return torch.equal(got.view(torch.int64), want.view(torch.int64)) or bool(
        ((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


def write(k, v, slots, cache, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sd.sd_kv_write(k, v, slots, *cache, err=err, **kw)
    torch.cuda.synchronize()
    return int(err)


def check_write(k, v, slots, cache, want_err=0):
    """Writes, and compares every byte's value and every scale with the definition."""
    before = [t.clone() for t in cache]
    err = write(k, v, slots, cache)
    assert err == want_err
    for i, x in ((0, k), (1, v)):
        values, scale = kvref.write_ref(x.double().cpu(), slots.cpu(),
                                        before[i].double().cpu(), before[i + 2].double().cpu())
        assert same(cache[i + 2].double().cpu(), scale)
        assert same(cache[i].double().cpu(), values)


def slots_of(table, bs, positions):
    """Slots of (request, position) pairs."""
    r = torch.tensor([a for a, _ in positions], device=DEV)
    p = torch.tensor([b for _, b in positions], device=DEV)
    return (table[r, p // bs] * bs + (p % bs)).to(torch.int32)


@pytest.mark.parametrize("D,H,bs", [(64, 8, 16), (128, 2, 16), (16, 1, 8), (80, 3, 32),
                                    (96, 2, 128), (112, 1, 64), (32, 5, 16), (48, 2, 8)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_steps_grow_scales(D, H, bs, layout):
    g = gen(D + H)
    lens = [3, 2 * bs - 1, 5 * bs]
    nb, table = kvref.make_table([n + 40 for n in lens], bs, g, DEV)
    cache = list(kvref.make_cache(nb, bs, H, D, g, DEV, layout))
    for step, size in enumerate([1.0, 40.0, 0.01, 3000.0]):  # the second and last make scales grow
        n = [1, 6, 9]
        pos = [(r, lens[r] + i) for r in range(3) for i in range(n[r])]
        qkv = size * torch.randn(len(pos), 3, H, D, generator=g, device=DEV)
        qkv = qkv.bfloat16()
        slots = slots_of(table, bs, pos)
        slots[4] = -1
        check_write(qkv[:, 1], qkv[:, 2], slots, cache)
        lens = [a + b for a, b in zip(lens, n)]


@pytest.mark.parametrize("n", [1, 7, 500, 4099])
def test_prompt_into_zeroed_cache(n):
    g = gen(n)
    bs, H, D = 16, 2, 64
    nb, table = kvref.make_table([n], bs, g, DEV)
    cache = [torch.zeros(nb, bs, H, D, device=DEV).to(E4M3), torch.zeros(nb, bs, H, D, device=DEV).to(E4M3),
             torch.zeros(nb, H, device=DEV), torch.zeros(nb, H, device=DEV)]
    k = torch.randn(n, H, D, generator=g, device=DEV).bfloat16()
    v = torch.randn(n, H, D, generator=g, device=DEV).bfloat16()
    check_write(k, v, slots_of(table, bs, [(0, i) for i in range(n)]), cache)


def test_values_at_the_borders():
    """Zeros, the smallest and largest bf16, amax at and beside 448 2^k, infinities and NaN."""
    bs, H, D = 16, 1, 16
    rows = [[0.0] * 16, [1e-38, -9e-41] + [0.0] * 14, [3.3895e38, 1.0] + [0.0] * 14,
            [448.0, 1e-3] + [0.5] * 14, [450.0, 2.0] + [-0.0] * 14, [3.5, 0.0068] + [1.0] * 14,
            [float("inf"), -2.0] + [7.0] * 14, [float("nan"), -2.0] + [7.0] * 14,
            [float("-inf")] * 16, [float("nan")] * 16]
    k = torch.tensor(rows, device=DEV).bfloat16().view(len(rows), H, D)
    g = gen(1)
    for fresh in (True, False):
        cache = list(kvref.make_cache(len(rows), bs, H, D, g, DEV))
        slots = torch.arange(len(rows), dtype=torch.int32, device=DEV) * bs + (0 if fresh else 5)
        check_write(k, -k, slots, cache)


def test_page_starts_afresh():
    """A write to slot 0 forgets the scale that the page had; a later slot keeps it."""
    g = gen(2)
    cache = list(kvref.make_cache(2, 16, 2, 64, g, DEV))
    cache[2].fill_(2.0 ** 20)
    cache[3].fill_(2.0 ** 20)
    k = torch.randn(2, 2, 64, generator=g, device=DEV).bfloat16()
    check_write(k, k, torch.tensor([0, 16 + 3], dtype=torch.int32, device=DEV), cache)
    assert float(cache[2][0].max()) < 1 and float(cache[2][1].min()) == 2.0 ** 20


def test_scales_that_are_no_powers_of_two():
    g = gen(3)
    cache = list(kvref.make_cache(3, 16, 2, 32, g, DEV))
    cache[2].copy_(torch.tensor([[0.013, 3.7], [0.0, -1.0], [0.3, 1e-5]], device=DEV))
    k = torch.randn(3, 2, 32, generator=g, device=DEV).bfloat16()
    slots = torch.tensor([5, 16 + 2, 32 + 9], dtype=torch.int32, device=DEV)
    before = [t.clone() for t in cache]
    assert write(k, k, slots, cache) == 0
    values, scale = kvref.write_ref(k.double().cpu(), slots.cpu(), before[0].double().cpu(),
                                    before[2].double().cpu())
    assert same(cache[2].double().cpu(), scale)
    # quotients and ratios of such scales are rounded to fp32 first, which can move a tie
    got = cache[0].double().cpu()
    assert float((got != values).double().mean()) < 0.01
    assert torch.all((got - values).abs() <= 2.0 ** -3 * values.abs() + 2.0 ** -9)


def test_order_and_repeats_within_a_page():
    g = gen(4)
    cache = list(kvref.make_cache(2, 32, 2, 48, g, DEV))
    k = torch.randn(9, 2, 48, generator=g, device=DEV).bfloat16()
    slots = torch.tensor([9, 3, 3, 31, 20, 9, 32 + 7, 32 + 1, 32 + 7], dtype=torch.int32, device=DEV)
    check_write(k, k, slots, cache)


def test_slots_beyond_the_cache_are_skipped():
    g = gen(5)
    bs, H, D, nb = 16, 2, 64, 3
    big = list(kvref.make_cache(nb + 2, bs, H, D, g, DEV))
    guard = [t.clone() for t in big]
    cache = [t[1:1 + nb] for t in big]
    k = torch.randn(5, H, D, generator=g, device=DEV).bfloat16()
    slots = torch.tensor([nb * bs, 5, -7, 2 ** 31 - 1, nb * bs - 1], dtype=torch.int32, device=DEV)
    check_write(k, k, slots, cache, sd.SD_ERR_KV_SLOT)
    for t, u in zip(big, guard):
        for i in (0, nb + 1):
            assert torch.equal(t[i].view(torch.uint8), u[i].view(torch.uint8))


def test_nothing_to_write():
    cache = list(kvref.make_cache(2, 16, 2, 64, gen(6), DEV))
    k = torch.randn(3, 2, 64, device=DEV).bfloat16()
    check_write(k, k, torch.full((3,), -1, dtype=torch.int32, device=DEV), cache)
    check_write(k[:0], k[:0], torch.empty(0, dtype=torch.int32, device=DEV), cache)


@pytest.mark.parametrize("D,H,bs", [(64, 8, 16), (128, 2, 32), (16, 1, 8), (80, 3, 128)])
def test_read(D, H, bs):
    g = gen(D)
    lens = [1, 0, 3 * bs, 7 * bs - 1, 2]
    nb, table = kvref.make_table(lens, bs, g, DEV)
    cache = kvref.make_cache(nb, bs, H, D, g, DEV, "head" if bs == 32 else "token")
    n = sum(lens)
    out = [torch.full((n + 3, H, D), 7.0, device=DEV).bfloat16() for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sd.sd_kv_read(*cache, table, kvref.prefix(lens, DEV), *out, err=err)
    assert int(err) == 0
    for i in range(2):
        want = torch.cat([kvref.held(cache[i], cache[i + 2], table[r], lens[r])
                          for r in range(len(lens))])
        assert torch.equal(out[i][:n].double(), want)
        assert torch.all(out[i][n:] == 7.0)


def test_read_a_range_and_uncovered_positions():
    g = gen(9)
    bs, H, D = 16, 2, 64
    nb, table = kvref.make_table([50, 20], bs, g, DEV)
    cache = kvref.make_cache(nb, bs, H, D, g, DEV)
    first = torch.tensor([13, 10], dtype=torch.int32, device=DEV)
    table[0, 2] = -1      # a hole in the first request's table
    table[1, 1] = nb + 5  # a page that there is not
    out = [torch.full((40, H, D), 7.0, device=DEV).bfloat16() for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sd.sd_kv_read(*cache, table, kvref.prefix([22, 18], DEV), *out, first_pos=first, err=err)
    assert int(err) == sd.SD_ERR_KV_RANGE
    for i in range(2):
        a = cache[i].double() * cache[i + 2].double()[:, None, :, None]
        for row in range(40):
            r, pos = (0, 13 + row) if row < 22 else (1, 10 + row - 22)
            page = int(table[r, pos // bs]) if pos // bs < table.shape[1] else -1
            want = a[page, pos % bs] if 0 <= page < nb else torch.zeros_like(a[0, 0])
            assert torch.equal(out[i][row].double(), want), (row, pos)


def test_offsets_beyond_32_bits():
    """Pages 2^31 and more elements apart."""
    g = gen(10)
    bs, H, D, nb = 16, 1, 64, 3
    stride = 2 ** 31 + 2 ** 20
    room = torch.zeros(2, (nb - 1) * stride + bs * H * D, dtype=torch.uint8, device=DEV)
    small = kvref.make_cache(nb, bs, H, D, g, DEV)
    cache = [torch.as_strided(room[i], (nb, bs, H, D), (stride, H * D, D, 1)) for i in range(2)]
    for i in range(2):
        cache[i].copy_(small[i].view(torch.uint8))
    scales = [small[2].clone(), small[3].clone()]
    k = torch.randn(2, H, D, generator=g, device=DEV).bfloat16()
    slots = torch.tensor([2 * bs + 3, bs + 5], dtype=torch.int32, device=DEV)
    check_write(k, k, slots, list(small))
    sd.sd_kv_write(k, k, slots, *cache, *scales)
    for i in range(2):
        assert torch.equal(cache[i], small[i].view(torch.uint8))
        assert torch.equal(scales[i], small[i + 2])
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    out = [torch.zeros(40, H, D, device=DEV).bfloat16() for _ in range(4)]
    sd.sd_kv_read(*cache, *scales, table, kvref.prefix([40], DEV), *out[:2])
    sd.sd_kv_read(*small, table, kvref.prefix([40], DEV), *out[2:])
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


def test_on_another_stream_and_in_a_graph():
    g = gen(11)
    bs, H, D = 16, 2, 64
    nb, table = kvref.make_table([64], bs, g, DEV)
    cache = list(kvref.make_cache(nb, bs, H, D, g, DEV))
    fresh = [t.clone() for t in cache]
    k = torch.randn(20, H, D, generator=g, device=DEV).bfloat16()
    slots = slots_of(table, bs, [(0, 20 + i) for i in range(20)])
    out = [torch.zeros(64, H, D, device=DEV).bfloat16() for _ in range(2)]
    cu = kvref.prefix([64], DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sd.sd_kv_write(k, k, slots, *cache)
        sd.sd_kv_read(*cache, table, cu, *out)
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for t, u in zip(cache, fresh):
        t.copy_(u)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_kv_write(k, k, slots, *cache)
        sd.sd_kv_read(*cache, table, cu, *out)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("gap", [[2 ** 31 - 1], [-1, 1 << 20, -7], [1 << 20] * 31])
def test_a_page_around_slots_beyond_the_cache(gap):
    """Skipped entries inside a page's tokens, of either kind, leave them one stretch."""
    g = gen(12)
    bs, H, D = 16, 2, 64
    nb, table = kvref.make_table([40], bs, g, DEV)
    cache = list(kvref.make_cache(nb, bs, H, D, g, DEV))
    pos = [(0, i) for i in range(16, 30)]
    slots = slots_of(table, bs, pos)
    slots = torch.cat([slots[:6], torch.tensor(gap, dtype=torch.int32, device=DEV), slots[6:]])
    k = 100 * torch.randn(slots.numel(), H, D, generator=g, device=DEV)
    check_write(k.bfloat16(), (k / 3).bfloat16(), slots, cache,
                sd.SD_ERR_KV_SLOT if max(gap) > 0 else 0)
