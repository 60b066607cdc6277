"""sd_rope against angles from whole numbers, in 64 bits."""

import pytest
import torch

import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"


def check(x, got, positions, turns, pairs, scale=1.0, inverse=False):
    want, tol = stepref.rope_ref(x.double().cpu(), positions.tolist(),
                                 [t % stepref.TWO64 for t in turns.tolist()], pairs, scale, inverse)
    assert torch.all((got.double().cpu() - want).abs() <= tol)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("n,Hq,Hk,D,rot", [
    (1, 1, 0, 8, 2), (1, 8, 2, 64, 64), (5, 0, 3, 128, 128), (7, 7, 1, 80, 40), (3, 4, 4, 96, 48),
    (6, 2, 1, 128, 64), (2, 3, 1, 40, 6), (4, 1, 1, 512, 512), (3, 2, 2, 264, 30), (2, 1, 1, 512, 6),
    (19, 5, 3, 64, 32)])
def test_shapes(n, Hq, Hk, D, rot, pairs):
    g = torch.Generator(device=DEV)
    g.manual_seed(n * 1000 + D + rot)
    turns, _ = sd.sd_rope_table(rot, base=10000.0, device=DEV)
    pos = torch.randint(0, 131072, (n,), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn(n, Hq + Hk + 1, D, generator=g, device=DEV, dtype=torch.bfloat16)
    q, k = (x[:, :Hq] if Hq else None), (x[:, Hq:Hq + Hk] if Hk else None)
    outs = [None if t is None else torch.full_like(t, 9.0, memory_format=torch.contiguous_format)
            for t in (q, k)]
    sd.sd_rope(pos, turns, q=q, k=k, q_out=outs[0], k_out=outs[1], pairs=pairs)
    torch.cuda.synchronize()
    for t, o in zip((q, k), outs):
        if t is not None:
            check(t, o, pos, turns, pairs)
            assert torch.equal(o[..., rot:], t[..., rot:])
    # in place, within the projection: the same bits, and nothing else touched
    y = x.clone()
    sd.sd_rope(pos, turns, q=y[:, :Hq] if Hq else None, k=y[:, Hq:Hq + Hk] if Hk else None, pairs=pairs)
    for t, o in zip((y[:, :Hq], y[:, Hq:Hq + Hk]), outs):
        assert o is None or torch.equal(t, o)
    assert torch.equal(y[:, Hq + Hk:], x[:, Hq + Hk:])


@pytest.mark.parametrize("kind,p", [
    ("linear", dict(factor=4.0)), ("ntk", dict(factor=4.0)),
    ("bands", dict(factor=8.0, original_len=8192, low=1.0, high=4.0)),
    ("yarn", dict(factor=8.0, original_len=4096, low=1.0, high=32.0))])
def test_stretched(kind, p):
    turns, scale = sd.sd_rope_table(64, base=5e5, kind=kind, device=DEV, **p)
    pos = torch.tensor([0, 1, 8191, 65535], dtype=torch.int32, device=DEV)
    q = torch.randn(4, 3, 64, device=DEV).bfloat16()
    out = torch.empty_like(q)
    sd.sd_rope(pos, turns, q=q, q_out=out, scale=scale)
    check(q, out, pos, turns, "halves", scale=scale)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_far_and_negative_positions(pairs):
    """Every int32 is a position; the fastest pair has turned 3 10^8 times at the largest."""
    turns, _ = sd.sd_rope_table(128, base=10000.0, device=DEV)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1 << 30, 123456789], dtype=torch.int32, device=DEV)
    k = torch.randn(5, 2, 128, device=DEV).bfloat16()
    out = torch.empty_like(k)
    sd.sd_rope(pos, turns, k=k, k_out=out, pairs=pairs)
    check(k, out, pos, turns, pairs)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_gradient(pairs):
    """inverse gives the gradient: the formula's transpose, and differences of the forward formula."""
    torch.manual_seed(0)
    n, H, D, rot, scale = 3, 2, 32, 16, 1.25
    turns, _ = sd.sd_rope_table(rot, device=DEV)
    pos = torch.tensor([0, 5, 1000], dtype=torch.int32, device=DEV)
    g = torch.randn(n, H, D, device=DEV).bfloat16()
    dx = torch.empty_like(g)
    sd.sd_rope(pos, turns, q=g, q_out=dx, pairs=pairs, scale=scale, inverse=True)
    check(g, dx, pos, turns, pairs, scale=scale, inverse=True)
    ints = [t % stepref.TWO64 for t in turns.tolist()]
    x = torch.randn(n, H, D, dtype=torch.float64)

    def loss(v):
        return (stepref.rope_ref(v, pos.tolist(), ints, pairs, scale, False)[0] * g.double().cpu()).sum()
    # (linear: a difference is exact but for the sums' rounding)
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 9), (2, 1, 15), (1, 0, 20)]:
        e = torch.zeros_like(x)
        e[at] = 0.5
        want = loss(x + e) - loss(x - e)
        if at[2] >= rot:  # what does not turn is not scaled
            want = g[at].double().cpu()
        assert abs(float(dx[at]) - float(want)) <= 2.0 ** -8 * abs(float(want)) + 2.0 ** -18


def test_large_heads_and_strides():
    """Many heads, rows far apart, several heads a group."""
    pos = torch.arange(40, dtype=torch.int32, device=DEV) * 37
    turns, _ = sd.sd_rope_table(128, device=DEV)
    base = torch.randn(40, 3, 97, 128, device=DEV).bfloat16()
    q, k = base[:, 1, :65], base[:, 2, 65:]
    qo, ko = torch.empty(97, 40, 128, device=DEV).bfloat16().transpose(0, 1)[:, :65], torch.empty_like(k)
    sd.sd_rope(pos, turns, q=q, k=k, q_out=qo, k_out=ko)
    check(q, qo, pos, turns, "halves")
    check(k, ko, pos, turns, "halves")


def test_long_call_matches_short_ones():
    """A long call gives every token the bits that a call of its own gives."""
    n = 20000
    pos = torch.randint(0, 1 << 20, (n,), device=DEV, dtype=torch.int32)
    turns, _ = sd.sd_rope_table(64, device=DEV)
    q = torch.randn(n, 9, 64, device=DEV).bfloat16()
    out = torch.empty_like(q)
    sd.sd_rope(pos, turns, q=q, q_out=out)
    for i in (0, 1, 8, 9999, n - 1):
        one = torch.empty_like(q[:1])
        sd.sd_rope(pos[i:i + 1], turns, q=q[i:i + 1], q_out=one)
        assert torch.equal(out[i:i + 1], one)
        check(q[i:i + 1], one, pos[i:i + 1], turns, "halves")


def test_nothing_and_captured():
    turns, _ = sd.sd_rope_table(64, device=DEV)
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    sd.sd_rope(torch.empty(0, dtype=torch.int32, device=DEV), turns, q=empty)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    q = torch.randn(6, 4, 64, device=DEV).bfloat16()
    out, want = torch.empty_like(q), torch.empty_like(q)
    sd.sd_rope(pos, turns, q=q, q_out=want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.sd_rope(pos, turns, q=q, q_out=out)
    for shift in (0, 100):
        pos += shift
        sd.sd_rope(pos, turns, q=q, q_out=want)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.current_stream().synchronize()
    sd.sd_rope(pos, turns, q=q, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_back_to_the_unrotated_key(pairs):
    """Forward with a scale, then inverse with 1 / scale: the key again, rounded to bf16 twice."""
    turns, scale = sd.sd_rope_table(64, base=5e5, kind="yarn", factor=16.0, original_len=4096, device=DEV)
    pos = torch.tensor([0, 3, 4095, 60000], dtype=torch.int32, device=DEV)
    k = torch.randn(4, 2, 80, device=DEV).bfloat16()
    there, back = torch.empty_like(k), torch.empty_like(k)
    sd.sd_rope(pos, turns, k=k, k_out=there, pairs=pairs, scale=scale)
    sd.sd_rope(pos, turns, k=there, k_out=back, pairs=pairs, scale=1.0 / scale, inverse=True)
    assert torch.equal(back[..., 64:], k[..., 64:])
    x, y = k[..., :64].double(), back[..., :64].double()
    pair = (x.view(4, 2, 2, 32).norm(dim=2, keepdim=True).expand(4, 2, 2, 32) if pairs == "halves"
            else x.view(4, 2, 32, 2).norm(dim=3, keepdim=True).expand(4, 2, 32, 2)).reshape(4, 2, 64)
    # each value of the turned pair is off by 2^-8 of itself, so the pair by 2^-8 of its length; then once more
    assert torch.all((x - y).abs() <= pair * (2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -18) + 2.0 ** -8 * x.abs())
