"""Refusals of the rotary, weight, eviction and cut-row calls, in the C library and in the Python
binding, and the host's table of turns: nothing here needs a GPU."""

import ctypes
import math

import pytest
import torch

import verify_draft_prep_gb300 as sd

P = 256  # a well aligned dummy address; no call below gets as far as using it


@pytest.fixture(scope="module")
def lib():
    sd.build()
    return sd.load()


def weights_args(**over):
    a = dict(B=2, n=3, max_q=2, Hq=4, Hkv=2, D=64, q=P, ld_q=256, hs_q=64, lse=P, k_cache=P,
             st_block=2048, st_tok=128, st_head=64, k_scale=P, num_blocks=4, block_size=16, table=P,
             max_blocks=4, ctx=P, cu=P, live=None, sm_scale=0.125, causal=1, decay=1.0, before=None,
             weights=P, err=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


def evict_args(**over):
    a = dict(B=2, Hkv=2, D=64, k_cache=P, v_cache=P, st_block=2048, st_tok=128, st_head=64, k_scale=P,
             v_scale=P, num_blocks=4, block_size=16, weights=P, table=P, max_blocks=4, to=None,
             to_blocks=0, ctx=P, budget=8, sink=2, recent=3, kept=P, new_lens=2 * P, err=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


def rope_args(**over):
    a = dict(n=3, Hq=4, Hk=2, D=64, rot=64, pairs=0, pos=P, turns=P, scale=1.0, inverse=0, q=P,
             ld_q=256, hs_q=64, q_out=P, ld_qo=256, hs_qo=64, k=P, ld_k=128, hs_k=64, k_out=P,
             ld_ko=128, hs_ko=64, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


def cut_args(draw, **over):
    a = dict(B=2, J=3, V=100, dtype=1, rows=P, ld=100, temperature=None, top_k=None, top_p=None,
             min_p=None)
    a.update(dict(u=P, tokens=P, prob=None) if draw else dict(probs=1 << 30, ld_out=100))
    a.update(kept=None, err=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


CACHE = [(dict(D=8), -2), (dict(D=72), -2), (dict(D=144), -2), (dict(Hkv=0), -2),
         (dict(block_size=4), -2), (dict(block_size=24), -2), (dict(num_blocks=-1), -2),
         (dict(num_blocks=1 << 28), -2), (dict(st_block=0), -2), (dict(st_head=24), -4),
         (dict(k_cache=None), -1), (dict(k_scale=None), -1), (dict(k_cache=P + 8), -4),
         (dict(B=-1), -2), (dict(B=65536), -2), (dict(max_blocks=-1), -2), (dict(table=None), -1),
         (dict(ctx=None), -1), (dict(weights=None), -1), (dict(B=0), 0)]


@pytest.mark.parametrize("over,rc", CACHE + [
    (dict(n=-1), -2), (dict(max_q=0), -2), (dict(Hq=5), -2), (dict(num_blocks=0), -2),
    (dict(sm_scale=0.0), -2), (dict(sm_scale=math.inf), -2), (dict(sm_scale=math.nan), -2),
    (dict(decay=-0.5), -2), (dict(decay=math.nan), -2), (dict(decay=math.inf), -2),
    (dict(n=1 << 30), -2), (dict(Hkv=65537, Hq=65537), -2), (dict(q=None), -1), (dict(lse=None), -1),
    (dict(cu=None), -1), (dict(q=P + 8), -4), (dict(ld_q=260), -4)])
def test_weights_refuses(lib, over, rc):
    assert lib.sd_kv_weights(*weights_args(**over)) == rc


@pytest.mark.parametrize("over,rc", CACHE + [
    (dict(v_cache=None), -1), (dict(v_scale=None), -1), (dict(budget=0), -2), (dict(sink=-1), -2),
    (dict(recent=-1), -2), (dict(sink=5, recent=4), -2), (dict(to_blocks=-1), -2),
    (dict(Hkv=65536), -2), (dict(kept=None), -1), (dict(new_lens=None), -1), (dict(v_cache=P + 4), -4)])
def test_evict_refuses(lib, over, rc):
    assert lib.sd_kv_evict(*evict_args(**over)) == rc


@pytest.mark.parametrize("over,rc", [
    (dict(n=-1), -2), (dict(Hq=-1), -2), (dict(Hk=-1), -2), (dict(Hq=1 << 20), -2), (dict(D=4), -2),
    (dict(D=60), -2), (dict(D=520, rot=64), -2), (dict(rot=0), -2), (dict(rot=63), -2),
    (dict(rot=66), -2), (dict(pairs=2), -2), (dict(scale=math.nan), -2), (dict(scale=math.inf), -2),
    (dict(ld_q=-8), -2), (dict(hs_ko=-8), -2), (dict(pos=None), -1), (dict(turns=None), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(k=None), -1), (dict(k_out=None), -1),
    (dict(q=P + 8), -4), (dict(k_out=P + 2), -4), (dict(ld_q=260), -4), (dict(hs_k=68), -4),
    (dict(turns=P + 4), -4), (dict(n=0), 0), (dict(Hq=0, Hk=0), 0)])
def test_rope_refuses(lib, over, rc):
    assert lib.sd_rope(*rope_args(**over)) == rc


@pytest.mark.parametrize("draw", [False, True])
@pytest.mark.parametrize("over,rc", [
    (dict(dtype=2), -3), (dict(B=-1), -2), (dict(J=0), -2), (dict(V=0), -2), (dict(ld=99), -2),
    (dict(V=524225, ld=524225), -2), (dict(B=1 << 27), -2), (dict(rows=None), -1),
    (dict(rows=P + 1), -4), (dict(dtype=0, rows=P + 2), -4), (dict(B=0), 0)])
def test_cut_rows_refuse(lib, draw, over, rc):
    fn = lib.sd_sample if draw else lib.sd_truncate
    if not draw and "V" in over and over["V"]:
        over = dict(over, ld_out=over["V"])
    assert fn(*cut_args(draw, **over)) == rc


def test_cut_rows_refuse_their_own(lib):
    assert lib.sd_truncate(*cut_args(False, ld_out=99)) == -2
    assert lib.sd_truncate(*cut_args(False, probs=None)) == -1
    assert lib.sd_truncate(*cut_args(False, probs=(1 << 30) + 2)) == -4
    assert lib.sd_sample(*cut_args(True, u=None)) == -1
    assert lib.sd_sample(*cut_args(True, tokens=None)) == -1


def test_memory_that_may_not_be_shared(lib):
    """An output that is its input keeps the strides; lengths and rows that are read again stay."""
    assert lib.sd_rope(*rope_args(q_out=P, ld_qo=512)) == -2
    assert lib.sd_rope(*rope_args(k_out=P, hs_ko=128)) == -2
    assert lib.sd_kv_evict(*evict_args(new_lens=P, ctx=P)) == -2
    assert lib.sd_truncate(*cut_args(False, rows=4096, probs=4096)) == -2
    assert lib.sd_truncate(*cut_args(False, rows=4096, probs=4096 + 600 * 2 - 4)) == -2
    assert lib.sd_truncate(*cut_args(False, rows=4096, probs=4096 - 600 * 4 + 4)) == -2


@pytest.mark.parametrize("over", [
    dict(rot=0), dict(rot=7), dict(rot=514), dict(base=1.0), dict(base=math.inf), dict(kind=5),
    dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=2, factor=math.nan), dict(kind=4, factor=0.5),
    dict(kind=3, original_len=0.0), dict(kind=3, low=4.0), dict(kind=4, low=0.0)])
def test_table_refuses(lib, over):
    a = dict(rot=64, base=1e4, kind=0, factor=4.0, original_len=4096.0, low=1.0, high=4.0)
    a.update(over)
    turns, scale = (ctypes.c_uint64 * 256)(), ctypes.c_float(-1.0)
    assert lib.sd_rope_table(*a.values(), turns, ctypes.byref(scale)) == -2
    assert scale.value == -1.0 and not any(turns)
    assert lib.sd_rope_table(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, ctypes.byref(scale)) == -1


def frequencies(rot, base, kind, factor, original_len, low, high):
    """Radians a position of every pair, and the scale, as the definitions read."""
    out, scale = [], 1.0
    for i in range(rot // 2):
        b = base * factor ** (rot / max(1, rot - 2)) if kind == "ntk" else base
        f = b ** (-2 * i / rot)
        keep = 1.0
        if kind == "linear":
            keep = 0.0
        if kind == "bands":
            turns = original_len * f / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
        if kind == "yarn":
            pair = [rot * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))
                    for t in (high, low)]
            a, z = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
            keep = 1 - min(max((i - a) / max(z - a, 0.001), 0.0), 1.0)
            scale = 0.1 * math.log(factor) + 1
        out.append(f * keep + f / factor * (1 - keep))
    return out, scale


@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "bands", "yarn"])
@pytest.mark.parametrize("rot,base", [(2, 1e4), (40, 1e4), (64, 5e5), (128, 1e6)])
def test_table(kind, rot, base):
    sd.build()
    p = dict(factor=8.0, original_len=8192.0, low=1.0, high=32.0 if kind == "yarn" else 4.0)
    turns, scale = sd.sd_rope_table(rot, base=base, kind=kind, device="cpu", **p)
    want, want_scale = frequencies(rot, base, kind, **p)
    assert scale == pytest.approx(want_scale, rel=2.0 ** -23)
    for got, f in zip(turns.tolist(), want):
        # a power function and a handful of products in fp64: 2^-44 of it
        assert got / 2.0 ** 64 * 2 * math.pi == pytest.approx(f, rel=2.0 ** -44)


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pos, turns = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    for kw in (dict(), dict(q=q.float()), dict(q=q[0]), dict(q=q, k=q[:2]), dict(q=q, q_out=q[:, :2]),
               dict(q_out=q, k=q), dict(q=q, pairs="thirds"), dict(q=q)):
        with pytest.raises(sd.SDError):  # (the last: host memory that the GPU cannot address)
            sd.sd_rope(pos, turns, **kw)
    with pytest.raises(sd.SDError):
        sd.sd_rope(pos.long(), turns, q=q)
    with pytest.raises(sd.SDError):
        sd.sd_rope(pos, turns.int(), q=q)
    with pytest.raises(sd.SDError):
        sd.sd_rope_table(64, kind="other", device="cpu")
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    scale, w = torch.zeros(4, 2), torch.zeros(4, 2, 16)
    table, ctx, cu = (torch.zeros(*s, dtype=torch.int32) for s in ((2, 3), (2,), (3,)))
    good = dict(q=q, lse=torch.zeros(3, 4), k_cache=cache, k_scale=scale, block_table=table,
                ctx_lens=ctx, cu_q=cu, weights=w)
    for kw in (dict(lse=torch.zeros(3, 3)), dict(weights=w[:3]), dict(weights=w.double()),
               dict(before=w.half()), dict(live=ctx.long()), dict(q=q.float()), dict(cu_q=ctx),
               dict(k_scale=scale.double()), dict()):
        with pytest.raises(sd.SDError):
            sd.sd_kv_weights(**{**good, **kw})
    kept, lens = torch.zeros(2, 2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(k_cache=cache, v_cache=cache.clone(), k_scale=scale, v_scale=scale.clone(), weights=w,
                block_table=table, ctx_lens=ctx, kept=kept, new_lens=lens)
    for kw in (dict(kept=kept[0]), dict(kept=kept.long()), dict(kept=kept[:, :1]),
               dict(new_lens=lens[:1]), dict(weights=w.transpose(1, 2)), dict(to_table=table[:1]),
               dict(v_cache=cache[:2]), dict()):
        with pytest.raises(sd.SDError):
            sd.sd_kv_evict(**{**good, **kw})
    rows, f, i = torch.zeros(6, 10), torch.zeros(2), torch.zeros(2, 3, dtype=torch.int32)
    for kw in (dict(rows=rows.double()), dict(rows=rows[:5]), dict(top_p=f[:1]), dict(top_k=f),
               dict(min_p=f.double()), dict(temperature=f.half()), dict(kept=i.long()), dict()):
        a = dict(rows=rows, kept=i)
        a.update(kw)
        with pytest.raises(sd.SDError):
            sd.sd_truncate(a.pop("rows"), rows, **a)
        a.setdefault("tokens", i)
        with pytest.raises(sd.SDError):
            sd.sd_sample(kw.get("rows", rows), torch.zeros(2, 3), **{k: v for k, v in a.items()})
    with pytest.raises(sd.SDError):
        sd.sd_truncate(rows, rows[:, :9], i)
    with pytest.raises(sd.SDError):
        sd.sd_sample(rows, torch.zeros(6), i)
