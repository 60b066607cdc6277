"""Refusals of the cache and answer calls: the host's checks answer before any device work, in
the C library and in the Python binding."""

import pytest
import torch

import verify_draft_prep_gb300 as sd

P = 256  # a well aligned dummy address; no call below gets as far as using it


@pytest.fixture(scope="module")
def lib():
    sd.build()
    return sd.load()


CACHE = dict(k_cache=P, v_cache=P, st_block=2048, st_tok=128, st_head=64, k_scale=P, v_scale=P,
             num_blocks=4, block_size=16)


def write_args(**over):
    a = dict(n=3, Hkv=2, D=64, k=P, ld_k=128, hs_k=64, v=P, ld_v=128, hs_v=64, slots=P, **CACHE,
             err=None, stream=None)
    a.update(over)
    return list(a.values())


def read_args(**over):
    a = dict(B=2, n=3, Hkv=2, D=64, **CACHE, table=P, max_blocks=4, cu=P, first=None, k_out=P,
             v_out=P, ld=128, hs=64, err=None, stream=None)
    a.update(over)
    return list(a.values())


def attend_args(**over):
    a = dict(B=2, n=3, max_q=2, Hq=4, Hkv=2, D=64, q=P, ld_q=256, hs_q=64, **CACHE, table=P,
             max_blocks=4, ctx=P, cu=P, sm_scale=0.125, causal=1, out=P, ld_out=256, hs_out=64,
             lse=None, ws=P, ws_bytes=1 << 40, err=None, stream=None)
    a.update(over)
    return list(a.values())


def logprob_args(**over):
    a = dict(B=2, J=3, V=100, dtype=1, rows=P, ld=100, tokens=P, temperature=None, n_top=5,
             logprob=P, entropy=None, rank=None, top_ids=P, top_lp=P, err=None, stream=None)
    a.update(over)
    return list(a.values())


BAD_CACHE = [(dict(D=8), -2), (dict(D=72), -2), (dict(D=144), -2), (dict(Hkv=0), -2),
             (dict(block_size=4), -2), (dict(block_size=24), -2), (dict(block_size=256), -2),
             (dict(num_blocks=-1), -2), (dict(num_blocks=1 << 28, block_size=16), -2),
             (dict(st_block=0), -2), (dict(st_tok=-128), -2), (dict(st_head=24), -4),
             (dict(st_tok=130), -4), (dict(k_cache=None), -1), (dict(v_scale=None), -1),
             (dict(k_cache=P + 8), -4)]


@pytest.mark.parametrize("over,rc", BAD_CACHE + [
    (dict(n=-1), -2), (dict(ld_k=-8), -2), (dict(ld_k=129), -4), (dict(hs_v=60), -4),
    (dict(k=None), -1), (dict(slots=None), -1), (dict(v=P + 2), -4), (dict(n=0), 0)])
def test_write_refuses(lib, over, rc):
    assert lib.sd_kv_write(*write_args(**over)) == rc


@pytest.mark.parametrize("over,rc", BAD_CACHE + [
    (dict(B=-1), -2), (dict(n=-1), -2), (dict(max_blocks=-1), -2), (dict(table=None), -1),
    (dict(cu=None), -1), (dict(k_out=None), -1), (dict(v_out=P + 4), -4), (dict(ld=100), -4),
    (dict(B=0), 0), (dict(n=0), 0)])
def test_read_refuses(lib, over, rc):
    assert lib.sd_kv_read(*read_args(**over)) == rc


@pytest.mark.parametrize("over,rc", [(o, rc) for o, rc in BAD_CACHE] + [
    (dict(B=-1), -2), (dict(n=-1), -2), (dict(max_q=0), -2), (dict(Hq=5), -2), (dict(Hq=0), -2),
    (dict(sm_scale=0.0), -2), (dict(sm_scale=-1.0), -2), (dict(sm_scale=float("nan")), -2),
    (dict(sm_scale=float("inf")), -2), (dict(n=1 << 30), -2), (dict(q=None), -1),
    (dict(ctx=None), -1), (dict(cu=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(table=None), -1), (dict(q=P + 8), -4), (dict(ws=P + 8), -4), (dict(ld_q=260), -4),
    (dict(hs_out=68), -4), (dict(B=0), 0), (dict(n=0), 0)])
def test_attend_refuses(lib, over, rc):
    assert lib.sd_kv_attend(*attend_args(**over)) == rc


def test_attend_workspace(lib):
    need = lib.sd_kv_attend_workspace_bytes(64)
    assert lib.sd_kv_attend_workspace_bytes(0) == lib.sd_kv_attend_workspace_bytes(136) == 0
    if need:
        assert lib.sd_kv_attend(*attend_args(ws_bytes=need - 1)) == -2


@pytest.mark.parametrize("over,rc", [
    (dict(dtype=2), -3), (dict(B=-1), -2), (dict(J=0), -2), (dict(V=0), -2), (dict(ld=99), -2),
    (dict(V=33554433, ld=33554433), -2), (dict(n_top=33), -2), (dict(n_top=-1), -2),
    (dict(V=4, n_top=5), -2), (dict(B=1 << 28), -2), (dict(rows=None), -1), (dict(tokens=None), -1),
    (dict(logprob=None), -1), (dict(top_ids=None), -1), (dict(top_lp=None), -1),
    (dict(rows=P + 1), -4), (dict(dtype=0, rows=P + 2), -4), (dict(B=0), 0)])
def test_logprobs_refuses(lib, over, rc):
    assert lib.sd_token_logprobs(*logprob_args(**over)) == rc


def _cache(nb=4, bs=16, H=2, D=64):
    c = torch.zeros(2, nb, bs, H, D, dtype=torch.uint8)
    return [c[0], c[1], torch.zeros(nb, H), torch.zeros(nb, H)]


def test_binding_refuses_wrong_tensors():
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    c = _cache()
    for bad in ([c[0].float(), *c[1:]], [c[0], c[1][:3], *c[2:]], [c[0], c[1], c[2].double(), c[3]],
                [c[0].transpose(2, 3), c[1].transpose(2, 3), *c[2:]]):
        with pytest.raises(sd.SDError):
            sd.sd_kv_write(k, k, slots, *bad)
    for kw in (dict(k=k.float()), dict(k=k[:2]), dict(k=k[:, :1]), dict(slots=slots.long()),
               dict(slots=slots[:2])):
        a = dict(k=k, slots=slots)
        a.update(kw)
        with pytest.raises(sd.SDError):
            sd.sd_kv_write(a["k"], k, a["slots"], *c)
    with pytest.raises(sd.SDError):  # host memory that the GPU cannot address
        sd.sd_kv_write(k, k, slots, *c)
    with pytest.raises(sd.SDError):
        sd.sd_token_logprobs(torch.zeros(6, 10).half(), torch.zeros(2, 3, dtype=torch.int32),
                             torch.zeros(2, 3))
    with pytest.raises(sd.SDError):
        sd.sd_token_logprobs(torch.zeros(6, 10), torch.zeros(2, 3, dtype=torch.int32),
                             torch.zeros(2, 3), top_ids=torch.zeros(2, 3, 2, dtype=torch.int32))
