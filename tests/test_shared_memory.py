"""Memory that the rotary, weight, eviction and cut-row calls may not share: refusals (no GPU), the check of
strided heads against sets of places, and, on a GPU, neighbours in one array that they do take."""

import os
import random
import shutil
import subprocess

import pytest
import torch

import verify_draft_prep_gb300 as sd
from conftest import ROOT
from test_step_ops_host import P, cut_args, evict_args, rope_args, weights_args

# (dummy addresses of arrays apart: no call below gets as far as using one)
FAR = {name: (i + 1) << 40 for i, name in enumerate("abcdefghijklmnop")}


@pytest.fixture(scope="module")
def lib():
    sd.build()
    return sd.load()


def test_evict(lib):
    apart = dict(k_cache=FAR["a"], v_cache=FAR["b"], k_scale=FAR["c"], v_scale=FAR["d"], weights=FAR["e"],
                 table=FAR["f"], ctx=FAR["g"], kept=FAR["h"], new_lens=FAR["i"])
    table, ctx, kept, lens = (apart[f] for f in ("table", "ctx", "kept", "new_lens"))
    # B = 2 requests of 4 pages, 2 heads, 8 places: 32, 8, 128 and 8 bytes
    for over in (dict(to=table, to_blocks=4), dict(to=table + 28, to_blocks=4), dict(to=table - 12, to_blocks=2),
                 dict(new_lens=ctx), dict(new_lens=ctx + 4), dict(kept=ctx - 124), dict(kept=table + 28),
                 dict(new_lens=table + 16), dict(kept=lens - 124), dict(new_lens=kept + 124),
                 dict(to=kept + 64, to_blocks=1), dict(to=lens - 4, to_blocks=1),
                 dict(v_cache=FAR["a"]), dict(v_scale=FAR["c"]), dict(v_cache=FAR["a"], v_scale=FAR["c"]),
                 dict(v_cache=FAR["a"], to=FAR["j"], to_blocks=1),
                 dict(v_scale=FAR["c"], to=FAR["j"], to_blocks=1)):
        assert lib.sd_kv_evict(*evict_args(**{**apart, **over})) == -2, over


def test_weights(lib):
    # 4 pages of 2 heads of 16 tokens: 512 bytes
    for before in (FAR["a"] + 4, FAR["a"] - 4, FAR["a"] + 508):
        assert lib.sd_kv_weights(*weights_args(weights=FAR["a"], before=before)) == -2


def test_rope(lib):
    apart = dict(q=FAR["a"], q_out=FAR["b"], k=FAR["c"], k_out=FAR["d"], ld_k=256, ld_ko=256)
    for over in (dict(q_out=FAR["c"]), dict(k_out=FAR["a"]), dict(k_out=FAR["b"]), dict(q_out=FAR["a"] + 128),
                 dict(k_out=FAR["c"] - 128), dict(q_out=FAR["c"] - 3 * 128), dict(k_out=FAR["b"] + 512 * 2),
                 dict(ld_qo=0), dict(hs_qo=0), dict(hs_ko=56), dict(ld_ko=64, hs_ko=64),
                 dict(q_out=FAR["a"], ld_q=0, ld_qo=0), dict(q_out=FAR["a"], hs_q=0, hs_qo=0)):
        assert lib.sd_rope(*rope_args(**{**apart, **over})) == -2, over


def test_cut_rows(lib):
    apart = dict(rows=FAR["a"], temperature=FAR["b"], top_k=FAR["c"], top_p=FAR["d"], min_p=FAR["e"],
                 kept=FAR["f"])
    # 6 rows of 100 logits, 2 requests, 6 numbers: 1200, 8 and 24 bytes
    for f in ("temperature", "top_k", "top_p", "min_p", "rows"):
        at = apart[f]
        for out in ("probs", "kept"):
            for place in (at, at + 4):
                assert lib.sd_truncate(*cut_args(False, **{**apart, out: place})) == -2, (f, out)
        for out in ("tokens", "prob", "kept"):
            own = dict(u=FAR["g"], tokens=FAR["h"], prob=FAR["i"])
            for place in (at, at - 20, at + 4):
                assert lib.sd_sample(*cut_args(True, **{**apart, **own, out: place})) == -2, (f, out)
    assert lib.sd_truncate(*cut_args(False, **apart, probs=FAR["f"] - 2396)) == -2
    own = dict(u=FAR["g"], tokens=FAR["h"], prob=FAR["i"])
    for over in (dict(tokens=FAR["i"]), dict(kept=FAR["h"] + 20), dict(prob=FAR["f"] - 20), dict(tokens=FAR["g"]),
                 dict(kept=FAR["g"] + 4), dict(prob=FAR["g"] + 4)):
        assert lib.sd_sample(*cut_args(True, **{**apart, **own, **over})) == -2, over


HARNESS = """
#include <cstdio>
#include "sd_overlap.cuh"
int main() {
  long a, lda, hsa, b, ldb, hsb;
  int Ha, Hb, n, D;
  while (scanf("%ld %ld %ld %d %ld %ld %ld %d %d %d", &a, &lda, &hsa, &Ha, &b, &ldb, &hsb, &Hb, &n, &D) == 10) {
    const HeadRows x{(void*)(4096 + 2 * a), lda, hsa, Ha}, y{(void*)(4096 + 2 * b), ldb, hsb, Hb};
    printf("%d %d\\n", (int)heads_share(x, y, n, D), (int)heads_overlap(x, n, D));
  }
}
"""


def test_strided_heads_against_sets(tmp_path):
    """Every value's place, of small arrays with all kinds of strides."""
    if not shutil.which("g++"):
        pytest.skip("no g++")
    (tmp_path / "h.cpp").write_text(HARNESS)
    exe = tmp_path / "h"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "verify_draft_prep_gb300", "csrc"),
                    str(tmp_path / "h.cpp"), "-o", str(exe)], check=True)
    rng = random.Random(0)
    cases = []
    for _ in range(4000):
        D = rng.choice([8, 16, 24])
        n, Ha, Hb = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 4)
        ld, hs = 8 * rng.randint(0, 24), 8 * rng.randint(0, 24)
        other = rng.random() < 0.1
        cases.append((0, ld, hs, Ha, 8 * rng.randint(-30, 60), ld + 8 * other * rng.randint(0, 2),
                      hs + 8 * other * rng.randint(0, 2), Hb, n, D))
    got = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True,
                         capture_output=True, check=True).stdout.split()
    alike = shared = lying = 0
    for c, (s, o) in zip(cases, zip(got[::2], got[1::2])):
        a, lda, hsa, Ha, b, ldb, hsb, Hb, n, D = c
        places = lambda p, ld, hs, H: [p + i * ld + h * hs + d for i in range(n) for h in range(H)  # noqa: E731
                                       for d in range(D)]
        x, y = places(a, lda, hsa, Ha), places(b, ldb, hsb, Hb)
        assert bool(int(o)) == (len(set(x)) < len(x)), c
        lying += int(o)
        want = bool(set(x) & set(y))
        if (n > 1 and lda != ldb) or (Ha > 1 and Hb > 1 and hsa != hsb):
            assert bool(int(s)) == (a == b), c
        else:
            # (one array's head stride serves for both where the other has one head)
            assert bool(int(s)) == want, c
            alike += 1
            shared += want
    assert alike > 2000 and 400 < shared < alike - 400 and lying > 200


@pytest.mark.gpu
def test_neighbours_in_one_array():
    """Outputs side by side, and a number's place taken by its probability."""
    dev, i32 = "cuda", dict(dtype=torch.int32, device="cuda")
    torch.manual_seed(0)
    n, Hq, Hk, D = 5, 4, 2, 64
    turns, _ = sd.sd_rope_table(D, device=dev)
    pos = torch.arange(n, **i32) * 9
    q, k = torch.randn(n, Hq, D, device=dev).bfloat16(), torch.randn(n, Hk, D, device=dev).bfloat16()
    want = [torch.empty_like(q), torch.empty_like(k)]
    sd.sd_rope(pos, turns, q=q, k=k, q_out=want[0], k_out=want[1])
    both = torch.empty(n, Hq + Hk, D, dtype=torch.bfloat16, device=dev)
    for out in (both, both.new_empty(Hq + Hk, n, D).transpose(0, 1), both.new_empty(n, Hq + Hk, 3, D)[:, :, 1]):
        sd.sd_rope(pos, turns, q=q, k=k, q_out=out[:, :Hq], k_out=out[:, Hq:])
        assert torch.equal(out[:, :Hq], want[0]) and torch.equal(out[:, Hq:], want[1])
        out[:, :Hq], out[:, Hq:] = q, k  # in place, and into the neighbours of what is read
        sd.sd_rope(pos, turns, q=out[:, :Hq], k=out[:, Hq:])
        assert torch.equal(out[:, :Hq], want[0]) and torch.equal(out[:, Hq:], want[1])
    rows = torch.cat([torch.randn(6, 3000, device=dev), torch.randn(6, 3000, device=dev) * 1e-6]).bfloat16()
    u = torch.rand(12, 1, device=dev)
    tokens, prob = torch.empty(12, 1, **i32), torch.empty(12, 1, device=dev)
    sd.sd_sample(rows, u, tokens, prob=prob)
    again = torch.empty_like(tokens)
    sd.sd_sample(rows, u, again, prob=u)
    assert torch.equal(tokens, again) and torch.equal(u, prob)
    # one cache as K and V, into fresh pages
    cache, scale = torch.randint(0, 100, (6, 16, 1, 16), dtype=torch.uint8, device=dev), torch.ones(6, 1, device=dev)
    numbers = torch.empty(2 + 20, **i32)
    lens, kept = numbers[:1], numbers[2:].view(1, 1, 20)
    w = torch.rand(6, 1, 16, device=dev)
    sd.sd_kv_evict(cache, cache, scale, scale, w, torch.tensor([[0, 1, 2]], **i32), torch.tensor([40], **i32),
                   kept, lens, to_table=torch.tensor([[4, 3]], **i32))
    t = kept[0, 0].long()
    assert int(lens) == 20 and torch.all(t[1:] > t[:-1])
    moved = cache[torch.tensor([4, 3], device=dev)].view(32, 16)[:20]
    assert torch.equal(moved, cache[t // 16, t % 16, 0])
