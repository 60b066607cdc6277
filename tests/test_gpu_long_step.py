"""The rotary, weight, eviction and cut-row calls together with the cache and the verification they
stand beside: steps of a request whose cache is held to a budget."""

import pytest
import torch

import kvref
import stepref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu

DEV = "cuda"
B, K, H, G, D, BS, V, BUDGET, SINK, RECENT = 3, 3, 2, 4, 64, 16, 600, 96, 4, 16


class Loop:
    """Requests with a cache that is cut to BUDGET tokens after every step. Positions of the text go on;
    places in the cache do not."""

    def __init__(self, seed=0):
        g = self.gen = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.i32 = i32 = dict(dtype=torch.int32, device=DEV)
        self.text = torch.tensor([150, 40, 95], **i32)  # tokens so far
        per = -(-(200 + K + 1) // BS)
        nb = 2 * B * per
        self.tables = [p.contiguous() for p in torch.randperm(nb, generator=g, device=DEV).int().view(2, B, per)]
        shape = (nb, BS, H, D)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=DEV).view(kvref.E4M3) for _ in range(2))
        self.ks, self.vs = (torch.zeros(nb, H, device=DEV) for _ in range(2))
        self.weights = torch.zeros(nb, H, BS, device=DEV)
        self.turns, self.scale = sd.sd_rope_table(D, base=5e5, kind="yarn", factor=4.0, original_len=128,
                                                  device=DEV)
        self.err = torch.zeros(1, **i32)
        self.held = self.text.clone()  # tokens in the cache
        self.head = self.randn(H * G * D, V) * 0.05
        self.setting = dict(temperature=torch.tensor([0.7, 0.0, 1.1], device=DEV),
                            top_k=torch.tensor([40, 0, 0], **i32),
                            top_p=torch.tensor([0.9, 1.0, 0.95], device=DEV),
                            min_p=torch.tensor([0.0, 0.0, 0.01], device=DEV))
        n = int(self.text.sum())
        r = torch.arange(B, device=DEV).repeat_interleave(self.text.long())
        pos = torch.cat([torch.arange(int(t), device=DEV) for t in self.text]).int()
        qkv = self.randn(n, H * (G + 2), D)
        self.store(qkv, r, pos, pos)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=DEV, dtype=torch.bfloat16)

    def store(self, qkv, r, pos, place):
        """Turns the queries and keys of a projection in place and writes K and V to their places."""
        q, k, v = qkv[:, :H * G], qkv[:, H * G:H * (G + 1)], qkv[:, H * (G + 1):]
        sd.sd_rope(pos, self.turns, q=q, k=k, scale=self.scale)
        slots = self.tables[0][r, place.long() // BS] * BS + place % BS
        sd.sd_kv_write(k, v, slots.int().contiguous(), self.k, self.v, self.ks, self.vs, err=self.err)
        return q

    def step(self, qkv, draft_rows, u):
        """K+1 verify slots of every request; returns what the step makes."""
        i32, n = self.i32, B * (K + 1)
        r = torch.arange(B, device=DEV).repeat_interleave(K + 1)
        j = torch.arange(K + 1, **i32).repeat(B)
        q = self.store(qkv, r, (self.text[r] + j), self.held[r] + j)
        ctx = self.held + K + 1
        cu = torch.arange(0, n + 1, K + 1, **i32)
        out, lse = torch.empty(n, H * G, D, dtype=torch.bfloat16, device=DEV), torch.empty(n, H * G, device=DEV)
        sd.sd_kv_attend(q, self.k, self.v, self.ks, self.vs, self.tables[0], ctx, cu, out, lse=lse,
                        max_q=K + 1, err=self.err)
        logits = out.view(n, -1) @ self.head
        # drafts drawn from the drafter's cut rows, and checked against the target's
        drafts, tokens, acc = torch.empty(B, K, **i32), torch.empty(B, K + 1, **i32), torch.empty(B, **i32)
        p, d = torch.empty(n, V, device=DEV), torch.empty(B * K, V, device=DEV)
        kept = torch.empty(B, K + 1, **i32)
        sd.sd_truncate(logits, p, kept, err=self.err, **self.setting)
        sd.sd_truncate(draft_rows, d, torch.empty(B, K, **i32), err=self.err, **self.setting)
        sd.sd_sample(draft_rows, u, drafts, err=self.err, **self.setting)
        sd.sd_verify(p, d, drafts, tokens, acc, seed=7, err=self.err)
        # the accepted slots' weights, and the cache cut into the other pages
        sd.sd_kv_weights(q, lse, self.k, self.ks, self.tables[0], ctx, cu, self.weights,
                         before=self.weights, live=acc + 1, max_q=K + 1, decay=0.9, err=self.err)
        now = self.held + acc + 1
        rows, lens = torch.empty(B, H, BUDGET, **i32), torch.empty(B, **i32)
        sd.sd_kv_evict(self.k, self.v, self.ks, self.vs, self.weights, self.tables[0], now, rows, lens,
                       to_table=self.tables[1], sink=SINK, recent=RECENT, err=self.err)
        return dict(q=q, ctx=ctx, lse=lse, out=out, logits=logits, p=p, d=d, drafts=drafts, tokens=tokens,
                    acc=acc, kept_rows=rows, lens=lens, now=now)

    def go_on(self, got):
        self.text = self.text + got["acc"] + 1
        self.held = got["lens"]
        self.tables.reverse()


def test_steps():
    loop = Loop()
    assert int(loop.err) == 0
    for step in range(3):
        qkv = loop.randn(B * (K + 1), H * (G + 2), D)
        draft_rows = loop.randn(B * K, V)
        u = torch.rand(B, K, generator=loop.gen, device=DEV)
        unturned = qkv[:, :H * (G + 1)].clone()
        pos = (loop.text[:, None] + torch.arange(K + 1, **loop.i32)[None]).view(-1)
        was = loop.weights.clone()
        old_table = loop.tables[0]
        got = loop.step(qkv, draft_rows, u)
        torch.cuda.synchronize()
        assert int(loop.err) == 0
        # the turned queries and keys stand in the projection
        want, tol = stepref.rope_ref(unturned.double().cpu(), pos.tolist(),
                                     [t % stepref.TWO64 for t in loop.turns.tolist()], "halves", loop.scale,
                                     False)
        assert torch.all((qkv[:, :H * (G + 1)].double().cpu() - want).abs() <= tol)
        for r in range(B):
            T, m = int(got["ctx"][r]), K + 1
            sl = slice(r * m, (r + 1) * m)
            k = kvref.held(loop.k, loop.ks, old_table[r], T)
            v = kvref.held(loop.v, loop.vs, old_table[r], T)
            o, _, tol, _ = kvref.attend_ref(got["q"][sl].double(), k, v, D ** -0.5, True)
            assert torch.all((got["out"][sl].double() - o).abs() <= tol)
            # weights: what the accepted slots gave, on what there was
            t = torch.arange(T, device=DEV)
            page = old_table[r].long()[t // BS]
            w, tol = stepref.weights_ref(got["q"][sl].double(), got["lse"][sl].double(), k, D ** -0.5, True,
                                         int(got["acc"][r]) + 1, 0.9, was[page, :, t % BS].double())
            assert torch.all((loop.weights[page, :, t % BS].double() - w).abs() <= tol)
            # the cache that goes on: the first, the last and the heaviest tokens, each head its own
            n, keep = int(got["now"][r]), int(got["lens"][r])
            assert keep == min(n, BUDGET)
            for h in range(H):
                rows = got["kept_rows"][r, h]
                assert torch.all(rows[keep:] == -1) and torch.all(rows[1:keep] > rows[:keep - 1])
                if n > BUDGET:
                    mine = loop.weights[page, h, t % BS][:n]
                    stays = set(rows[:keep].tolist())
                    assert set(range(SINK)) <= stays and set(range(n - RECENT, n)) <= stays
                    mid = [x for x in range(SINK, n - RECENT)]
                    least = min(float(mine[x]) for x in mid if x in stays)
                    assert all(float(mine[x]) <= least for x in mid if x not in stays)
                kk = kvref.held(loop.k, loop.ks, loop.tables[1][r], keep)[:, h]
                scale = loop.ks[loop.tables[1][r, :-(-keep // BS)].long(), h].repeat_interleave(BS)[:keep]
                assert torch.all((kk - k[rows[:keep].long(), h]).abs() <= scale.double()[:, None] * 2.0 ** -10)
        # verification of cut rows: an answer is always among the kept entries of its target row
        live = got["tokens"] >= 0
        at = got["p"].view(B, K + 1, V).gather(2, got["tokens"].clamp(min=0).long()[..., None])[..., 0]
        assert torch.all(at[live] > 0)
        assert torch.all(got["d"].view(B, K, V).gather(2, got["drafts"].long()[..., None]) > 0)
        greedy = got["logits"].view(B, K + 1, V)[1].argmax(-1)
        a = int(got["acc"][1])
        assert got["tokens"][1, :a + 1].tolist() == greedy[:a + 1].tolist()
        loop.go_on(got)
        assert int(loop.held.max()) <= BUDGET


def test_captured_step_equals_the_eager_one():
    """The whole step in one graph, replayed on the state that the eager one began with."""
    loops = [Loop(seed=5), Loop(seed=5)]
    ins = [(lp.randn(B * (K + 1), H * (G + 2), D), lp.randn(B * K, V),
            torch.rand(B, K, generator=lp.gen, device=DEV)) for lp in loops]
    eager = loops[0].step(*ins[0])
    lp = loops[1]
    state = [t.clone() for t in (lp.k.view(torch.uint8), lp.v.view(torch.uint8), lp.ks, lp.vs, lp.weights, ins[1][0])]
    lp.step(*ins[1])  # what a first call sets up is set up before the capture

    def back():
        for t, s in zip((lp.k.view(torch.uint8), lp.v.view(torch.uint8), lp.ks, lp.vs, lp.weights, ins[1][0]), state):
            t.copy_(s)
    back()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = lp.step(*ins[1])
    for _ in range(2):
        back()
        g.replay()
        torch.cuda.synchronize()
        for f in ("q", "out", "lse", "logits", "p", "d", "drafts", "tokens", "acc", "kept_rows", "lens"):
            assert torch.equal(got[f], eager[f]), f
        assert torch.equal(lp.weights, loops[0].weights)
        assert torch.equal(lp.k.view(torch.uint8), loops[0].k.view(torch.uint8))
    assert int(lp.err) == 0
