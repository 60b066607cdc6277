"""One speculative decoding step around the paged 8-bit cache, with the framework's calls only.

    python examples/cached_step.py            # 64 requests, K = 5, contexts of 512..8192 tokens

The target's K and V of the K+1 verify slots enter the cache, the slots attend to their contexts,
the (here: random) head gives logits, the drafts are verified, the answer gets its log
probabilities, the drafter's batch is rebuilt, and its tokens enter the drafter's own cache and
attend to it. The model parts between the calls are random matrices: the point is which arrays go
from call to call, all of them on the device, without a synchronisation in between. At the end the
step's tokens are read back from the target's cache, as a move to another precision would.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import verify_draft_prep_gb300 as sd  # noqa: E402

BLOCK = 16


class Cache:
    """A zeroed paged cache in e4m3 with its scales."""

    def __init__(self, pages, heads, dim, device):
        shape = (pages, BLOCK, heads, dim)
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.k_scale = torch.zeros(pages, heads, device=device)
        self.v_scale = torch.zeros(pages, heads, device=device)

    def all(self):
        return self.k, self.v, self.k_scale, self.v_scale


class Step:
    """What a serving loop keeps between steps, and one step over it."""

    def __init__(self, B=64, K=5, V=32000, heads=8, groups=8, dim=64, H=512, ctx=(512, 8192),
                 device="cuda", seed=0):
        g = self.gen = torch.Generator(device=device)
        g.manual_seed(seed)
        self.B, self.K, self.V, self.heads, self.groups, self.dim, self.H = (B, K, V, heads, groups,
                                                                             dim, H)
        self.device = device
        i32 = self.i32 = dict(dtype=torch.int32, device=device)
        self.pos0 = torch.randint(ctx[0], ctx[1] + 1, (B,), generator=g, device=device).int()
        need = (self.pos0 + 2 * K) // BLOCK + 1
        pages = int(need.sum())
        perm = torch.randperm(pages, generator=g, device=device).int()
        self.table = torch.full((B, int(need.max())), -1, **i32)
        col = torch.arange(self.table.shape[1], device=device)
        self.table[col[None] < need[:, None]] = perm
        self.target_cache = Cache(pages, heads, dim, device)
        self.draft_cache = Cache(pages, heads, dim, device)
        # the contexts so far, as a prompt would have written them: the target's positions 0..pos0-1 (its
        # K+1 slots begin at pos0), the drafter's 0..pos0 (its rebuilt slots begin at pos0+1)
        for cache, n in ((self.target_cache, self.pos0), (self.draft_cache, self.pos0 + 1)):
            r = torch.arange(B, device=device).repeat_interleave(n.long())
            start = torch.cumsum(n, 0) - n
            p = torch.arange(r.numel(), device=device) - start[r]
            slots = self.table[r, p // BLOCK] * BLOCK + (p % BLOCK).int()
            kv = self.randn(r.numel(), 2, heads, dim)
            sd.sd_kv_write(kv[:, 0], kv[:, 1], slots.int(), *cache.all())
        W = self.W = 2 * K
        n = B * (K + 1)
        self.cu_verify = torch.arange(0, n + 1, K + 1, **i32)
        self.cu_draft = torch.arange(0, B * W + 1, W, **i32)
        self.head = self.randn(heads * groups * dim, V) * 0.02
        self.h_shared = self.randn(H)
        self.err = torch.zeros(1, **i32)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.device, dtype=torch.bfloat16)

    def attend(self, cache, q, ctx, cu, max_q):
        out = torch.empty_like(q)
        sd.sd_kv_attend(q, *cache.all(), self.table, ctx, cu, out, max_q=max_q, err=self.err)
        return out

    def read_back(self, cache, first, count):
        """Tokens first[r] .. first[r] + count - 1 of every request as the cache holds them, bf16."""
        cu = torch.arange(0, self.B * count + 1, count, **self.i32)
        k, v = (torch.empty(self.B * count, self.heads, self.dim, dtype=torch.bfloat16,
                            device=self.device) for _ in range(2))
        sd.sd_kv_read(*cache.all(), self.table, cu, k, v, first_pos=first, err=self.err)
        return k, v

    def run(self, drafts, draft_rows, seed=0, top=5):
        """drafts [B, K] and the drafter's logits [B*K, V] they came from. Returns what the step
        answers and the drafter's next batch."""
        B, K, V, i32 = self.B, self.K, self.V, self.i32
        n = B * (K + 1)
        # the target's pass over the K+1 verify slots of every request
        j = torch.arange(K + 1, **i32)
        pos = self.pos0[:, None] + j[None]
        slots = (torch.gather(self.table, 1, (pos // BLOCK).long()) * BLOCK + pos % BLOCK).view(-1)
        qkv = self.randn(n, (self.groups + 2) * self.heads, self.dim)
        hq = self.groups * self.heads
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + self.heads], qkv[:, hq + self.heads:]
        sd.sd_kv_write(k, v, slots.int(), *self.target_cache.all(), err=self.err)
        attended = self.attend(self.target_cache, q, self.pos0 + K + 1, self.cu_verify, K + 1)
        logits = attended.view(n, -1) @ self.head
        # verification, and what the answer says about itself
        out_tokens, accepted = torch.empty(B, K + 1, **i32), torch.empty(B, **i32)
        sd.sd_verify(logits, draft_rows, drafts, out_tokens, accepted, seed=seed, err=self.err)
        f32 = dict(device=self.device)
        said = dict(logprob=torch.empty(B, K + 1, **f32), entropy=torch.empty(B, K + 1, **f32),
                    rank=torch.empty(B, K + 1, **i32), top_ids=torch.empty(B, K + 1, top, **i32),
                    top_logprobs=torch.empty(B, K + 1, top, **f32))
        sd.sd_token_logprobs(logits, out_tokens, **said, err=self.err)
        # the drafter's next batch, in fixed rows of 2K slots
        size, hidden = B * self.W, self.randn(n, self.H)
        ids, where, slot, hmap = (torch.empty(size, **i32) for _ in range(4))
        masked, rejected = (torch.empty(size, dtype=torch.uint8, device=self.device)
                            for _ in range(2))
        scatter, new_idx = torch.empty(n, **i32), torch.empty(B, K, **i32)
        rows = torch.empty(size, self.H, dtype=torch.bfloat16, device=self.device)
        sd.sd_pdraft_prepare_padded(out_tokens, accepted, self.pos0, self.table, BLOCK, V, ids,
                                    where, slot, hmap, masked, rejected, scatter, new_idx, hidden,
                                    self.h_shared, rows, err=self.err)
        # its tokens enter the drafter's cache (rejected leftovers have slot -1 and write nothing)
        # and attend to it: W query slots a request, of which the last K - a_r are leftovers
        dkv = self.randn(size, 2, self.heads, self.dim)
        sd.sd_kv_write(dkv[:, 0], dkv[:, 1], slot, *self.draft_cache.all(), err=self.err)
        dq = self.randn(size, hq, self.dim)
        drafted = self.attend(self.draft_cache, dq, self.pos0 + 1 + self.W, self.cu_draft, self.W)
        return dict(out_tokens=out_tokens, accepted=accepted, logits=logits, attended=attended,
                    q=q, k=k, v=v, slots=slots, draft_slots=slot, draft_q=dq, drafted=drafted, **said)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--drafts", type=int, default=5)
    a = ap.parse_args()
    step = Step(B=a.requests, K=a.drafts)
    rows = step.randn(a.requests * a.drafts, step.V)
    drafts = torch.empty(a.requests, a.drafts, **step.i32)
    sd.sd_draft_sample(rows, drafts, seed=1, err=step.err)
    r = step.run(drafts, rows)
    k, _ = step.read_back(step.target_cache, step.pos0, step.K + 1)
    torch.cuda.synchronize()
    if int(step.err):
        raise SystemExit(f"data errors: {int(step.err):#x}")
    live = r["out_tokens"] >= 0
    print(f"accepted {r['accepted'].float().mean():.2f} of {a.drafts} drafts; answer of "
          f"{int(live.sum())} tokens, mean log probability {float(r['logprob'][live].mean()):.3f}, "
          f"mean entropy {float(r['entropy'][live].mean()):.3f}; K in the cache is "
          f"{float((k.float() - r['k'].float()).norm() / r['k'].float().norm()):.4f} off")


if __name__ == "__main__":
    main()
