"""Cases of the operators around a step's cache and its draws: sd_rope (rotary positions of queries
and keys), sd_kv_weights (the attention weight that each cached token gets), sd_kv_evict (a cache cut
to a budget by those weights), sd_truncate and sd_sample (top-k, top-p, min-p), each beside a plain
form in elementary torch operations.

Lengths, positions and tables stay on the device in every call; the host knows the sizes of the
arrays. The cache is the paged one in e4m3 with an fp32 scale for each page and KV head.

Sizes are those of the framework's workloads (batches of 1, 64, 256 and 1024 requests, 4 to 8
drafts, contexts of 37, 512..8192, 1000..16000 and 32000 tokens, pages of 16 tokens, vocabularies of
1024 and 201088 entries) with generic head layouts.

A case's lengths follow from the case alone; its values follow from the seed.
"""

import math
import random

import torch

own = False  # False: the plain forms; True: the framework's operators

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step's K+1 verify slots of every request (b64's batch), Q and K of one projection
        dict(name="rope-b64", op="rope", n=384, Hq=64, Hk=8, D=64, rot=64, pairs="halves",
             kind="plain", hi=8192, inverse=False),
        # two prompts of 8192 tokens, frequencies stretched for a context eight times as long
        dict(name="rope-prompt", op="rope", n=16384, Hq=32, Hk=8, D=128, rot=128, pairs="halves",
             kind="yarn", hi=131072, inverse=False),
        # the gradient of a prompt's queries and keys, half of each head rotated, neighbours paired
        dict(name="rope-back", op="rope", n=8192, Hq=32, Hk=8, D=128, rot=64, pairs="neighbours",
             kind="bands", hi=16000, inverse=True),
        # the weights that a single token gives to a long context; latency counts
        dict(name="weights-one", op="weights", B=1, n_q=1, ragged=False, Hq=32, Hkv=8, D=128, bs=16,
             lo=32000, hi=32000),
        # those of the target's verify pass over K+1 slots of b64, the accepted ones counted
        dict(name="weights-b64", op="weights", B=64, n_q=6, ragged=True, Hq=64, Hkv=8, D=64, bs=16,
             lo=512, hi=8192),
        # a prompt of 8192 tokens, causal
        dict(name="weights-prompt", op="weights", B=1, n_q=8192, ragged=False, Hq=32, Hkv=8, D=128,
             bs=16, lo=0, hi=0),
        # one long request cut in half
        dict(name="evict-one", op="evict", B=1, Hkv=8, D=128, bs=16, lo=32000, hi=32000,
             budget=16000, sink=4, recent=1024),
        # a batch held to 2048 tokens a request; some are shorter
        dict(name="evict-b64", op="evict", B=64, Hkv=8, D=64, bs=16, lo=512, hi=8192, budget=2048,
             sink=4, recent=256),
        # the verify rows of b64, probabilities, cut for a lossless check against the cut rows
        dict(name="truncate-b64", op="truncate", B=64, J=6, V=201088, kind="probs"),
        # the verify rows of b256mix's batch as logits, each request with settings of its own
        dict(name="truncate-b256", op="truncate", B=256, J=8, V=201088, kind="logits"),
        # one row of a small vocabulary; latency counts
        dict(name="sample-small", op="sample", B=1, J=1, V=1024, kind="logits"),
        # one token for each of 1024 requests
        dict(name="sample-b1024", op="sample", B=1024, J=1, V=201088, kind="logits"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "weights", "weights", "evict", "truncate", "sample"])
    if op in ("truncate", "sample"):
        V = _log_int(rng, 7, 201088)
        rows = _log_int(rng, 1, max(1, min(9216, int(2e8) // V)))
        J = rng.randint(1, min(17, rows))
        return dict(op=op, B=max(1, rows // J), J=J, V=V, kind=rng.choice(["probs", "logits"]))
    D = rng.choice([32, 64, 64, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
        n = _log_int(rng, 1, max(1, min(16384, 80_000_000 // ((Hq + Hkv) * D))))
        return dict(op=op, n=n, Hq=Hq, Hk=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16]),
                    pairs=rng.choice(["halves", "neighbours"]),
                    kind=rng.choice(["plain", "linear", "ntk", "bands", "yarn"]),
                    hi=_log_int(rng, 16, 1000000), inverse=rng.random() < 0.3)
    bs = rng.choice([8, 16, 16, 32, 64, 128])
    hi = _log_int(rng, 16, 32000)
    lo = rng.randint(0, hi)
    tokens = 60_000_000 // (Hkv * D)
    B = _log_int(rng, 1, max(1, min(256, tokens // (hi + 1))))
    if op == "evict":
        budget = _log_int(rng, 8, max(9, hi))
        sink = rng.randint(0, min(8, budget // 2))
        return dict(op=op, B=B, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi, budget=budget, sink=sink,
                    recent=rng.randint(0, (budget - sink) // 2))
    n_q, Hq = rng.randint(1, 17), Hkv * rng.choice([1, 2, 4, 7, 8])
    if rng.random() < 0.3:  # a chunk of a prompt
        B = min(B, 4)
        n_q = min(_log_int(rng, 18, 2048), max(1, 1_000_000_000 // (B * Hq * (hi + 2048))))
    return dict(op=op, B=B, n_q=n_q, ragged=rng.random() < 0.5, Hq=Hq, Hkv=Hkv, D=D, bs=bs, lo=lo,
                hi=hi)


def _lens(case):
    """Tokens before this call, tokens of this call and those of them that count, per request."""
    rng = random.Random("%d %d %d %d" % (case["B"], case["lo"], case["hi"], case.get("n_q", 0)))
    n = case.get("n_q", 0)
    prior = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    live = [rng.randint(1, n) if case.get("ragged") else n for _ in range(case["B"])]
    return prior, [n] * case["B"], live


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["n"] * (case["Hq"] + case["Hk"])
        return {"bytes": values * case["D"] * 4 + case["n"] * 4 + case["rot"] * 4,
                "flops": values * case["rot"] * 3}
    if op in ("truncate", "sample"):
        rows, V = case["B"] * case["J"], case["V"]
        b = rows * V * (4 if case["kind"] == "probs" else 2)
        if op == "truncate":
            b += rows * V * 4
        return {"bytes": b + rows * 16 + case["B"] * 16, "flops": rows * V * 4}
    prior, count, live = _lens(case)
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    if op == "evict":
        kept = sum(min(c, case["budget"]) for c in prior)
        # every score read; of the tokens kept, K and V read and written, and their scores written
        return {"bytes": sum(prior) * Hkv * 4 + kept * Hkv * (4 * D + 4 + 4)
                + 2 * sum(-(-c // bs) for c in prior) * (4 + 8 * Hkv), "flops": kept * Hkv * D * 2}
    kv = [a + b for a, b in zip(prior, count)]
    pairs = sum(c * (a + 1) + c * (c - 1) // 2 for a, c in zip(prior, live))
    return {"bytes": sum(kv) * Hkv * (D + 8) + sum(-(-c // bs) for c in kv) * (4 + 4 * Hkv)
            + sum(live) * case["Hq"] * (2 * D + 4), "flops": 2 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _filled_cache(nb, bs, Hkv, D, gen):
    """A cache in use: values with heads of different size, quantised page by page with powers of
    two as scales."""
    x = torch.randn(nb, bs, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16).float()
    x *= torch.exp(0.5 * torch.randn(nb, 1, Hkv, 1, generator=gen, device=DEV))
    k = torch.ceil(torch.log2(x.abs().amax(dim=(1, 3)) / 448)).to(torch.int32)
    s = ((k + 127) << 23).view(torch.float32)
    return (x / s[:, None, :, None]).clamp(-448, 448).to(E4M3), s.contiguous()


def _pages(kv, bs, gen, more=None):
    """A shuffled block table that covers kv[r] tokens of every request, -1 where unused, and with
    `more` a second one, of other pages, that covers more[r]."""
    counts = list(kv) + list(more or [])
    need = torch.tensor([-(-c // bs) for c in counts], device=DEV)
    nb = int(need.sum())
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(counts), max(1, int(need.max()))), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(table.shape[1], device=DEV)[None] < need[:, None]] = perm
    if more is None:
        return max(1, nb), table
    B = len(kv)
    return max(1, nb), table[:B].contiguous(), table[B:, :max(1, int(need[B:].max()))].contiguous()


def _prefix(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


# the stretches that a case's frequencies are made with
STRETCH = {"plain": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
           "bands": dict(factor=8.0, original_len=8192, low=1.0, high=4.0),
           "yarn": dict(factor=8.0, original_len=16384, low=1.0, high=32.0)}
BASE = 500000.0


def _angles(rot, kind, base=BASE):
    """Radians a position for every pair, in 64 bits, and the factor that the rotated values take."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV)
    f = base ** (-i / rot)
    p = STRETCH[kind]
    if kind == "linear":
        f = f / p["factor"]
    if kind == "ntk":
        f = (base * p["factor"] ** (rot / max(1, rot - 2))) ** (-i / rot)
    if kind == "bands":  # by the turns that a pair makes over the original length
        turns = p["original_len"] * f / (2 * math.pi)
        keep = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * keep + f / p["factor"] * (1 - keep)
    if kind == "yarn":  # a ramp over the pairs, between those that make high and low turns
        at = [rot * math.log(p["original_len"] / (t * 2 * math.pi)) / (2 * math.log(base))
              for t in (p["high"], p["low"])]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1 - ((i / 2 - first) / max(last - first, 0.001)).clamp(0, 1)
        return f * keep + f / p["factor"] * (1 - keep), 0.1 * math.log(p["factor"]) + 1
    return f, 1.0


def prepare(case, seed):
    return {"rope": _prep_rope, "weights": _prep_weights, "evict": _prep_evict,
            "truncate": _prep_rows, "sample": _prep_rows}[case["op"]](case, _gen(seed))


def _prep_rope(case, gen):
    n, Hq, Hk, D = case["n"], case["Hq"], case["Hk"], case["D"]
    qkv = torch.randn(n, Hq + 2 * Hk, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    first = int(torch.randint(0, case["hi"], (1,), generator=gen, device=DEV))
    pos = (torch.arange(n, device=DEV) + first) % case["hi"]
    freqs, scale = _angles(case["rot"], case["kind"])
    s = dict(op="rope", q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], pos=pos.to(torch.int32),
             rot=case["rot"], pairs=case["pairs"], inverse=case["inverse"], freqs=freqs, scale=scale,
             turns=(freqs / (2 * math.pi) * 2.0 ** 64).to(torch.int64),  # a program makes it once
             q_out=torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV),
             k_out=torch.empty(n, Hk, D, dtype=torch.bfloat16, device=DEV))
    return s


def _prep_weights(case, gen):
    prior, count, live = _lens(case)
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    kv = [a + b for a, b in zip(prior, count)]
    nb, table = _pages(kv, bs, gen)
    k_cache, k_scale = _filled_cache(nb, bs, Hkv, D, gen)
    n = sum(count)
    q = torch.randn(n, Hq, D, generator=gen, device=DEV)
    q *= torch.exp(0.3 * torch.randn(n, Hq, 1, generator=gen, device=DEV))
    s = dict(op="weights", q=q.bfloat16(), k_cache=k_cache, k_scale=k_scale, table=table,
             cu=_prefix(count), ctx=torch.tensor(kv, dtype=torch.int32, device=DEV),
             live=torch.tensor(live, dtype=torch.int32, device=DEV), max_q=case["n_q"],
             sm_scale=1.0 / math.sqrt(D), decay=0.98,
             before=torch.rand(nb, Hkv, bs, generator=gen, device=DEV),
             after=torch.zeros(nb, Hkv, bs, device=DEV), err=torch.zeros(1, dtype=torch.int32, device=DEV))
    # what the attention pass left beside its output: the log of every row's sum
    x, seen = _scores(s)
    x.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    M = case["n_q"]
    s["lse"] = lse.permute(0, 2, 1, 3).reshape(B * M, Hq).contiguous()
    return s


def _prep_evict(case, gen):
    prior, _, _ = _lens(case)
    B, Hkv, D, bs, budget = case["B"], case["Hkv"], case["D"], case["bs"], case["budget"]
    nb, table, fresh = _pages(prior, bs, gen, more=[min(c, budget) for c in prior])
    k_cache, k_scale = _filled_cache(nb, bs, Hkv, D, gen)
    v_cache, v_scale = _filled_cache(nb, bs, Hkv, D, gen)
    # a few tokens have gathered much weight, most little, some none
    w = torch.exp(2 * torch.randn(nb, Hkv, bs, generator=gen, device=DEV))
    w *= torch.rand(nb, Hkv, bs, generator=gen, device=DEV) > 0.05
    return dict(op="evict", k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                weights=w, table=table, fresh=fresh, sink=case["sink"], recent=case["recent"],
                ctx=torch.tensor(prior, dtype=torch.int32, device=DEV),
                new_lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                kept=torch.zeros(B, Hkv, budget, dtype=torch.int32, device=DEV),
                err=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prep_rows(case, gen):
    B, J, V = case["B"], case["J"], case["V"]
    rows = torch.randn(B * J, V, generator=gen, device=DEV, dtype=torch.bfloat16)
    # flat rows and peaked ones
    rows *= (1.0 + 3.0 * torch.rand(B * J, 1, generator=gen, device=DEV)).bfloat16()
    if case["kind"] == "probs":
        rows = torch.softmax(rows.float(), dim=-1)
    else:  # entries that a grammar forbids
        rows.masked_fill_(torch.rand(1, V, generator=gen, device=DEV) < 0.02, -math.inf)
        rows[:, 0] = 1.0
    r = torch.arange(B, device=DEV)
    T = 0.5 + 0.9 * torch.rand(B, generator=gen, device=DEV)
    T[r % 16 == 9] = 0.0  # greedy requests
    top_k = torch.randint(1, 200, (B,), generator=gen, device=DEV, dtype=torch.int32)
    top_k[r % 3 != 1] = 0  # off
    top_p = 0.5 + 0.49 * torch.rand(B, generator=gen, device=DEV)
    top_p[r % 4 == 2] = 1.0
    min_p = 0.1 * torch.rand(B, generator=gen, device=DEV)
    min_p[r % 2 == 0] = 0.0
    s = dict(op=case["op"], rows=rows, kind=case["kind"], J=J, T=T, top_k=top_k, top_p=top_p,
             min_p=min_p, kept=torch.empty(B, J, dtype=torch.int32, device=DEV),
             err=torch.zeros(1, dtype=torch.int32, device=DEV))
    if case["op"] == "truncate":
        s["probs"] = torch.empty(B * J, V, device=DEV)
    else:
        s["u"] = torch.rand(B, J, generator=gen, device=DEV)
        s["tokens"] = torch.empty(B, J, dtype=torch.int32, device=DEV)
        s["prob"] = torch.empty(B, J, device=DEV)
    return s


# ------------------------------------------------------------------------------------- one pass
def run(s):
    return {"rope": _rope, "weights": _weights, "evict": _evict, "truncate": _truncate,
            "sample": _sample}[s["op"]](s)


def _rope(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_rope(s["pos"], s["turns"], q=s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"],
                   pairs=s["pairs"], scale=s["scale"], inverse=s["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    a = s["pos"].double()[:, None] * s["freqs"]
    c, w = torch.cos(a).float()[:, None] * s["scale"], torch.sin(a).float()[:, None] * s["scale"]
    if s["inverse"]:
        w = -w
    return {"q": _turn(s["q"], c, w, s), "k": _turn(s["k"], c, w, s)}


def _turn(x, c, w, s):
    rot, x = s["rot"], x.float()
    if s["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * w, b * c + a * w], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).bfloat16()


def _scores(s):
    """Every query row against every place of its request's table: [B, Hkv, M, G, T] fp32, and
    whether it sees it."""
    table, page = s["table"], s["table"].clamp(min=0).long()
    k = s["k_cache"].view(torch.uint8)[page].view(E4M3).float()
    k *= (s["k_scale"][page] * (table >= 0)[..., None])[:, :, None, :, None]
    B, mb, bs, H, D = k.shape
    k = k.reshape(B, mb * bs, H, D)
    M, Hq = s["max_q"], s["q"].shape[1]
    q = s["q"].float().view(B, M, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    x = (torch.matmul(q, k.permute(0, 2, 3, 1)) * s["sm_scale"]).view(B, H, M, Hq // H, mb * bs)
    last = s["ctx"].long()[:, None] - M + torch.arange(M, device=DEV)[None]
    seen = torch.arange(mb * bs, device=DEV)[None, None] <= last[..., None]
    return x, seen[:, None, :, None]


def _weights(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_kv_weights(s["q"], s["lse"], s["k_cache"], s["k_scale"], s["table"], s["ctx"], s["cu"],
                         s["after"], before=s["before"], live=s["live"], sm_scale=s["sm_scale"],
                         decay=s["decay"], err=s["err"])
        return s["after"]
    x, seen = _scores(s)
    B, H, M, G, T = x.shape
    j = torch.arange(M, device=DEV)
    seen = seen & (j[None] < s["live"][:, None])[:, None, :, None, None]
    x -= s["lse"].view(B, M, H, G).permute(0, 2, 1, 3)[..., None]
    w = torch.exp(x.masked_fill_(~seen, -math.inf)).sum((2, 3))  # [B, H, T]
    bs, t = s["after"].shape[2], torch.arange(T, device=DEV)
    page, off = s["table"].long()[:, t // bs], t % bs
    old = s["before"][page.clamp(min=0), :, off[None]].permute(0, 2, 1) * s["decay"]
    ctx = s["ctx"].long()[:, None]
    w += torch.where((t[None] < ctx - M)[:, None], old, torch.zeros_like(old))
    r, at = torch.nonzero(t[None] < ctx, as_tuple=True)
    s["after"][page[r, at], :, off[at]] = w[r, :, at]
    return s["after"]


def _evict(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_kv_evict(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["weights"],
                       s["table"], s["ctx"], s["kept"], s["new_lens"], to_table=s["fresh"],
                       sink=s["sink"], recent=s["recent"], err=s["err"])
    else:
        _plain_evict(s)
    return {f: s[f] for f in ("k_cache", "v_cache", "k_scale", "v_scale", "weights", "kept",
                              "new_lens")}


def _plain_evict(s):
    B, H, budget = s["kept"].shape
    nb, bs = s["k_cache"].shape[:2]
    T = s["table"].shape[1] * bs
    t = torch.arange(T, device=DEV)
    ctx = s["ctx"].long()[:, None, None]
    page = s["table"].long()[:, t // bs].clamp(min=0)
    w = s["weights"][page, :, (t % bs)[None]].permute(0, 2, 1)  # [B, H, T]
    middle = (t >= s["sink"]) & (t < ctx - s["recent"])
    order = torch.sort(torch.where(middle, w, torch.full_like(w, -1.0)), dim=-1, descending=True,
                       stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    best = middle & (rank < budget - s["sink"] - s["recent"])
    keep = (t < ctx) & (best | ~middle | (ctx <= budget))
    s["kept"].fill_(-1)
    r, h, at = torch.nonzero(keep, as_tuple=True)
    j = (torch.cumsum(keep, -1) - 1)[r, h, at]
    s["kept"][r, h, j] = at.to(torch.int32)
    s["new_lens"].copy_(s["ctx"].clamp(max=budget))
    src, dst = page[r, at], s["fresh"].long()[r, j // bs]
    s["weights"][dst, h, j % bs] = s["weights"][src, h, at % bs]
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        now = torch.zeros(nb * H, device=DEV)
        now.index_reduce_(0, dst * H + h, scale[src, h], "amax")
        ratio = scale[src, h] / now[dst * H + h]
        raw = cache.view(torch.uint8)
        x = raw[src, at % bs, h].view(E4M3).float() * ratio[:, None]
        raw[dst, j % bs, h] = x.to(E4M3).view(torch.uint8)
        scale[dst, h] = now[dst * H + h]


def _cut(s):
    """The entries of every row in order (larger first, equal ones by index), their weights in 64 bits
    in that order, those kept, and the kept weights' running sums."""
    J = s["J"]
    T, k, p, m = (s[f].repeat_interleave(J) for f in ("T", "top_k", "top_p", "min_p"))
    x, at = torch.sort(s["rows"].float(), dim=-1, descending=True, stable=True)
    greedy = T == 0
    if s["kind"] == "probs":
        w = x.double()
    else:
        T = torch.where(greedy, torch.ones_like(T), T).double()
        w = torch.exp((x.double() - x[:, :1].double()) / T[:, None])
    i = torch.arange(x.shape[1], device=DEV)
    k = torch.where(greedy, torch.ones_like(k), torch.where(k > 0, k, torch.full_like(k, 2**31 - 1)))
    keep = (i < k[:, None]) & (w > 0)
    w *= keep
    run = torch.cumsum(w, -1)
    before, total = run - w, run[:, -1:].clone()
    keep &= (before < p.double()[:, None] * total) | (p >= 1)[:, None] | (i == 0)
    keep &= (w >= m.double()[:, None] * w[:, :1]) | (i == 0)
    w *= keep
    return at, w, keep, torch.cumsum(w, -1)


def _truncate(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_truncate(s["rows"], s["probs"], s["kept"], temperature=s["T"], top_k=s["top_k"],
                       top_p=s["top_p"], min_p=s["min_p"], err=s["err"])
    else:
        at, w, keep, run = _cut(s)
        w /= run[:, -1:]
        s["probs"].scatter_(1, at, w.float())
        s["kept"].copy_(keep.sum(-1).view_as(s["kept"]))
    return {"probs": s["probs"], "kept": s["kept"]}


def _sample(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_sample(s["rows"], s["u"], s["tokens"], prob=s["prob"], kept=s["kept"],
                     temperature=s["T"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                     err=s["err"])
    else:
        at, w, keep, run = _cut(s)
        n = keep.sum(-1, keepdim=True)
        goal = s["u"].view(-1, 1).double() * run[:, -1:]
        j = torch.minimum((run <= goal).sum(-1, keepdim=True), n - 1)
        s["tokens"].copy_(at.gather(1, j).view_as(s["tokens"]))
        s["prob"].copy_((w.gather(1, j) / run[:, -1:]).view_as(s["prob"]))
        s["kept"].copy_(n.view_as(s["kept"]))
    return {"tokens": s["tokens"], "prob": s["prob"], "kept": s["kept"]}


# ------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "weights": _exact_weights, "evict": _exact_evict,
            "truncate": _exact_rows, "sample": _exact_rows}[case["op"]](case, s)


def _exact_rope(case, s):
    f, scale = _angles(case["rot"], case["kind"])
    z = torch.polar(torch.full_like(f, scale)[None].expand(case["n"], -1).contiguous(),
                    s["pos"].double()[:, None] * f)
    if case["inverse"]:
        z = z.conj()
    res = {}
    for name in ("q", "k"):
        x = s[name].double()
        rot = case["rot"]
        part = x[..., :rot]
        pair = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["pairs"] == "halves" \
            else part.unflatten(-1, (rot // 2, 2))
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None])
        y = y.transpose(-1, -2) if case["pairs"] == "halves" else y
        x[..., :rot] = y.flatten(-2)
        res[name] = x
    return res


def _exact_weights(case, s):
    prior, count, live = _lens(case)
    if work(case)["flops"] > 2e12:
        return None
    res = torch.zeros_like(s["after"], dtype=torch.float64)
    G, bs, at = case["Hq"] // case["Hkv"], case["bs"], 0
    for r in range(case["B"]):
        n = prior[r] + count[r]
        page = s["table"][r, :-(-n // bs)].long()
        k = s["k_cache"].view(torch.uint8)[page].view(E4M3).double()
        k = (k * s["k_scale"][page].double()[:, None, :, None]).flatten(0, 1)
        pos = torch.arange(k.shape[0], device=DEV)
        seen = pos[None] <= prior[r] + torch.arange(live[r], device=DEV)[:, None]
        old = s["before"][page].double() * s["decay"]  # [pages, Hkv, bs]
        old = torch.where((pos < prior[r]).view(-1, 1, bs), old, torch.zeros_like(old))
        for h in range(case["Hq"]):
            x = s["q"][at:at + live[r], h].double() @ k[:, h // G].T * s["sm_scale"]
            e = torch.exp(x - s["lse"][at:at + live[r], h].double()[:, None])
            old[:, h // G] += torch.where(seen, e, torch.zeros_like(e)).sum(0).view(-1, bs)
        old = torch.where((pos < n).view(-1, 1, bs), old, torch.zeros_like(old))
        res[page] = old
        at += count[r]
    return res


def _exact_evict(case, s):
    """Request by request and head by head; a value moves to its new page's scale by its step there (a
    multiple of 2^(exponent - 3), 2^-9 at the least, halves to even)."""
    prior, _, _ = _lens(case)
    bs, budget, sink, recent = case["bs"], case["budget"], case["sink"], case["recent"]
    caches = [s[f].view(torch.uint8).view(E4M3).double() for f in ("k_cache", "v_cache")]
    scales = [s[f].double() for f in ("k_scale", "v_scale")]
    w, kept = s["weights"].double(), torch.full_like(s["kept"], -1)
    for r in range(case["B"]):
        n = prior[r]
        page = s["table"][r].long()
        pos = torch.arange(n, device=DEV)
        for h in range(case["Hkv"]):
            take = pos
            if n > budget:
                mid = pos[sink:n - recent]
                by = w[page[mid // bs], h, mid % bs]
                best = mid[torch.sort(by, descending=True, stable=True).indices]
                take = torch.cat([pos[:sink], best[:budget - sink - recent], pos[n - recent:]])
                take = torch.sort(take).values
            m = take.numel()
            if not m:
                continue
            kept[r, h, :m] = take.to(torch.int32)
            to = s["fresh"][r].long()[:-(-m // bs)]
            src, off = page[take // bs], take % bs
            pad = to.numel() * bs - m
            j = torch.arange(m, device=DEV)
            w[to[j // bs], h, j % bs] = w[src, h, off]
            for x, sc in zip(caches, scales):
                fill = torch.nn.functional.pad(sc[src, h], (0, pad)).view(-1, bs)
                big = fill.amax(1)
                y = x[src, off, h] * (sc[src, h] / big[j // bs])[:, None]
                _, e = torch.frexp(y)
                step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
                x[to[j // bs], j % bs, h] = torch.round(y / step) * step
                sc[to, h] = big
    return {"k_cache": caches[0], "v_cache": caches[1], "k_scale": scales[0], "v_scale": scales[1],
            "weights": w, "kept": kept, "new_lens": s["ctx"].clamp(max=budget)}


def _exact_rows(case, s):
    """Row by row blocks: thresholds in the order of the weights, by searching the running sums."""
    J, out = case["J"], {"probs": [], "kept": [], "tokens": [], "prob": []}
    V = case["V"]
    for a in range(0, s["rows"].shape[0], 128):
        x = s["rows"][a:a + 128].double()
        r = (a + torch.arange(x.shape[0], device=DEV)) // J
        T, top_k, top_p, min_p = (s[f][r] for f in ("T", "top_k", "top_p", "min_p"))
        T = torch.where(T > 0, T, torch.ones_like(T)).double()
        p = x if case["kind"] == "probs" else torch.softmax(x / T[:, None], -1)
        by, at = torch.sort(x, dim=-1, descending=True, stable=True)
        p = p.gather(1, at)
        run = torch.cumsum(p, -1)
        live = (p > 0).sum(-1)
        n = torch.where(top_k > 0, torch.minimum(top_k.long(), live), live).clamp(min=1)
        whole = run.gather(1, n[:, None] - 1)
        lead = torch.searchsorted(run, top_p.double()[:, None] * whole)[:, 0] + 1
        n = torch.where(top_p < 1, torch.minimum(n, lead), n)
        n = torch.minimum(n, (p >= min_p.double()[:, None] * p[:, :1]).sum(-1).clamp(min=1))
        n = torch.where(s["T"][r] > 0, n, torch.ones_like(n))
        total = run.gather(1, n[:, None] - 1)
        p = torch.where(torch.arange(V, device=DEV)[None] < n[:, None], p / total, torch.zeros_like(p))
        out["kept"].append(n.to(torch.int32))
        if case["op"] == "truncate":
            out["probs"].append(torch.zeros_like(p).scatter_(1, at, p))
        else:
            goal = s["u"].view(-1)[a:a + 128].double()[:, None] * total
            j = torch.minimum(torch.searchsorted(run, goal, right=True), n[:, None] - 1)
            out["tokens"].append(at.gather(1, j).to(torch.int32))
            out["prob"].append(p.gather(1, j))
    kept = torch.cat(out["kept"]).view_as(s["kept"])
    if case["op"] == "truncate":
        return {"probs": torch.cat(out["probs"]), "kept": kept}
    return {"tokens": torch.cat(out["tokens"]).view_as(kept), "kept": kept,
            "prob": torch.cat(out["prob"]).view(kept.shape)}
