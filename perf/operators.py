"""Cases of the cache and answer operators: sd_kv_write, sd_kv_read, sd_kv_attend and
sd_token_logprobs, each beside a plain form in elementary torch operations.

Lengths, slots and tables stay on the device in every call; the host knows the sizes of the
arrays and an upper bound of a request's tokens. The cache is paged, in e4m3, with one fp32
scale (a power of two) for each page and KV head.

Sizes are those of the framework's workloads (batches of 1, 64, 128, 256 and 1024 requests, 4 to
8 drafts, contexts of 37, 512..8192, 1000..16000 and 128..32000 tokens, pages of 16 tokens,
vocabularies of 1024 and 201088 entries) with generic head layouts.

A case's lengths follow from the case alone; its values follow from the seed.
"""

import math
import random

import torch

own = False  # False: the plain forms; True: the framework's operators

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
LOG_MIN_SCALE = -100  # the smallest scale a page is given is 2^-100


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step's K+1 verify slots of every request, appended to a cache in use (b64's batch)
        dict(name="write-b64", op="write", B=64, n_q=6, Hkv=8, D=64, bs=16, lo=512, hi=8192),
        # two prompts of 8192 tokens entering fresh pages, K and V as slices of one projection
        dict(name="write-prompt", op="write", B=2, n_q=8192, Hkv=8, D=128, bs=16, lo=0, hi=0),
        # one long request leaving the cache (32000 tokens), for a move to another precision
        dict(name="read-one", op="read", B=1, Hkv=8, D=128, bs=16, lo=32000, hi=32000),
        # a whole batch's contexts read back
        dict(name="read-b64", op="read", B=64, Hkv=8, D=64, bs=16, lo=512, hi=8192),
        # the smallest step: one request, K = 4, 37 tokens of context; latency counts
        dict(name="attend-small", op="attend", B=1, n_q=5, ragged=False, Hq=8, Hkv=2, D=64,
             bs=16, lo=37, hi=37),
        # a single token of one request over a long context
        dict(name="attend-one", op="attend", B=1, n_q=1, ragged=False, Hq=32, Hkv=8, D=128,
             bs=16, lo=32000, hi=32000),
        # the target's verify pass over K+1 slots of b64
        dict(name="attend-b64", op="attend", B=64, n_q=6, ragged=False, Hq=64, Hkv=8, D=64,
             bs=16, lo=512, hi=8192),
        # the target's verify pass of b256mix
        dict(name="attend-b256", op="attend", B=256, n_q=8, ragged=False, Hq=32, Hkv=8, D=128,
             bs=16, lo=1000, hi=16000),
        # the drafter's pass over the rebuilt batch: a_r + K slots per request, uneven contexts
        dict(name="attend-draft", op="attend", B=128, n_q=16, ragged=True, Hq=64, Hkv=8, D=64,
             bs=16, lo=128, hi=32000),
        # a prompt of 8192 tokens, causal
        dict(name="attend-prompt", op="attend", B=1, n_q=8192, ragged=False, Hq=32, Hkv=8, D=128,
             bs=16, lo=0, hi=0),
        # log probabilities of one small step's answer, on probability rows
        dict(name="logprobs-small", op="logprobs", B=1, J=5, V=1024, kind="probs", top=5),
        # log probabilities of b1024lg's answers: 9216 rows of logits, 20 alternatives each
        dict(name="logprobs-b1024", op="logprobs", B=1024, J=9, V=201088, kind="logits", top=20),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "logprobs"])
    if op == "logprobs":
        V = _log_int(rng, 7, 201088)
        rows = _log_int(rng, 1, max(1, min(9216, int(4e8) // V)))
        J = rng.randint(1, min(17, rows))
        return dict(op=op, B=max(1, rows // J), J=J, V=V, kind=rng.choice(["probs", "logits"]),
                    top=min(V, rng.randint(0, 32)))
    D = rng.choice([32, 64, 64, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    bs = rng.choice([8, 16, 16, 32, 64, 128])
    hi = _log_int(rng, 16, 32000)
    lo = rng.randint(0, hi)
    tokens = 60_000_000 // (Hkv * D)  # caches of up to 120 MB, K and V together
    B = _log_int(rng, 1, max(1, min(256, tokens // (hi + 1))))
    if op == "read":
        return dict(op=op, B=B, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi)
    if op == "write":
        return dict(op=op, B=B, n_q=_log_int(rng, 1, max(1, min(8192, 16384 // B))), Hkv=Hkv,
                    D=D, bs=bs, lo=lo, hi=hi)
    G = rng.choice([1, 2, 4, 7, 8])
    long = rng.random() < 0.3
    n_q = rng.randint(1, 17)
    if long:  # a chunk of a prompt
        B = min(B, 4)
        n_q = _log_int(rng, 18, 2048)
    return dict(op=op, B=B, n_q=n_q, ragged=rng.random() < 0.5, Hq=G * Hkv, Hkv=Hkv, D=D, bs=bs,
                lo=lo, hi=hi)


def _lens(case):
    """Tokens before this call, and tokens of this call, per request: from the case alone."""
    rng = random.Random("%d %d %d %d" % (case["B"], case["lo"], case["hi"], case.get("n_q", 0)))
    lo, hi, n = case["lo"], case["hi"], case.get("n_q", 0)
    uneven = lo > 0 and hi >= 32 * lo
    prior = [_log_int(rng, lo, hi) if uneven else rng.randint(lo, hi) for _ in range(case["B"])]
    count = [rng.randint((n + 1) // 2, n) if case.get("ragged") else n for _ in range(case["B"])]
    return prior, count


def work(case):
    op = case["op"]
    if op == "logprobs":
        size = 4 if case["kind"] == "probs" else 2
        rows = case["B"] * case["J"]
        live = sum(_emitted(case))
        return {"bytes": live * case["V"] * size + rows * (16 + 8 * case["top"]),
                "flops": live * case["V"] * 6}
    prior, count = _lens(case)
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    if op == "write":
        n = sum(count)
        return {"bytes": n * Hkv * D * 2 * (2 + 1) + n * 4, "flops": n * Hkv * D * 2 * 2}
    kv = [a + b for a, b in zip(prior, count)]
    pages = sum(-(-c // bs) for c in kv)
    if op == "read":
        n = sum(kv)
        return {"bytes": n * Hkv * D * 2 * (1 + 2) + pages * (4 + 8 * Hkv), "flops": n * Hkv * D * 2}
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(prior, count))
    n, Hq = sum(count), case["Hq"]
    return {"bytes": sum(kv) * Hkv * D * 2 + pages * (4 + 8 * Hkv) + n * Hq * (D * 4 + 4),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _two_to(e):
    """2^e exactly, in 64 bits, for whole e from -140 to 140 (a power function may round)."""
    table = torch.tensor([2.0 ** i for i in range(-140, 141)], dtype=torch.float64, device=DEV)
    return table[e.long() + 140]


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-100."""
    m, e = torch.frexp(amax.float() / 448.0)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, LOG_MIN_SCALE)).clamp(min=LOG_MIN_SCALE)
    return _two_to(e).float()


def _filled_cache(nb, bs, Hkv, D, gen):
    """A cache in use: bf16-like values with heads of different size, quantised page by page."""
    x = torch.randn(nb, bs, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16).float()
    x *= torch.exp(0.5 * torch.randn(nb, 1, Hkv, 1, generator=gen, device=DEV))
    s = _pow2_scale(x.abs().amax(dim=(1, 3)))
    return (x / s[:, None, :, None]).to(E4M3), s


def _pages(kv, bs, gen):
    """A shuffled block table that covers kv[r] tokens of every request, -1 where unused."""
    need = torch.tensor([-(-c // bs) for c in kv], device=DEV)
    nb = int(need.sum())
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(kv), max(1, int(need.max()))), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(table.shape[1], device=DEV)[None] < need[:, None]] = perm
    return max(1, nb), table


def _prefix(counts):
    t = torch.tensor([0] + list(counts), dtype=torch.int64)
    return t.cumsum(0).to(torch.int32).to(DEV)


def _emitted(case):
    """Tokens of each request's answer: its accepted drafts and one more."""
    rng = random.Random("%d %d" % (case["B"], case["J"]))
    return [rng.randint(1, case["J"]) for _ in range(case["B"])]


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    if op == "logprobs":
        B, J, V = case["B"], case["J"], case["V"]
        rows = torch.randn(B * J, V, generator=gen, device=DEV, dtype=torch.bfloat16)
        rows *= 2
        if case["kind"] == "probs":
            rows = torch.softmax(rows.float(), dim=-1)
        tokens = torch.randint(0, V, (B, J), generator=gen, device=DEV, dtype=torch.int32)
        best = rows.view(B, J, V).argmax(-1).to(torch.int32)
        tokens = torch.where(torch.rand(B, J, generator=gen, device=DEV) < 0.5, best, tokens)
        live = torch.tensor(_emitted(case), device=DEV)
        tokens[torch.arange(J, device=DEV)[None] >= live[:, None]] = -1
        temp = 0.5 + 0.7 * torch.rand(B, generator=gen, device=DEV)
        temp[::7] = 0.0  # greedy requests
        top = case["top"]
        f32, i32 = dict(device=DEV), dict(device=DEV, dtype=torch.int32)
        return dict(op=op, rows=rows, tokens=tokens, kind=case["kind"], top=top,
                    temperature=temp, logprob=torch.empty(B, J, **f32),
                    entropy=torch.empty(B, J, **f32), rank=torch.empty(B, J, **i32),
                    top_ids=torch.empty(B, J, top, **i32),
                    top_logprobs=torch.empty(B, J, top, **f32),
                    err=torch.zeros(1, **i32))
    prior, count = _lens(case)
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    kv = [a + b for a, b in zip(prior, count)]
    nb, table = _pages(kv, bs, gen)
    k_cache, k_scale = _filled_cache(nb, bs, Hkv, D, gen)
    v_cache, v_scale = _filled_cache(nb, bs, Hkv, D, gen)
    s = dict(op=op, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
             block_table=table, err=torch.zeros(1, dtype=torch.int32, device=DEV))
    if op == "read":
        n = sum(kv)
        s.update(cu=_prefix(kv), k_out=torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV),
                 v_out=torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV))
        return s
    n = sum(count)
    start = torch.tensor(prior, device=DEV).repeat_interleave(torch.tensor(count, device=DEV))
    cu = _prefix(count)
    r = torch.arange(len(count), device=DEV).repeat_interleave(torch.tensor(count, device=DEV))
    pos = start + torch.arange(n, device=DEV) - cu.long()[r]
    if op == "write":
        # K and V are slices of one projection [n, 3, Hkv, D]; some slots are rejected (-1)
        qkv = torch.randn(n, 3, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16)
        qkv *= torch.exp(0.7 * torch.randn(n, 1, Hkv, 1, generator=gen, device=DEV)).bfloat16()
        slot = table[r, pos // bs] * bs + (pos % bs).to(torch.int32)
        if case["n_q"] > 1 and case["n_q"] < 32:
            kept = torch.randint(1, case["n_q"] + 1, (len(count),), generator=gen, device=DEV)
            slot[torch.arange(n, device=DEV) - cu.long()[r] >= kept[r]] = -1
        s.update(k=qkv[:, 1], v=qkv[:, 2], slots=slot)
        return s
    Hq = case["Hq"]
    q = torch.randn(n, Hq, D, generator=gen, device=DEV)
    q *= torch.exp(0.3 * torch.randn(n, Hq, 1, generator=gen, device=DEV))
    s.update(q=q.bfloat16(), cu=cu, max_q=case["n_q"], sm_scale=1.0 / math.sqrt(D),
             ctx=torch.tensor(kv, dtype=torch.int32, device=DEV),
             out=torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(n, Hq, device=DEV))
    return s


# ------------------------------------------------------------------------------------- one pass
def run(s):
    return {"write": _write, "read": _read, "attend": _attend, "logprobs": _logprobs}[s["op"]](s)


def _write(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                       s["v_scale"], err=s["err"])
    else:
        _plain_store(s["k"], s["slots"], s["k_cache"], s["k_scale"])
        _plain_store(s["v"], s["slots"], s["v_cache"], s["v_scale"])
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _plain_store(x, slots, cache, scale):
    """A page's scale grows to hold what is written to it; what it held is rounded again to the
    new scale. A write to a page's first slot starts the page afresh."""
    nb, bs, H, D = cache.shape
    x, slots = x[slots >= 0].float(), slots[slots >= 0].long()
    page, off = slots // bs, slots % bs
    amax = torch.zeros(nb, H, device=DEV).index_reduce_(0, page, x.abs().amax(-1), "amax")
    fresh = torch.zeros(nb, dtype=torch.bool, device=DEV)
    fresh[page[off == 0]] = True
    touched = torch.zeros(nb, dtype=torch.bool, device=DEV)
    touched[page] = True
    old = torch.where(fresh[:, None], torch.zeros_like(scale), scale)
    new = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(amax)), scale)
    again = touched & ~fresh
    ratio = torch.where(again[:, None], old / new, torch.ones_like(new))[page]
    raw = cache.view(torch.uint8)
    held = raw[page].view(E4M3).float() * ratio[:, None, :, None]
    raw[page] = held.to(E4M3).view(torch.uint8)
    raw[page, off] = (x / new[page][:, :, None]).to(E4M3).view(torch.uint8)
    scale.copy_(new)


def _plain_gather(s, cache, scale):
    """[B, T, Hkv, D] fp32 of every request's pages (zeros where there is none)."""
    table = s["block_table"]
    page = table.clamp(min=0).long()
    x = cache.view(torch.uint8)[page].view(E4M3).float()
    x *= (scale[page] * (table >= 0)[..., None])[:, :, None, :, None]
    B, mb, bs, H, D = x.shape
    return x.reshape(B, mb * bs, H, D)


def _read(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                      s["cu"], s["k_out"], s["v_out"], err=s["err"])
        return {"k": s["k_out"], "v": s["v_out"]}
    n, cu = s["k_out"].shape[0], s["cu"].long()
    i = torch.arange(n, device=DEV)
    r = torch.searchsorted(cu, i, right=True) - 1
    k, v = (_plain_gather(s, s[c], s[f])[r, i - cu[r]].bfloat16()
            for c, f in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
    return {"k": k, "v": v}


def _attend(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_kv_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                        s["block_table"], s["ctx"], s["cu"], s["out"], lse=s["lse"],
                        max_q=s["max_q"], sm_scale=s["sm_scale"], err=s["err"])
        return {"out": s["out"], "lse": s["lse"]}
    k, v = _plain_gather(s, s["k_cache"], s["k_scale"]), _plain_gather(s, s["v_cache"], s["v_scale"])
    (B, T, H, D), M = k.shape, s["max_q"]
    n, Hq = s["lse"].shape
    G, cu, ctx = Hq // H, s["cu"].long(), s["ctx"].long()
    j = torch.arange(M, device=DEV)
    count = cu[1:] - cu[:-1]
    pad = (cu[:-1, None] + j[None]).clamp(max=n - 1)
    q = s["q"].float()[pad].view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["sm_scale"]
    last = ctx[:, None] - count[:, None] + j[None]  # the last token that slot j sees
    hidden = torch.arange(T, device=DEV)[None, None] > last[..., None]
    x = x.view(B, H, M, G, T).masked_fill_(hidden[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)))
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, M * G, T), v.permute(0, 2, 1, 3)).view(B, H, M, G, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    lse = (m + torch.log(z))[..., 0]
    i = torch.arange(n, device=DEV)
    r = torch.searchsorted(cu, i, right=True) - 1
    out = o.permute(0, 2, 1, 3, 4).reshape(B, M, Hq, D)[r, i - cu[r]].bfloat16()
    return {"out": out, "lse": lse.permute(0, 2, 1, 3).reshape(B, M, Hq)[r, i - cu[r]]}


def _logprobs(s):
    if own:
        import verify_draft_prep_gb300 as sd
        sd.sd_token_logprobs(s["rows"], s["tokens"], s["logprob"], entropy=s["entropy"],
                             rank=s["rank"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"],
                             temperature=s["temperature"], err=s["err"])
        return {k: s[k] for k in ("logprob", "entropy", "rank", "top_ids", "top_logprobs")}
    tokens, top = s["tokens"].long(), s["top"]
    B, J = tokens.shape
    x = s["rows"].float().view(B, J, -1)
    V = x.shape[-1]
    live = tokens >= 0
    if s["kind"] == "probs":
        lp = torch.log(x)
        ent = -torch.where(x > 0, x * lp, torch.zeros_like(x)).sum(-1)
    else:
        T = torch.where(s["temperature"] > 0, s["temperature"], torch.ones_like(s["temperature"]))
        y = x / T[:, None, None]
        y -= y.amax(-1, keepdim=True)
        e = torch.exp(y)
        z = e.sum(-1, keepdim=True)
        ent = torch.log(z[..., 0]) - (e * y).sum(-1) / z[..., 0]
        lp = y - torch.log(z)
    at = tokens.clamp(min=0)[..., None]
    own_x = x.gather(-1, at)
    i = torch.arange(V, device=DEV)
    rank = 1 + ((x > own_x) | ((x == own_x) & (i < at))).sum(-1)
    # one whole number for value and index together: the highest value first, then the lowest index
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * 2**32 + (2**31 - 1 - i)
    ids = 2**31 - 1 - torch.remainder(torch.topk(key, top, dim=-1).values, 2**32)
    top_lp = lp.gather(-1, ids)
    none = ~live
    return {"logprob": lp.gather(-1, at)[..., 0].masked_fill(none, 0.0),
            "entropy": ent.masked_fill(none, 0.0),
            "rank": rank.masked_fill(none, 0).to(torch.int32),
            "top_ids": ids.masked_fill(none[..., None], -1).to(torch.int32),
            "top_logprobs": top_lp.masked_fill(none[..., None], -math.inf)}


# ------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        return _exact_logprobs(s)
    if op == "write":
        res = {}
        for side in ("k", "v"):
            res[side], res[side + "_scale"] = _exact_store(s[side], s["slots"], s[side + "_cache"],
                                                           s[side + "_scale"])
        return res
    prior, count = _lens(case)
    kv = [a + b for a, b in zip(prior, count)]
    bs = case["bs"]

    def held(cache, scale, r):  # request r's tokens, [T, Hkv, D]
        page = s["block_table"][r, :-(-kv[r] // bs)].long()
        x = cache.view(torch.uint8)[page].view(E4M3).double() * scale[page].double()[:, None, :, None]
        return x.flatten(0, 1)[:kv[r]]

    if op == "read":
        k = torch.cat([held(s["k_cache"], s["k_scale"], r) for r in range(case["B"])])
        v = torch.cat([held(s["v_cache"], s["v_scale"], r) for r in range(case["B"])])
        return {"k": k, "v": v}
    if work(case)["flops"] > 4e12:
        return None
    out, lse, at = [], [], 0
    G = case["Hq"] // case["Hkv"]
    for r in range(case["B"]):
        q = s["q"][at:at + count[r]].double()
        at += count[r]
        k, v = held(s["k_cache"], s["k_scale"], r), held(s["v_cache"], s["v_scale"], r)
        pos = torch.arange(kv[r], device=DEV)
        seen = pos[None] <= prior[r] + torch.arange(count[r], device=DEV)[:, None]
        o_r, l_r = [], []
        for h in range(case["Hq"]):
            x = (q[:, h] @ k[:, h // G].T) * s["sm_scale"]
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            l_r.append(torch.logsumexp(x, -1))
            o_r.append(torch.softmax(x, -1) @ v[:, h // G])
        out.append(torch.stack(o_r, 1))
        lse.append(torch.stack(l_r, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_store(x, slots, cache, scale):
    """The same definition page by page on the host's side of the arithmetic: e4m3 rounding by
    its step (a multiple of 2^(exponent - 3), 2^-9 at the least), halves to even."""
    def e4m3(y):
        _, e = torch.frexp(y)
        step = _two_to((e - 1).clamp(min=-6) - 3)
        return torch.round(y / step) * step

    nb, bs, H, D = cache.shape
    values = cache.view(torch.uint8).view(E4M3).double()
    scale = scale.double()
    slot = torch.full((nb * bs,), -1, dtype=torch.long, device=DEV)
    n = torch.arange(slots.numel(), device=DEV)
    slot[slots[slots >= 0].long()] = n[slots >= 0]
    slot = slot.view(nb, bs)
    hit = (slot >= 0).any(1).nonzero()[:, 0]
    at, held = slot[hit], values[hit]
    new = (at >= 0)[:, :, None, None]
    put = torch.where(new, x.double()[at.clamp(min=0)], 0.0)
    peak = put.abs().amax(dim=(1, 3))
    need = torch.round(torch.log2(peak / 448)).clamp(min=LOG_MIN_SCALE)
    need = torch.where(448 * _two_to(need) < peak, need + 1, need)
    need = torch.where(448 * _two_to(need - 1) >= peak, need - 1, need).clamp(min=LOG_MIN_SCALE)
    s_old = torch.where(at[:, :1] >= 0, torch.zeros_like(peak), scale[hit])
    s_new = torch.maximum(s_old, _two_to(need))
    kept = torch.where((at[:, :1] >= 0), torch.ones_like(peak), s_old / s_new)
    values[hit] = torch.where(new, e4m3(put / s_new[:, None, :, None]),
                              e4m3(held * kept[:, None, :, None]))
    scale[hit] = s_new
    return values, scale


def _exact_logprobs(s):
    B, J = s["tokens"].shape
    V, top = s["rows"].shape[1], s["top"]
    out = {"logprob": [], "entropy": [], "top_logprobs": []}
    T = s["temperature"].double()
    T = torch.where(T > 0, T, torch.ones_like(T)).repeat_interleave(J)
    for a in range(0, B * J, 256):
        x, t = s["rows"][a:a + 256].double(), s["tokens"].view(-1)[a:a + 256].long()
        if s["kind"] == "probs":
            lp = torch.log(x)
            p = x
        else:
            lp = torch.log_softmax(x / T[a:a + 256, None], -1)
            p = torch.exp(lp)
        dead = t < 0
        out["logprob"].append(lp.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(dead, 0.0))
        out["entropy"].append(torch.special.xlogy(p, p).sum(-1).neg().masked_fill(dead, 0.0))
        best = torch.sort(lp, dim=-1, descending=True).values[:, :top]
        out["top_logprobs"].append(best.masked_fill(dead[:, None], -math.inf))
    res = {k: torch.cat(v) for k, v in out.items()}
    return {"logprob": res["logprob"].view(B, J), "entropy": res["entropy"].view(B, J),
            "rank": None, "top_ids": None, "top_logprobs": res["top_logprobs"].view(B, J, top)}
