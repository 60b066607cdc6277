"""Plain forms of the operators around a step's cache and draws, for the tests: 64-bit arithmetic
on small inputs, with the tolerances of computed numbers."""

import math

import torch

import kvref

TWO64 = 1 << 64


def rope_ref(x, positions, turns, pairs, scale, inverse):
    """x [n, H, D] float64 on the CPU; positions, turns: Python ints. Angles come from whole numbers
    modulo 2^64. Returns the rotated values and their tolerance: bf16's half step, and 2^-20 of the
    pair for an angle off by 10^-7, a sine off by 2^-22 and four fp32 roundings."""
    y, tol = x.clone(), 2.0 ** -8 * x.abs()
    rot = 2 * len(turns)
    for i, p in enumerate(positions):
        for j, f in enumerate(turns):
            t = (p * f) % TWO64
            a = 2 * math.pi * (t / TWO64) * (-1 if inverse else 1)
            u, v = (j, j + rot // 2) if pairs == "halves" else (2 * j, 2 * j + 1)
            c, s = math.cos(a) * scale, math.sin(a) * scale
            y[i, :, u] = x[i, :, u] * c - x[i, :, v] * s
            y[i, :, v] = x[i, :, v] * c + x[i, :, u] * s
            both = 2.0 ** -20 * abs(scale) * (x[i, :, u].abs() + x[i, :, v].abs())
            for d in (u, v):
                tol[i, :, d] = 2.0 ** -8 * y[i, :, d].abs() + both
    return y, tol


def weights_ref(q, lse, k, sm_scale, causal, live, decay, old):
    """One request: q [n, Hq, D], lse [n, Hq], k [T, H, D], old [T, H] or None, all float64. Returns
    the weights [T, H] and their tolerance: scores as kvref.attend_ref has them, the exponential's
    argument in fp32 and 2^-20 of it, sums in fp32."""
    n, Hq, D = q.shape
    T, H = k.shape[:2]
    w, tol = (torch.zeros(T, H, dtype=torch.float64, device=q.device) for _ in range(2))
    pos = torch.arange(T, device=q.device)
    seen = pos[None] <= (T - n + torch.arange(n, device=q.device))[:, None] if causal \
        else torch.ones(n, T, dtype=torch.bool, device=q.device)
    seen = seen & (torch.arange(n, device=q.device) < live)[:, None]
    rows = max(1, live * (Hq // H))
    for h in range(Hq):
        kh = k[:, h // (Hq // H)]
        x = (q[:, h] @ kh.T) * sm_scale
        p = torch.where(seen, torch.exp(x - lse[:, h, None]), torch.zeros_like(x))
        ds = (2.0 ** -18 * q[:, h].abs().amax(1)[:, None] * kh.abs().sum(1)[None]
              + (D + 8) * 2.0 ** -24 * (q[:, h].abs() @ kh.abs().T)) * sm_scale
        arg = 2.0 ** -22 * (x.abs() + lse[:, h, None].abs())
        w[:, h // (Hq // H)] += p.sum(0)
        tol[:, h // (Hq // H)] += torch.where(seen, p * (ds + arg + 2.0 ** -20), torch.zeros_like(x)).sum(0)
    # (fp32 may hold 0 for a number below its smallest normal one: 2^-126 a row)
    tol += rows * (2.0 ** -24 * w + 2.0 ** -126)
    if old is not None:
        fresh = (pos >= T - n)[:, None]
        add = torch.where(fresh, torch.zeros_like(old), decay * old)
        w = w + add
        tol = tol + 2.0 ** -23 * add
    return w, tol


def evict_ref(values, scales, weights, table, to, ctx, budget, sink, recent):
    """values: (k, v) [nb, bs, H, D] float64; scales: (k, v) [nb, H] float64; weights [nb, H, bs];
    tables as lists (to: None for in place). Returns the new ones, kept and new_lens, token by token."""
    values, scales, weights = [v.clone() for v in values], [s.clone() for s in scales], weights.clone()
    was_v, was_s, was_w = [v.clone() for v in values], [s.clone() for s in scales], weights.clone()
    nb, bs, H, _ = values[0].shape
    ok = lambda p: 0 <= p < nb  # noqa: E731
    page_of = lambda row, b: row[b] if b < len(row) and ok(row[b]) else -1  # noqa: E731
    kept, lens = [], []
    for r, n in enumerate(ctx):
        n = min(max(n, 0), len(table[r]) * bs)
        m = min(n, budget)
        lens.append(m)
        row_kept = []
        for h in range(H):
            take = list(range(n))
            if n > budget:
                def weight(t):
                    p = page_of(table[r], t // bs)
                    x = float(was_w[p, h, t % bs]) if p >= 0 else 0.0
                    return (0 if x != x else 1, 0.0 if x != x else -x, t)
                mid = sorted(range(sink, n - recent), key=weight)[:budget - sink - recent]
                take = sorted(list(range(sink)) + mid + list(range(n - recent, n)))
            row_kept.append(take + [-1] * (budget - m))
            dest = table[r] if to is None else to[r]
            for b in range(-(-m // bs)):
                toks = take[b * bs:(b + 1) * bs]
                d = page_of(dest, b)
                if d < 0:
                    continue
                for x, s, wx, ws in zip(values, scales, was_v, was_s):
                    src = [page_of(table[r], t // bs) for t in toks]
                    big = max([float(ws[p, h]) if p >= 0 else 0.0 for p in src])
                    for j, (t, p) in enumerate(zip(toks, src)):
                        f = float(ws[p, h]) if p >= 0 else 0.0
                        x[d, j, h] = kvref.e4m3_round(wx[p, t % bs, h] * (f / big)) if f > 0 else 0.0
                    s[d, h] = big
                for j, t in enumerate(toks):
                    p = page_of(table[r], t // bs)
                    weights[d, h, j] = was_w[p, h, t % bs] if p >= 0 else 0.0
        kept.append(row_kept)
    return values, scales, weights, torch.tensor(kept, dtype=torch.int32).view(len(ctx), H, budget), \
        torch.tensor(lens, dtype=torch.int32)


def cut_ref(row, logits, T, top_k, top_p, min_p):
    """One row (float64): (order, weights in that order and normalised, how many are kept)."""
    x = row.clone()
    if logits:
        x[torch.isnan(x)] = -math.inf
        order = torch.sort(x, descending=True, stable=True).indices
        y = x[order]
        if y[0] == math.inf:
            w = (y == math.inf).double()
        elif y[0] == -math.inf:
            w = torch.zeros_like(y)
        else:
            w = torch.exp((y - y[0]) / min(max(T, 2.0 ** -100), 2.0 ** 100) if T > 0 else y - y[0])
        live = int((y > -math.inf).sum()) if y[0] < math.inf else int(w.sum())
    else:
        x = torch.where(x > 0, x, torch.zeros_like(x)).clamp(max=1)
        order = torch.sort(x, descending=True, stable=True).indices
        w = x[order]
        live = int((w > 0).sum())
    if live == 0:
        return order, torch.zeros_like(w), 0
    if not T > 0:
        top_k, top_p, min_p = 1, 1.0, 0.0
    n = live if top_k <= 0 else min(live, top_k)
    run = torch.cumsum(w, 0)
    if top_p < 1:
        before = run - w
        lead = int((before[:n] < max(top_p, 0.0) * run[n - 1]).sum())
        n = min(n, max(1, lead))
    if min_p > 0:
        n = min(n, max(1, int((w >= min(min_p, 1.0) * w[0]).sum())))
    p = torch.where(torch.arange(w.numel()) < n, w / run[n - 1], torch.zeros_like(w))
    return order, p, n


def draw_ref(order, p, n, u):
    """(token, its probability) of a cut row and a number."""
    if n == 0:
        return 0, 0.0
    run = torch.cumsum(p, 0)
    u = min(u, 1.0) if u > 0 else 0.0
    j = min(int((run[:n] <= u * run[n - 1]).sum()), n - 1)
    return int(order[j]), float(p[j])
