"""Plain forms of the paged 8-bit cache's operators, for the tests: 64-bit arithmetic on small
inputs, and builders of caches, tables and prefixes."""

import math

import torch

E4M3 = torch.float8_e4m3fn


def e4m3_round(y):
    """y (float64) to the nearest e4m3 value, halves to even; +-448 beyond; NaN stays."""
    m, e = torch.frexp(torch.where(torch.isfinite(y), y, torch.ones_like(y)))
    step = torch.tensor([2.0 ** i for i in range(-20, 1000)], dtype=torch.float64,
                        device=y.device)[((e - 1).clamp(min=-6) - 3 + 20).clamp(max=1019).long()]
    r = torch.round(y / step) * step
    r = r.clamp(-448, 448)
    return torch.where(torch.isnan(y), y, torch.where(torch.isinf(y), torch.sign(y) * 448, r))


def pow2_scale(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s, for one Python float."""
    k = -100
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def write_ref(x, slots, values, scale):
    """values [nb, bs, H, D] (e4m3 values in float64) and scale [nb, H] float64, on the CPU, after
    sd_kv_write of x [n, H, D] (float64): slot by slot, as the definition reads."""
    values, scale = values.clone(), scale.clone()
    nb, bs, H, D = values.shape
    by_page = {}
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < nb * bs:
            by_page.setdefault(s // bs, {})[s % bs] = i
    for page, toks in by_page.items():
        for h in range(H):
            new = torch.stack([x[i, h] for i in toks.values()])
            fin = new[torch.isfinite(new)]
            amax = float(fin.abs().max()) if fin.numel() else 0.0
            old = float(scale[page, h])
            held = 0.0 if 0 in toks or not old > 0 else old
            s = max(held, pow2_scale(amax))
            if 0 not in toks and s != old:
                values[page, :, h] = e4m3_round(values[page, :, h] * ((old if old > 0 else 0.0) / s))
            for off, i in toks.items():
                values[page, off, h] = e4m3_round(x[i, h] / s)
            scale[page, h] = s
    return values, scale


def make_cache(nb, bs, H, D, gen, device, layout="token", spread=0.5):
    """(k, v, k_scale, v_scale): filled caches. layout "head": [nb, H, bs, D] in memory."""
    out = []
    for _ in range(2):
        x = torch.randn(nb, bs, H, D, generator=gen, device=device)
        x *= torch.exp(spread * torch.randn(nb, 1, H, 1, generator=gen, device=device))
        k = torch.ceil(torch.log2(x.abs().amax(dim=(1, 3)) / 448)).to(torch.int32)
        s = ((k + 127) << 23).view(torch.float32)  # 2^k exactly
        q = (x / s[:, None, :, None]).clamp(-448, 448).to(E4M3)
        if layout == "head":
            q = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        out += [q, s.contiguous()]
    return out[0], out[2], out[1], out[3]


def make_table(lens, bs, gen, device, extra=2):
    """(num_blocks, block_table): shuffled pages for lens[r] tokens each, -1 beyond."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + extra
    perm = torch.randperm(nb, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32,
                       device=device)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return nb, table


def prefix(counts, device):
    t = torch.tensor([0] + list(counts))
    return t.cumsum(0).to(torch.int32).to(device)


def held(cache, scale, table_row, n):
    """The n first tokens of a request, float64 [n, H, D]."""
    bs = cache.shape[1]
    page = table_row[:-(-n // bs)].long()
    x = cache.view(torch.uint8)[page].view(E4M3).double()
    return (x * scale[page].double()[:, None, :, None]).flatten(0, 1)[:n]


def attend_ref(q, k, v, sm_scale, causal, hide=None):
    """One request in 64 bits: q [n, Hq, D] float64, k, v [T, H, D] float64; hide [T]: tokens left
    out. Returns out, lse and the tolerances of both: each weight off by half a step of 8 bits or
    2^-18 of the row's largest, q by 2^-18 of its largest, products and sums in fp32, out rounded
    to bf16 once."""
    n, Hq, D = q.shape
    T, H = k.shape[:2]
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros(n, Hq, dtype=torch.float64, device=q.device)
    if T == 0 or n == 0:
        return out, lse, tol, tol_lse
    pos = torch.arange(T, device=q.device)[None]
    seen = pos <= (T - n + torch.arange(n, device=q.device))[:, None] if causal \
        else torch.ones(n, T, dtype=torch.bool, device=q.device)
    if hide is not None:
        seen = seen & ~hide[None]
    some = seen.any(1)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
        kf = torch.where(torch.isfinite(kh), kh, torch.zeros_like(kh))
        x = (q[:, h] @ kf.T) * sm_scale
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        m = torch.where(some, x.amax(1), torch.zeros(n, dtype=x.dtype, device=x.device))
        e = torch.exp(x - m[:, None])
        z = e.sum(1)
        p = e / torch.where(z > 0, z, torch.ones_like(z))[:, None]
        vis = seen.any(0)
        vf = torch.where(vis[:, None], vh, torch.zeros_like(vh))
        vf = torch.where(torch.isfinite(vf), vf, torch.zeros_like(vf))
        o = p @ vf
        a = p @ vf.abs()
        ds = (2.0 ** -18 * q[:, h].abs().amax(1)[:, None] * kf.abs().sum(1)[None]
              + (D + 8) * 2.0 ** -24 * (q[:, h].abs() @ kf.abs().T)) * sm_scale
        ds = torch.where(seen, ds, torch.zeros_like(ds)).amax(1)
        fp32 = 2.0 ** -20 + T * 2.0 ** -24
        out[:, h] = o
        lse[:, h] = torch.where(some, m + torch.log(z), torch.full_like(m, -math.inf))
        tol[:, h] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * ds + fp32)[:, None] * a \
            + 2.0 ** -18 * (p.amax(1)[:, None] * vf.abs().sum(0)[None])
        tol_lse[:, h] = ds + fp32 + 2.0 ** -22 * torch.where(some, lse[:, h], torch.zeros_like(m)).abs()
    return out, lse, tol, tol_lse
