"""The softmax-attention operators from their formulas in 64 bits (CPU, plain loops over sequences and
new tokens), with the error bounds their tests use.

Bounds.  A rounding is off by at most half a step: BF16 = 2^-8, E4M3 = 2^-4 relative.  fp32 chains
are counted in units of F32 = 2^-24 per operation, against the sum of the terms' magnitudes.
"""
import math

import torch

BF16, E4M3, F32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24
SCALE_FLOOR = 2.0 ** -64


def table(rot, n, base=10000.0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pairs(rot, interleaved):
    h = rot // 2
    if interleaved:
        return [(2 * i, 2 * i + 1, i) for i in range(h)]
    return [(i, i + h, i) for i in range(h)]


def rotate(n, cos_sin, positions, interleaved, back=False):
    """fp64 n [tokens, heads, d] rotated; returns the result and the magnitudes of its terms."""
    y, mag = n.clone(), n.abs()
    if cos_sin is None:
        return y, mag
    rot = cos_sin.shape[1]
    cs = cos_sin.double()[positions.long()]
    for a, b, i in _pairs(rot, interleaved):
        c, s = cs[:, None, i], cs[:, None, rot // 2 + i] * (-1 if back else 1)
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        mag[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
        mag[..., b] = (n[..., b] * c).abs() + (n[..., a] * s).abs()
    return y, mag


def norm_rope(x, w, eps, cos_sin, positions, interleaved):
    x = x.double()
    n = x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    return rotate(n, cos_sin, positions, interleaved)


# fp32 operations behind one value before its last rounding: the sum of squares (d / 16 .. 8 terms a
# lane, 4 shuffles), the mean, eps, the reciprocal root (2 units in the last place), three products
# and the rotation's three: below 32 units
CHAIN = 32 * F32


def norm_rope_tol(y, mag):
    return BF16 * y.abs() + (1 + BF16) * CHAIN * mag + 1e-38


def norm_rope_bwd(x, w, eps, cos_sin, positions, interleaved, dy):
    """dx, dw, and the tolerances of both."""
    x, dy = x.double(), dy.double()
    g, gmag = rotate(dy, cos_sin, positions, interleaved, back=True)
    if w is None:
        return g, None, BF16 * g.abs() + CHAIN * gmag + 1e-38, None
    d = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u, umag = g * w.double(), gmag * w.double().abs()
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    mag = r * (umag + x.abs() * r * r * (umag * x.abs()).sum(-1, keepdim=True) / d)
    dw = (g * x * r).sum((0, 1))
    # a lane adds its rows, a block its lanes, the last launch the blocks: below 64 additions in a row
    # at the sizes tested, after the chain of each term
    dw_tol = (64 * F32 + CHAIN) * (gmag * x.abs() * r).sum((0, 1)) + 1e-38
    return dx, dw, BF16 * dx.abs() + 2 * CHAIN * mag + 1e-38, dw_tol


def cached_rows(cache, scale, pages, length):
    """fp64 [length, hk, d]: the values a sequence's rows stand for (CPU tensors)."""
    x = cache[pages].double() if scale is None else cache[pages].float().double() * scale[pages].double()[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:length]


def attention(q, k_cache, v_cache, page_table, lens, scale, k_scale=None, v_scale=None, softcap=0.0, window=0):
    """out, lse and their tolerances (fp64), from CPU tensors; q [b, new, hq, d]."""
    b_n, new, hq, d = q.shape
    hk, page = k_cache.shape[1], k_cache.shape[2]
    group = hq // hk
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(b_n):
        n = int(lens[b])
        for t in range(new):
            last = n - new + t + 1
            first = max(0, last - window) if window else 0
            if last <= first:
                continue
            lo_page = first // page
            pages = page_table[b, lo_page:-(-last // page)].long()
            cut = slice(first - lo_page * page, last - lo_page * page)
            k = cached_rows(k_cache, k_scale, pages, 1 << 40)[cut]
            v = cached_rows(v_cache, v_scale, pages, 1 << 40)[cut]
            qt = q[b, t].double().view(hk, group, d)
            z = torch.einsum("hgd,jhd->hgj", qt, k) * scale
            zmag = torch.einsum("hgd,jhd->hgj", qt.abs(), k.abs()) * abs(scale)
            # scores: d products accumulated in fp32 (the tensor core's sum may drop twice a rounding),
            # and a few roundings of z in base 2; a cap's tanh is 1 - 2 / (e^2x + 1): 4 roundings of 1
            dz = 2 * (d + 8) * F32 * zmag + 8 * F32 * z.abs()
            if softcap:
                z = softcap * torch.tanh(z / softcap)
                dz = dz + 16 * F32 * softcap
            m = z.max(-1, keepdim=True).values
            dz = dz + 8 * F32 * (z.abs() + m.abs())  # the difference, and the logarithm of an e4m3 scale
            p = torch.exp(z - m)
            l = p.sum(-1, keepdim=True)
            o = torch.einsum("hgj,jhd->hgd", p, v) / l
            # a weight's relative error: twice its score's (numerator and sum), the exponentials'
            # approximation (2^-21), the rounding of P (bf16 pair 2^-16; fp16 for an e4m3 cache 2^-11), and
            # fp32 sums over the keys
            count = last - first
            rel = 2 * dz + 2.0 ** -20 + (2.0 ** -11 if k_scale is not None else 2.0 ** -16) + 2 * (count + 300) * F32
            dz_l = (p * dz).sum(-1, keepdim=True) / l  # the sum's part of it
            tol = torch.einsum("hgj,jhd->hgd", p * (rel + dz_l), v.abs()) / l
            # fp16 weights are p s 2^7 in units of a reference that is at most the largest p s; where they are
            # subnormal they are off by up to 2^-25, which is 2^-32 of the largest p s, times a code: 2^-32 of the
            # largest value for each key (l >= 1)
            if k_scale is not None:
                big = (v.abs().amax((0, 2)))[:, None, None]
                tol = tol + count * 2.0 ** -32 * big
            out[b, t] = o.reshape(hq, d)
            out_tol[b, t] = (BF16 * o.abs() + (1 + BF16) * tol).reshape(hq, d) + 1e-38
            lse[b, t] = (m + torch.log(l)).flatten()
            lse_tol[b, t] = ((p * (dz + 2.0 ** -21)).sum(-1) / l.squeeze(-1) + 4 * F32 * (m.abs().squeeze(-1) + 30)
                             + (count + 300) * F32).flatten()
    return out, lse, out_tol, lse_tol


def make_cache(gen, pages, hk, page, d, quant, fill=float("nan")):
    """An unwritten pool: every row is `fill` (a quantised one: codes 0x7f or 0, scales `fill`)."""
    if not quant:
        return torch.full((pages, hk, page, d), fill, dtype=torch.bfloat16), None
    codes = torch.full((pages, hk, page, d), 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return codes, torch.full((pages, hk, page), fill, dtype=torch.float32)


def quantise(x):
    """e4m3 codes and scales of fp32 rows, in fp32 as the definition says."""
    s = (x.abs().amax(-1) / 448).clamp(min=SCALE_FLOOR)
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def fill_sequences(gen, lens, k_cache, v_cache, k_scale, v_scale, first=None, k_std=1.0, v_std=1.0, max_pages=None):
    """Writes random rows of every sequence to pages in random order; returns the page table (unused entries -1).
    With `first`, sequence b's tokens before first[b] and their pages are left unwritten."""
    pages, hk, page, d = k_cache.shape
    wide = max([-(-int(n) // page) for n in lens] + [1]) if max_pages is None else max_pages
    tab = torch.full((len(lens), wide), -1, dtype=torch.int32)
    free = torch.randperm(pages, generator=gen).tolist()
    for b, n in enumerate(lens):
        f = 0 if first is None else int(first[b])
        for i in range(f // page, -(-int(n) // page)):
            tab[b, i] = free.pop()
        for j in range(f, int(n)):
            p, r = int(tab[b, j // page]), j % page
            for cache, scale, std in ((k_cache, k_scale, k_std), (v_cache, v_scale, v_std)):
                x = torch.randn(hk, d, generator=gen) * std
                if scale is None:
                    cache[p, :, r] = x.to(torch.bfloat16)
                else:
                    c, s = quantise(x)
                    cache.view(torch.uint8)[p, :, r] = c.view(torch.uint8)
                    scale[p, :, r] = s
    return tab
