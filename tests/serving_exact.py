"""Attention of single tokens over a whole paged cache in 64 bits, vectorised (torch, any device),
and its error bound for the arithmetic of csrc/swa_paged.cu; from the definitions in include/ptb.h.

Bound.  H = 2^-8 is half a step of bf16.  A score is q.k scale in fp32, each product and partial sum
off by at most 2^-23 of the sum of magnitudes (tensor-core sums truncate):
    e = (d + 8) 2^-23 max_j sum |q| mag_k scale + x,
with mag_k = |k| in bf16.  With 4 bits q.k = sum_w scale_w (q.u)_w + (centre_w - 8 scale_w) Q_w, so
mag_k = scale (u + 8) + |centre|, and x counts, per key and times the score's scale:
    Q_w, the sum of q over a group, is held in two bf16 terms, each off by H of what it rounds:
        H^2 |Q_w| (8 scale_w + |centre_w|);
    q is held in fp16 with its largest entry in [2^14, 2^15), half the channels 2^-4 of that: below
    2^-14 an entry is off by 2^-25, in units of the largest 2^-39 or 2^-35: 2^-35 max |q| 15 scale.
exp2 and the factor log2(e) scale add 2^-21.  Weights off by a relative e move numerator and
denominator: 2 e A, A = sum_j p_j |v_j|.  Weights are rounded once before the weighted sum (4 bits:
p scale once for the codes, p once for the centres, |v| counts as scale |u - 8| + |centre|) but not
in their own sum: H B, where B = A less the term of the key with the largest score in the paged
kernel (it is the reference of its part of the row: its weight there is 1, and 1 and a scale are bf16
numbers), B = A in the packed one.  Both sums run over n keys in fp32: (n + d) 2^-22 A.  The output is
rounded:
    |o - o64| <= H |o64| + 1.01 (H B + (2 e + (n + d) 2^-22) A).

Over thousands of keys that bound is far above a row's real error, and above what a lost block of
keys changes.  For values that are independent and centred at zero the length of a row says more:
|o64|^2 is sum p_j^2 |v_j|^2 on average, the roundings of the weights (independent, at most H each)
add at most H^2 of that, the output's at most H |o64|, and so |o - o64| <= 2 H |o64|; the limit is
ROW_LIMIT = 3 H.  One key lost of n weighs n^-1/2 of the row: 1.3 ROW_LIMIT at 4000.
"""
import torch

H = 2.0 ** -8
ROW_LIMIT = 3 * H


def row_error(o, want):
    """The largest error of a row [..., d] relative to its length (rows of zeros have to be zeros)."""
    err, size = (o - want).norm(dim=-1), want.norm(dim=-1)
    return float(torch.where(size > 0, err / size.clamp(min=1e-300), err * 1e300).max())


def nibble_of_channel(d, keys):
    """Which nibble of a row holds channel c: the orders of include/ptb.h."""
    ng = d // 32
    c = torch.arange(d)
    w, r = c // 32, c % 32
    return 8 * (r // 8 * ng + w) + r % 8 if keys else (d // 8) * (r // 4) + 4 * w + r % 4


def rows64(cache, pages, offs, kv, page, d, bits, which):
    """Rows `offs` of pages `pages` (index tensors [n]) of every kv head, keys (0) or values (1):
    values [n, kv, d] in float64 and, with 4 bits, (u, scale, centre) per channel."""
    block = cache.view(cache.shape[0], 2, kv, -1)[pages, which]  # [n, kv, bytes]
    n = block.shape[0]
    if bits == 16:
        rows = block.reshape(n, kv, page, 2 * d)[torch.arange(n, device=cache.device), :, offs]
        return rows.contiguous().view(torch.bfloat16).double(), None
    pick = torch.arange(n, device=cache.device)
    codes = block[..., : page * d // 2].reshape(n, kv, page, d // 2)[pick, :, offs]
    pairs = block[..., page * d // 2:].reshape(n, kv, page, d // 8)[pick, :, offs]
    pairs = pairs.contiguous().view(torch.bfloat16).double().unflatten(-1, (-1, 2))
    place = nibble_of_channel(d, which == 0).to(cache.device)
    u = ((codes[..., place // 2] >> (4 * (place % 2)).to(torch.uint8)) & 15).double()
    scale, centre = (pairs[..., i].repeat_interleave(32, -1) for i in (0, 1))
    return centre + scale * (u - 8), (u, scale, centre)


def paged(q, cache, table, lens, kv, page, bits, window, scale):
    """q [B, heads, d] -> (o, bound) [B, heads, d] in float64, on q's device; lens: a list."""
    batch, heads, d = q.shape
    g = heads // kv
    o = torch.zeros(batch, heads, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for b, n in enumerate(lens):
        lo = max(0, n - window)
        if n <= 0:
            continue
        at = torch.arange(lo, n, device=q.device)
        pages, offs = table[b][at // page].long(), at % page
        k, kc = rows64(cache, pages, offs, kv, page, d, bits, 0)
        v, vc = rows64(cache, pages, offs, kv, page, d, bits, 1)
        x = q[b].double().view(kv, g, d)
        s = torch.einsum("hgd,nhd->hgn", x, k) * scale
        if kc is None:
            mag_k, mag_v, extra = k.abs(), v.abs(), 0.0
        else:
            u, sc, ce = kc
            mag_k = sc * (8 + u) + ce.abs()
            mag_v = vc[1] * (vc[0] - 8).abs() + vc[2].abs()
            group_sum = x.unflatten(-1, (-1, 32)).sum(-1).abs()
            extra = H * H * torch.einsum("hgw,nhw->hgn", group_sum, (8 * sc + ce.abs())[..., ::32])
            extra += 2.0 ** -35 * 15 * x.abs().amax(-1)[..., None] * sc.sum(-1).T[:, None]
        e = ((d + 8) * 2.0 ** -23 * torch.einsum("hgd,nhd->hgn", x.abs(), mag_k) + extra) * scale
        e = e.amax(-1) + 2.0 ** -21
        p = torch.softmax(s, -1)
        o[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(heads, d)
        a = torch.einsum("hgn,nhd->hgd", p, mag_v).reshape(heads, d)
        top = p.argmax(-1, keepdim=True)  # [kv, g, 1]
        of_top = torch.gather(mag_v.transpose(0, 1), 1, top.expand(-1, -1, d)) * p.gather(-1, top)
        rest = (a - of_top.reshape(heads, d)).clamp(min=0)
        bound[b] = H * o[b].abs() + 1.01 * (H * rest + (2 * e.reshape(heads, 1) + (n - lo + d) * 2.0 ** -22) * a) + 1e-30
    return o, bound


def packed(q, k, v, cu_q, cu_k, window, scale):
    """q [Tq, heads, d], k, v [Tk, kv, d] -> (o, bound, written): float64 on q's device, and which
    rows belong to a sequence.  Query i of nq is at position nk - nq + i."""
    heads, d = q.shape[1:]
    kv = k.shape[1]
    g = heads // kv
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    written = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        m, n = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        written[rows] = True
        if m == 0 or n == 0:
            continue
        x, kk, vv = q[rows].double().view(m, kv, g, d), k[keys].double(), v[keys].double()
        p = n - m + torch.arange(m, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)
        seen = ((j <= p) & (p - j < window))[:, None, None]
        s = (torch.einsum("mhgd,nhd->mhgn", x, kk) * scale).masked_fill(~seen, float("-inf"))
        some = seen.any(-1, keepdim=True)
        w = torch.where(some, torch.softmax(torch.where(some, s, torch.zeros_like(s)), -1), torch.zeros_like(s))
        e = (d + 8) * 2.0 ** -23 * torch.einsum("mhgd,nhd->mhgn", x.abs(), kk.abs()) * scale
        e = torch.where(seen, e, torch.zeros_like(e)).amax(-1, keepdim=True) + 2.0 ** -21
        o[rows] = torch.einsum("mhgn,nhd->mhgd", w, vv).reshape(m, heads, d)
        a = torch.einsum("mhgn,nhd->mhgd", w, vv.abs())
        bound[rows] = H * o[rows].abs() + (1.01 * (H + 2 * e + (min(n, window) + d) * 2.0 ** -22) * a).reshape(m, heads, d) + 1e-30
    return o, bound, written
