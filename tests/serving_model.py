"""Plain 64-bit model of the serving operators (packed and paged sliding-window attention, cache
appends and reads), written from the definitions in include/ptb.h, and the error bounds that the
tests hold the kernels to.

Bounds.  A rounding to bf16 is off by at most H = 2^-8 of the value (half a step).  The attention
kernels round each softmax weight p to bf16 once before the weighted sum (the 4-bit kernel rounds
p * scale once for the codes and p once for the centres), and the result once:
    |o - o64| <= H |o| + H A + 2 E A,      A = sum_j p_j |v_j|,
where with 4 bits |v| counts scale |u - 8| + |centre|.  E bounds the error of a score
s = q.k * scale in fp32: every one of d products and sums is off by at most 2^-23 of the sum of
magnitudes (tensor-core sums truncate), and so E = (d + 8) 2^-23 max_j sum |q||k| scale; a relative
error E of each weight moves numerator and denominator, hence 2 E.  The 4-bit kernel forms
q.k = sum_w scale_w (q.(64 + u))_w + (centre_w - 72 scale_w) Q_w: magnitudes are counted as
|q| (scale (136 + u) + |centre|).  Q_w, the sum of q over a group, is held in two bf16 terms (off by
2^-16 of it): 2^-16 |Q| (72 scale + |centre|) is added.  q is held in fp16 after scaling its largest
entry into [128, 256): an entry is off by at most 2^-25 / 128 of the largest, which the first term
covers.
"""
import numpy as np
import torch

H = 2.0 ** -8
GROUP = 32


def bf16_np(x):
    """float array -> the nearest bf16 values, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ attention --

def attend(q, k, v, first, window, scale, mag_k=None, mag_v=None, extra=None):
    """q [m, h, d] at positions first.. against k, v [n, kvh, d] (float64): (o, bound) [m, h, d].
    mag_k, mag_v: the magnitudes that the bound counts for keys and values (default |k|, |v|);
    extra [m, h, n]: an absolute error of the unscaled score."""
    m, h, d = q.shape
    n, kvh, _ = k.shape
    g = h // kvh
    mag_k = np.abs(k) if mag_k is None else mag_k
    mag_v = np.abs(v) if mag_v is None else mag_v
    o, bound = np.zeros((m, h, d)), np.zeros((m, h, d))
    for i in range(m):
        p = first + i
        lo, hi = max(0, p - window + 1), min(p, n - 1)
        if p < 0 or lo > hi:
            continue
        for x in range(h):
            kk, vv = k[lo:hi + 1, x // g], v[lo:hi + 1, x // g]
            s = kk @ q[i, x] * scale
            e = (d + 8) * 2.0 ** -23 * (mag_k[lo:hi + 1, x // g] @ np.abs(q[i, x])) * scale
            if extra is not None:
                e = e + extra[i, x, lo:hi + 1] * scale
            e = e.max() + 2.0 ** -21
            w = np.exp(s - s.max())
            w /= w.sum()
            o[i, x] = w @ vv
            a = w @ mag_v[lo:hi + 1, x // g]
            bound[i, x] = H * np.abs(o[i, x]) + (H + 2 * e) * 1.01 * a + 1e-30
    return o, bound


def packed(q, k, v, cu_q, cu_k, window, scale):
    """(o, bound, written) over packed rows; written marks rows of a sequence."""
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    written = np.zeros(q.shape[0], dtype=bool)
    for b in range(len(cu_q) - 1):
        a, z, ka, kz = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        o[a:z], bound[a:z] = attend(q[a:z], k[ka:kz], v[ka:kz], (kz - ka) - (z - a), window, scale)
        written[a:z] = True
    return o, bound, written


# --------------------------------------------------------------------- cache --

def quantize(x):
    """bf16 values (float32) [..., d] -> codes u8 [..., NG, 32], scale, centre (float32), in the
    fp32 steps of the definition."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        rng = np.float32(hi) - np.float32(lo)
        ok = np.isfinite(g).all(-1) & np.isfinite(rng)
        scale = bf16_np(np.where(ok, rng, 0) / np.float32(15))
        centre = bf16_np(np.where(ok, lo, 0) + np.float32(8) * scale)
        div = np.where(scale > 0, scale, np.float32(1))
        u = np.clip(np.rint((np.where(ok[..., None], g, 0) - centre[..., None]) / div[..., None]) + 8, 0, 15)
    u = np.where(ok[..., None], u, 0).astype(np.uint8)
    return u, np.where(ok, scale, np.float32(np.nan)), np.where(ok, centre, np.float32(np.nan))


def key_nibble(c, d):
    return 8 * ((c % 32) // 8 * (d // 32) + c // 32) + c % 8


def value_nibble(c, d):
    return (d // 8) * ((c % 32) // 4) + 4 * (c // 32) + c % 4


class Cache:
    """A host image of a cache in the documented byte layout."""

    def __init__(self, raw, kv_heads, page, d, bits):
        self.raw, self.kv, self.page, self.d, self.bits = raw, kv_heads, page, d, bits
        self.row = 2 * d if bits == 16 else d // 2 + d // 8

    def block(self, page, head, which):
        n = self.page * self.row
        at = (which * self.kv + head) * n
        return self.raw[page, at:at + n]

    def put(self, page, off, head, which, x):
        """x: bf16 values (float32) [d]."""
        b, d = self.block(page, head, which), self.d
        if self.bits == 16:
            b[off * 2 * d:(off + 1) * 2 * d] = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.uint8).numpy()
            return
        u, scale, centre = quantize(x)
        u = u.reshape(-1)
        row = np.zeros(d // 2, np.uint8)
        for c in range(d):
            at = key_nibble(c, d) if which == 0 else value_nibble(c, d)
            row[at // 2] |= u[c] << (4 * (at % 2))
        b[off * (d // 2):(off + 1) * (d // 2)] = row
        pair = np.stack([scale, centre], -1).reshape(-1)
        t = torch.from_numpy(pair.astype(np.float32)).to(torch.bfloat16)
        t[torch.isnan(t)] = torch.tensor([0x7fc0], dtype=torch.int16).view(torch.bfloat16)[0]
        at = self.page * (d // 2) + off * (d // 8)
        b[at:at + d // 8] = t.view(torch.uint8).numpy()

    def get(self, page, off, head, which):
        """(value [d], magnitudes: scale |u - 8| and |centre| per channel, scale, centre, code)"""
        b, d = self.block(page, head, which), self.d
        if self.bits == 16:
            x = torch.from_numpy(b[off * 2 * d:(off + 1) * 2 * d].copy()).view(torch.bfloat16).double().numpy()
            return x, None, None, None
        row = b[off * (d // 2):(off + 1) * (d // 2)]
        at = self.page * (d // 2) + off * (d // 8)
        pair = torch.from_numpy(b[at:at + d // 8].copy()).view(torch.bfloat16).double().numpy().reshape(-1, 2)
        place = np.array([key_nibble(c, d) if which == 0 else value_nibble(c, d) for c in range(d)])
        u = ((row[place // 2] >> (4 * (place % 2))) & 15).astype(np.float64)
        s, z = np.repeat(pair[:, 0], 32), np.repeat(pair[:, 1], 32)
        return z + s * (u - 8), u, s, z


def paged(q, cache, table, lens, window, scale):
    """One query row per sequence: (o, bound) [B, h, d]."""
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    kv, d = cache.kv, cache.d
    for b, n in enumerate(lens):
        lo = max(0, n - window)
        if n <= 0:
            continue
        k, v = np.zeros((n - lo, kv, d)), np.zeros((n - lo, kv, d))
        mk, mv = np.zeros_like(k), np.zeros_like(v)
        extra = np.zeros((1, q.shape[1], n - lo)) if cache.bits == 4 else None
        g = q.shape[1] // kv
        for j in range(lo, n):
            page, off = table[b][j // cache.page], j % cache.page
            for h in range(kv):
                k[j - lo, h], u, s, z = cache.get(page, off, h, 0)
                if u is None:
                    mk[j - lo, h] = np.abs(k[j - lo, h])
                else:
                    mk[j - lo, h] = s * (136 + u) + np.abs(z)
                    for x in range(h * g, (h + 1) * g):
                        qs = np.abs(q[b, x].reshape(-1, 32).sum(-1))
                        extra[0, x, j - lo] = 2.0 ** -16 * (qs * (72 * s + np.abs(z)).reshape(-1, 32)[:, 0]).sum()
                v[j - lo, h], u, s, z = cache.get(page, off, h, 1)
                mv[j - lo, h] = np.abs(v[j - lo, h]) if u is None else s * np.abs(u - 8) + np.abs(z)
        ob, bb = attend(q[b:b + 1], k, v, n - lo - 1, n, scale, mk, mv, extra)
        o[b], bound[b] = ob[0], bb[0]
    return o, bound


def rotate32(x, cos, sin, interleaved):
    """The rotation in its fp32 steps, rounded to bf16: x float32 [..., d], cos / sin [rot / 2]."""
    r = 2 * len(cos)
    y = np.asarray(x, np.float32).copy()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = np.float32(a), np.float32(b)
    with np.errstate(all="ignore"):
        u, w = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = u, w
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, w
    return bf16_np(y)
