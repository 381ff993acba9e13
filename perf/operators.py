"""Timed cases of the serving operators: attention over packed prompts, attention of one new token
per sequence over a paged cache (bf16 or 4-bit), and the appends to that cache and reads from it.

`run` computes a case with elementary torch operations in fp32, or, with `own` set, through the
calls of block_sliding_window_gb300 that a serving program makes.  `exact` is the definition in
64 bits, written apart from both.

The cache is one uint8 tensor [pages, page_bytes].  A page holds, for keys and then for values and
for each kv head, a block of `page` token rows:
  bits 16   [page][d] bf16;
  bits  4   [page][d / 2] bytes of codes, then [page][d / 32] pairs (scale, centre) of bf16.  Value
            of a code u in 0..15: centre + scale * (u - 8), one pair for 32 neighbouring channels.
            Codes are stored low nibble first; channel 32 w + 8 t + e of a key is nibble
            8 (t NG + w) + e of its row (NG = d / 32), channel 32 w + 4 g + e of a value is nibble
            (d / 8) g + 4 w + e.
"""
import math
import random

import torch

own = False

GROUP = 32


# ------------------------------------------------------------------------------------- the cases --

def listed():
    prefill = dict(kind="prefill")
    decode = dict(kind="decode")
    append = dict(kind="append")
    return [
        # One short prompt on the heads of the 13B-class layer: latency.
        dict(prefill, name="prefill_1x37_h40", n=1, lo=37, hi=37, kv=40, group=1, d=128, window=512),
        # A ragged batch of prompts, grouped heads, the 13B-class window.
        dict(prefill, name="prefill_64_ragged_h64kv8", n=64, lo=9, hi=1000, kv=8, group=8, d=128, window=512),
        # Four prompts of the 175B-shaped layer: 128 heads of 96, window 1024.
        dict(prefill, name="prefill_4_175b_heads", n=4, lo=300, hi=2048, kv=128, group=1, d=96, window=1024),
        # One long prompt under plain causal attention.
        dict(prefill, name="prefill_1x16001_causal", n=1, lo=16001, hi=16001, kv=2, group=8, d=128, window=1 << 20),
        # One sequence answering on the 13B-class heads: latency.
        dict(decode, name="decode16_1x2000_h40", n=1, lo=2000, hi=2000, kv=40, group=1, d=128, window=2048, bits=16, page=64),
        # A full batch of sequences of many lengths.
        dict(decode, name="decode16_64_ragged_h64kv8", n=64, lo=500, hi=8192, kv=8, group=8, d=128, window=1 << 20, bits=16, page=64),
        # One sequence with a long 4-bit cache: few rows, so the keys have to be split.
        dict(decode, name="decode4_1x16000_h32kv4", n=1, lo=16000, hi=16000, kv=4, group=8, d=128, window=1 << 20, bits=4, page=32),
        # The largest batch on a 4-bit cache.
        dict(decode, name="decode4_64_long_h64kv8", n=64, lo=6000, hi=16384, kv=8, group=8, d=128, window=1 << 20, bits=4, page=64),
        # Sliding window over long sequences on heads of 96 (the pages before the window are gone).
        dict(decode, name="decode4_96_window_h128kv16_d96", n=96, lo=200, hi=32768, kv=16, group=8, d=96, window=1024, bits=4, page=16),
        # One decode step's append for 64 sequences, and the new rows read back.
        dict(append, name="append4_64_tokens", n=64, lo=1, hi=1, past=5000, heads=64, kv=8, d=128, rot=128, pairs=False, bits=4, page=64, keys=False),
        # Whole prompts into a bf16 cache, rotated keys kept for the prompt's attention.
        dict(append, name="append16_prompts_8k", n=12, lo=100, hi=2048, past=0, heads=64, kv=8, d=128, rot=128, pairs=False, bits=16, page=64, keys=True),
        # Later chunks of prompts into a 4-bit cache, rotation of half the channels, read back.
        dict(append, name="append4_prompts_16k", n=24, lo=300, hi=1500, past=700, heads=32, kv=32, d=64, rot=32, pairs=True, bits=4, page=16, keys=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        kind = rng.choice(["prefill", "decode", "decode", "append"])
        d = rng.choice([32, 64, 96, 128, 128])
        kv = rng.choice([1, 2, 3, 4, 8, 8, 10, 16, 40])
        group = rng.choice([1, 1, 2, 3, 4, 5, 8, 8, 16])
        n = _log(rng, 1, 96)
        if kind == "prefill":
            hi = _log(rng, 1, 8192)
            lo = _log(rng, 1, hi)
            case = dict(kind=kind, n=n, lo=lo, hi=hi, kv=kv, group=group, d=d, window=_log(rng, 1, 16384))
            if n * kv * group * hi * hi > 3e9 or n * hi > 40000 or work(case)["flops"] > 1e12:
                continue
        elif kind == "decode":
            hi = _log(rng, 1, 32768)
            lo = _log(rng, 1, hi)
            case = dict(kind=kind, n=n, lo=lo, hi=hi, kv=kv, group=group, d=d, window=_log(rng, 1, 65536),
                        bits=rng.choice([16, 4, 4]), page=rng.choice([16, 32, 64, 128]))
            if n * kv * d * min(hi, case["window"]) > 1e9:
                continue
        else:
            hi = _log(rng, 1, 4096)
            lo = _log(rng, 1, hi)
            case = dict(kind=kind, n=n, lo=lo, hi=hi, past=rng.choice([0, 1, 15, _log(rng, 1, 20000)]), heads=kv * group, kv=kv, d=d,
                        rot=rng.choice([0, 32, d, d]), pairs=rng.random() < 0.4, bits=rng.choice([16, 4, 4]),
                        page=rng.choice([16, 32, 64, 128]), keys=rng.random() < 0.5)
            if n * hi * (kv * group + 2 * kv) * d > 1.5e8 or n * (hi + case["past"]) * kv * d > 5e8:
                continue
        return case


def _lengths(c):
    """The sequences' lengths: spread over [lo, hi] by their logarithm, the same for every seed."""
    r = random.Random("%d-%d-%d" % (c["n"], c["lo"], c["hi"]))
    return [_log(r, c["lo"], c["hi"]) for _ in range(c["n"])]


def _row_bytes(c):
    return 2 * c["d"] if c["bits"] == 16 else c["d"] // 2 + 4 * (c["d"] // GROUP)


def work(c):
    """Bytes and operations that a pass cannot do without."""
    ls, d = _lengths(c), c["d"]
    if c["kind"] == "prefill":
        heads, w = c["kv"] * c["group"], c["window"]
        pairs = sum(m * (m + 1) // 2 + (n - m) * m for n in ls for m in [min(n, w)])
        return {"bytes": 4.0 * sum(ls) * d * (heads + c["kv"]), "flops": 4.0 * d * heads * pairs}
    if c["kind"] == "decode":
        heads, keys = c["kv"] * c["group"], sum(min(n, c["window"]) for n in ls)
        return {"bytes": 2.0 * keys * c["kv"] * _row_bytes(c) + 4.0 * c["n"] * heads * d, "flops": 4.0 * d * heads * keys}
    t, rows = sum(ls), c["heads"] + c["kv"] * c["keys"]
    b = 2.0 * t * d * (c["heads"] + 2 * c["kv"]) + 2.0 * t * d * rows + 2.0 * t * c["kv"] * _row_bytes(c) + 4.0 * t * c["rot"]
    if c["bits"] == 4:  # the rows read back: codes in, bf16 out
        b += 2.0 * t * c["kv"] * (_row_bytes(c) + 2 * d)
    return {"bytes": b, "flops": 6.0 * t * d * (c["heads"] + 2 * c["kv"])}


# ------------------------------------------------------------------------------------ the inputs --

def _normal(gen, *shape, dtype=torch.bfloat16):
    """N(0, 1) values with a spread of channel sizes, as keys and values of a trained layer have."""
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)
    return x.mul_(torch.exp2(torch.linspace(-1, 1, shape[-1], device="cuda")).to(dtype))


def _blocks(c, cache):
    """The codes and the pairs of a 4-bit cache as views [pages, 2, kv, page, .], or its bf16 rows."""
    p, kv, d = c["page"], c["kv"], c["d"]
    if c["bits"] == 16:
        return cache.view(torch.bfloat16).view(-1, 2, kv, p, d), None
    b = cache.view(-1, 2, kv, p * _row_bytes(c))
    codes, pairs = b[..., : p * d // 2], b[..., p * d // 2 :]
    return codes.unflatten(-1, (p, d // 2)), pairs.unflatten(-1, (p, d // GROUP * 4))


def _to_codes(x):
    """bf16 values [..., d] -> (u, scale, centre): the 4-bit form, by fp32 arithmetic."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / 15).to(torch.bfloat16)
    s = scale.float()
    centre = (lo + 8 * s).to(torch.bfloat16)
    z = centre.float()
    u = (torch.round((g - z.unsqueeze(-1)) / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)) + 8).clamp_(0, 15)
    return u.to(torch.uint8), scale, centre


def _pack(u, keys):
    """Codes [..., NG, 32] -> the bytes [..., d / 2] of a row."""
    u = u.unflatten(-1, (4, 8)).transpose(-3, -2) if keys else u.unflatten(-1, (8, 4)).transpose(-3, -2)
    u = u.flatten(-3).unflatten(-1, (-1, 2))
    return u[..., 0] | (u[..., 1] << 4)


def _unpack(b, keys):
    """The bytes [..., d / 2] of a row -> codes [..., NG, 32]."""
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    ng = u.shape[-1] // GROUP
    u = u.unflatten(-1, (4, ng, 8)) if keys else u.unflatten(-1, (8, ng, 4))
    return u.transpose(-3, -2).flatten(-2)


def _pair_bytes(scale, centre):
    return torch.stack([scale, centre], -1).flatten(-2).contiguous().view(torch.uint8)


def _filled_cache(c, gen, pages):
    cache = torch.empty(pages, 2 * c["kv"] * c["page"] * _row_bytes(c), dtype=torch.uint8, device="cuda")
    codes, pairs = _blocks(c, cache)
    if pairs is None:
        codes.copy_(_normal(gen, *codes.shape))
        return cache
    for i, keys in ((0, True), (1, False)):
        u, scale, centre = _to_codes(_normal(gen, pages, c["kv"], c["page"], c["d"]))
        codes[:, i] = _pack(u, keys)
        pairs[:, i] = _pair_bytes(scale, centre)
    return cache


def _table(c, gen, first, last):
    """Pages of the positions first..last-1 of every sequence, scattered over the cache; page 0 stands
    for pages that are no longer there."""
    p = c["page"]
    spans = [(a // p, -(-b // p)) for a, b in zip(first, last)]
    total = sum(j - i for i, j in spans) + 1
    order = (torch.randperm(total - 1, generator=gen, device="cuda") + 1).to(torch.int32)
    table = torch.zeros(len(spans), max(1, max(j for _, j in spans)), dtype=torch.int32, device="cuda")
    at = 0
    for b, (i, j) in enumerate(spans):
        table[b, i:j] = order[at : at + j - i]
        at += j - i
    return table, total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cumulated(ls):
    out = [0]
    for n in ls:
        out.append(out[-1] + n)
    return out


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ls, d, kv = _lengths(c), c["d"], c["kv"]
    s = {"case": c, "lengths": ls}
    if c["kind"] == "prefill":
        heads, cu = kv * c["group"], _cumulated(ls)
        # q, k and v as a fused projection leaves them: column blocks of one matrix.
        u = _normal(gen, cu[-1], heads + 2 * kv, d)
        s.update(q=u[:, :heads], k=u[:, heads : heads + kv], v=u[:, heads + kv :], cu=_ints(cu))
    elif c["kind"] == "decode":
        first = [max(0, n - c["window"]) for n in ls]
        s["table"], pages = _table(c, gen, first, ls)
        s.update(cache=_filled_cache(c, gen, pages), lens=_ints(ls), q=_normal(gen, c["n"], kv * c["group"], d))
    else:
        cu, past = _cumulated(ls), [c["past"]] * c["n"]
        s["table"], pages = _table(c, gen, past, [a + n for a, n in zip(past, ls)])
        u = _normal(gen, cu[-1], c["heads"] + 2 * kv, d)
        s.update(q=u[:, : c["heads"]], k=u[:, c["heads"] : c["heads"] + kv], v=u[:, c["heads"] + kv :],
                 cu=_ints(cu), past=_ints(past), cache=_filled_cache(c, gen, pages))
        if c["rot"]:
            angle = torch.arange(c["past"] + max(ls), device="cuda", dtype=torch.float64)[:, None] * torch.pow(
                10000.0, -torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
            s.update(cos=angle.cos().float(), sin=angle.sin().float())
    return s


# ------------------------------------------------------------------------------- the plain forms --

def _softmax_over(scores, keep):
    """exp(scores - max) over the kept keys and its sums, in place; rows that keep nothing give zeros."""
    scores.masked_fill_(~keep, -math.inf)
    m = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(m.isfinite(), m, torch.zeros_like(m))).exp_()
    return scores, scores.sum(-1, keepdim=True)


def _prefill_plain(s):
    c = s["case"]
    n, L, kv, G, d = c["n"], max(s["lengths"]), c["kv"], c["group"], c["d"]
    start, lens = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    at = torch.arange(L, device="cuda")
    rows = (start[:, None] + at).clamp_(max=s["q"].shape[0] - 1)  # [n, L], padded
    q = s["q"][rows].float().view(n, L, kv, G, d).permute(0, 2, 3, 1, 4).reshape(n, kv, G * L, d)
    k, v = (s[x][rows].float().transpose(1, 2) for x in ("k", "v"))
    scores = torch.matmul(q.mul_(d ** -0.5), k.transpose(-1, -2)).view(n, kv, G, L, L)
    keep = (at <= at[:, None]) & (at > at[:, None] - c["window"]) & (at < lens[:, None])[:, None, :]
    p, total = _softmax_over(scores, keep[:, None, None])
    o = torch.matmul(p.view(n, kv, G * L, L), v).view(n, kv, G, L, d).div_(total)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, L, kv * G, d)
    return o[(at < lens[:, None])].to(torch.bfloat16)


def _rows_of(c, cache, table, positions, i):
    """Keys (i = 0) or values (i = 1) at positions [n, m] of every sequence: fp32 [n, m, kv, d]."""
    rows, pairs = _blocks(c, cache)
    page = table.gather(1, (positions // c["page"]).long()).long()
    off = (positions % c["page"]).long()
    if pairs is None:
        return rows[:, i][page, :, off].float()
    u = _unpack(rows[:, i][page, :, off], i == 0)
    pair = pairs[:, i][page, :, off].view(torch.bfloat16).unflatten(-1, (-1, 2)).float()
    return (u.float().sub_(8).mul_(pair[..., :1]).add_(pair[..., 1:])).flatten(-2)


def _decode_plain(s):
    c = s["case"]
    n, kv, G, d = c["n"], c["kv"], c["group"], c["d"]
    span = min(max(s["lengths"]), c["window"])
    first = (s["lens"] - c["window"]).clamp_(min=0)
    at = first[:, None] + torch.arange(span, device="cuda")
    keep = at < s["lens"][:, None]
    at = torch.minimum(at, (s["lens"][:, None] - 1).clamp_(min=0))
    q = s["q"].float().view(n, kv, G, d) * d ** -0.5
    k = _rows_of(c, s["cache"], s["table"], at, 0).transpose(1, 2)
    p, total = _softmax_over(torch.matmul(q, k.transpose(-1, -2)), keep[:, None, None])
    del k
    v = _rows_of(c, s["cache"], s["table"], at, 1).transpose(1, 2)
    return (torch.matmul(p, v) / total).view(n, kv * G, d).to(torch.bfloat16)


def _rotated(c, x, cos, sin):
    """The position rotation of the first `rot` channels: halves against each other, or neighbours."""
    r = c["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["pairs"] else (x[..., : r // 2], x[..., r // 2 : r])
    a, b = a.float(), b.float()
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if c["pairs"] else torch.cat([y, z], -1)
    return torch.cat([turned.to(torch.bfloat16), x[..., r:]], -1)


def _append_plain(s):
    c = s["case"]
    t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    position = s["past"][seq] + t - s["cu"][seq]
    q, k, v = s["q"], s["k"], s["v"]
    if c["rot"]:
        cos, sin = s["cos"][position][:, None], s["sin"][position][:, None]
        q, k = _rotated(c, q, cos, sin), _rotated(c, k, cos, sin)
    else:
        q, k = q.clone(), k.clone()
    page, off = s["table"][seq, position // c["page"]].long(), (position % c["page"]).long()
    rows, pairs = _blocks(c, s["cache"])
    out = {"q": q}
    if c["keys"]:
        out["k"] = k
    if pairs is None:
        rows[:, 0][page, :, off] = k
        rows[:, 1][page, :, off] = v
        out["cache"] = rows
        return out
    for i, x, name in ((0, k, "k_read"), (1, v, "v_read")):
        u, scale, centre = _to_codes(x)
        rows[:, i][page, :, off] = _pack(u, i == 0)
        pairs[:, i][page, :, off] = _pair_bytes(scale, centre)
        out[name] = ((u.float() - 8) * scale.float().unsqueeze(-1) + centre.float().unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
    return out


# -------------------------------------------------------------------------- the framework's calls --

def _own(s):
    import block_sliding_window_gb300 as bsw

    c = s["case"]
    if c["kind"] == "prefill":
        return bsw.swa_attention_packed(s["q"], s["k"], s["v"], s["cu"], c["window"])
    if c["kind"] == "decode":
        return bsw.swa_attention_paged(s["q"], s["cache"], s["table"], s["lens"], c["kv"], c["page"], c["bits"], c["window"])
    q, k = bsw.kv_append(s["q"], s["k"], s["v"], s["cache"], s["table"], s["cu"], s["past"], c["page"], c["bits"],
                         cos=s.get("cos"), sin=s.get("sin"), interleaved=c["pairs"], keep_keys=c["keys"])
    out = {"q": q}
    if c["keys"]:
        out["k"] = k
    if c["bits"] == 16:
        out["cache"] = _blocks(c, s["cache"])[0]
    else:
        out["k_read"], out["v_read"] = bsw.kv_gather(s["cache"], s["table"], s["cu"], s["past"], q.shape[0], c["kv"], c["d"], c["page"], c["bits"])
    return out


def run(s):
    if own:
        return _own(s)
    return {"prefill": _prefill_plain, "decode": _decode_plain, "append": _append_plain}[s["case"]["kind"]](s)


# -------------------------------------------------------------------- the definitions in 64 bits --

def _attend64(q, k, v, first_query, window):
    """q [m, h, d] at positions first_query.. against all keys k, v [n, d]: float64 [m, h, d]."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    step = max(1, int(2e8) // max(1, k.shape[0] * q.shape[1]))
    for i in range(0, q.shape[0], step):
        x = q[i : i + step].double()
        where = first_query + i + torch.arange(x.shape[0], device="cuda")
        lo = max(0, int(where[0]) - window + 1)
        hi = int(where[-1]) + 1
        j = torch.arange(lo, hi, device="cuda")
        z = torch.einsum("mhd,nd->mhn", x, k[lo:hi].double()) / math.sqrt(q.shape[-1])
        seen = (j[None] <= where[:, None]) & (where[:, None] - j[None] < window)
        z = torch.softmax(z.masked_fill(~seen[:, None], float("-inf")), -1)
        out[i : i + step] = torch.einsum("mhn,nd->mhd", z, v[lo:hi].double())
    return out


def _nibble_places(d, keys):
    """Which nibble of a row holds each channel."""
    c = [0] * d
    for w in range(d // 32):
        for x in range(32):
            c[32 * w + x] = 8 * (x // 8 * (d // 32) + w) + x % 8 if keys else (d // 8) * (x // 4) + 4 * w + x % 4
    return torch.tensor(c, device="cuda")


def _held64(c, cache, table_row, lo, hi, head):
    """Keys and values of one head at positions lo..hi-1 of one sequence, in float64."""
    p, d, row = c["page"], c["d"], _row_bytes(c)
    at = torch.arange(lo, hi, device="cuda")
    pages = cache.view(cache.shape[0], 2, c["kv"], p * row)[:, :, head][table_row[at // p].long()]  # [m, 2, p * row]
    got = []
    for i in (0, 1):
        flat, off = pages[:, i], at % p
        if c["bits"] == 16:
            got.append(flat.gather(1, off[:, None] * row + torch.arange(row, device="cuda")).contiguous().view(torch.bfloat16).double())
            continue
        place = _nibble_places(d, i == 0)
        byte = flat.gather(1, off[:, None] * (d // 2) + place // 2)
        u = torch.where(place % 2 == 1, byte // 16, byte % 16).double()
        pair = flat.gather(1, p * (d // 2) + off[:, None] * (d // 8) + torch.arange(d // 8, device="cuda")).contiguous().view(torch.bfloat16).double()
        got.append((u - 8) * pair[:, 0::2].repeat_interleave(32, 1) + pair[:, 1::2].repeat_interleave(32, 1))
    return got


def _turned64(c, x, position):
    r, x = c["rot"], x.double()
    if not r:
        return x
    freq = torch.tensor([10000.0 ** (-2 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    angle = position.double()[:, None, None] * freq
    co, si = angle.cos().float().double(), angle.sin().float().double()  # the tables are fp32 inputs
    first = [2 * i for i in range(r // 2)] if c["pairs"] else list(range(r // 2))
    second = [2 * i + 1 for i in range(r // 2)] if c["pairs"] else list(range(r // 2, r))
    y = x.clone()
    y[..., first] = x[..., first] * co - x[..., second] * si
    y[..., second] = x[..., second] * co + x[..., first] * si
    return y


def _quantized64(x):
    """What a 4-bit row stands for, from bf16 values held in float64."""
    out = torch.empty_like(x)
    for w in range(0, x.shape[-1], 32):
        g = x[..., w : w + 32]
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        s = ((hi - lo) / 15).to(torch.bfloat16).double()
        z = (lo + 8 * s).to(torch.bfloat16).double()
        u = torch.round((g - z) / s.masked_fill(s == 0, 1.0)).clamp(-8, 7)
        out[..., w : w + 32] = z + s * u
    return out


def exact(c, seed):
    s = prepare(c, seed)
    ls, kv, d = s["lengths"], c["kv"], c["d"]
    if c["kind"] == "prefill":
        G, cu, out = c["group"], _cumulated(ls), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for a, b in zip(cu, cu[1:]):
            for h in range(kv):
                out[a:b, h * G : (h + 1) * G] = _attend64(s["q"][a:b, h * G : (h + 1) * G], s["k"][a:b, h], s["v"][a:b, h], 0, c["window"])
        return out
    if c["kind"] == "decode":
        G, out = c["group"], torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(ls):
            lo = max(0, n - c["window"])
            for h in range(kv):
                k, v = _held64(c, s["cache"], s["table"][b], lo, n, h)
                z = torch.softmax(s["q"][b, h * G : (h + 1) * G].double() @ k.T / math.sqrt(d), -1)
                out[b, h * G : (h + 1) * G] = z @ v
        return out
    position = torch.cat([torch.arange(c["past"], c["past"] + n, device="cuda") for n in ls])
    q, k, v = _turned64(c, s["q"], position), _turned64(c, s["k"], position), s["v"].double()
    out = {"q": q}
    if c["keys"]:
        out["k"] = k
    if c["bits"] == 4:
        out["k_read"], out["v_read"] = _quantized64(k.to(torch.bfloat16).double()), _quantized64(v)
        return out
    held = s["cache"].view(torch.bfloat16).view(-1, 2, kv, c["page"], d).double()
    row = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(ls)])
    page, off = s["table"][row, position // c["page"]].long(), position % c["page"]
    held[page, 0, :, off] = k
    held[page, 1, :, off] = v
    out["cache"] = held
    return out
