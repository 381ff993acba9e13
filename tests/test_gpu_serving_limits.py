"""The serving operators on the GPU at the limits of what they document: refusals through the
binding, partly filled tiles, values of extreme size, calls of many items and long shares."""
import numpy as np
import pytest
import torch

from block_sliding_window_gb300 import workloads
from tests import serving_model as M

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(ptb_lib):
    ptb_lib.last_device_error()
    yield
    assert ptb_lib.last_device_error() == 0, "a kernel recorded a device-side error"


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def normal(shape, seed, std=1.0):
    return workloads.normal_bf16(shape, seed=seed, std=std).cuda()


# ------------------------------------------------------------------------------- refusals --

@pytest.mark.parametrize("heads", [129, 256])
def test_packed_refuses_groups_beyond_a_tile(ptb_lib, heads):
    q, k, v = normal((10, heads, 16), 1), normal((10, 1, 16), 2), normal((10, 1, 16), 3)
    with pytest.raises(ptb_lib.PTBError, match="SHAPE"):
        ptb_lib.swa_attention_packed(q, k, v, ints([0, 10]), 4)


@pytest.mark.parametrize("window", [0, -1, -(1 << 31) - 5, -(1 << 32) + 5, -(1 << 40) + 1])
def test_attention_refuses_windows_below_one(ptb_lib, window):
    """Also those whose low 32 bits are a positive number."""
    q, kv, page = normal((10, 2, 16), 1), normal((10, 1, 16), 2), 16
    cache = torch.zeros(1, ptb_lib.kv_page_size(1, page, 16, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(ptb_lib.PTBError, match="ARG"):
        ptb_lib.swa_attention_packed(q, kv, kv.clone(), ints([0, 10]), window)
    with pytest.raises(ptb_lib.PTBError, match="ARG"):
        ptb_lib.swa_attention_paged(q[:1], cache, ints([0])[None], ints([5]), 1, page, 16, window)


# ----------------------------------------------------------------------- partly filled tiles --

def cumulated(ls):
    out = [0]
    for n in ls:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("heads,kv,d", [(5, 1, 128), (6, 2, 96), (71, 1, 64), (2, 2, 128)])
def test_packed_partly_filled_tiles_with_infinite_values(ptb_lib, heads, kv, d):
    """Tiles whose lanes part ways in every block of 32 columns: rows that belong to no token, and
    rows that look through different numbers of keys for an infinite value of theirs."""
    lens, window = [3, 30, 70, 1, 131], 20
    cu = cumulated(lens)
    t = cu[-1] + 2
    q, k, v = normal((t, heads, d), 11), normal((t, kv, d), 12), normal((t, kv, d), 13)
    inf_at = [cu[0] + 1, cu[1] + 7, cu[2] + 40, cu[4] + 64, cu[4] + 120]
    special = list(range(3, d, 16))
    for at in inf_at:
        v[at, :, special] = float("inf")
    o = torch.full_like(q, 77.0)
    ptb_lib.swa_attention_packed(q, k, v, ints(cu), window, o=o)
    v64 = M.to64(v)
    v64[~np.isfinite(v64)] = 0
    want, bound, written = M.packed(M.to64(q), M.to64(k), v64, cu, cu, window, d ** -0.5)
    got = M.to64(o)
    assert (got[~written] == 77).all()
    sees = np.zeros(t, dtype=bool)
    for at in inf_at:
        end = next(b for b in cu if b > at)
        sees[at:min(at + window, end)] = True
    plain = [c for c in range(d) if c not in special]
    assert (got[sees][..., special] == np.inf).all()
    for rows, columns in ((written & ~sees, list(range(d))), (sees, plain)):
        over = np.abs(got - want)[rows][..., columns] - bound[rows][..., columns]
        assert (over <= 0).all(), over.max()


@pytest.mark.parametrize("heads", [3, 11])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_paged_4bit_rows_that_hold_nan_in_one_group(ptb_lib, heads, d):
    """Every number of groups a row: NaN in one group of keys or values that the window has left
    reaches nothing, and in a key inside the window it reaches its sequence alone."""
    lens, window, page = [75, 64, 33], 30, 16
    pages = sum(-(-n // page) for n in lens)
    table = np.full((3, 5), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = range(at, at + need)
        at += need
    cache = torch.full((pages, ptb_lib.kv_page_size(1, page, d, 4)), 0xFF, dtype=torch.uint8, device="cuda")
    cu = cumulated(lens)
    k, v, q = normal((cu[-1], 1, d), 21), normal((cu[-1], 1, d), 22), normal((3, heads, d), 23)
    first, last = 0, d // 32 - 1
    for b, n in enumerate(lens):
        for p in range(n - window):
            k[cu[b] + p, 0, 32 * (first if p % 2 else last)] = float("nan")
            v[cu[b] + p, 0, 32 * (last if p % 2 else first)] = float("nan")
    dev = torch.from_numpy(table).cuda()
    ptb_lib.kv_append(None, k, v, cache, dev, ints(cu), ints([0] * 3), page, 4, keep_keys=False)
    host = M.Cache(cache.cpu().numpy(), 1, page, d, 4)
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, dev, ints(lens), 1, page, 4, window))
    want, bound = M.paged(M.to64(q), host, table, lens, window, d ** -0.5)
    assert (np.abs(o - want) <= bound).all()
    k[cu[1] + 50, 0, 32 * last] = float("nan")
    ptb_lib.kv_append(None, k, v, cache, dev, ints(cu), ints([0] * 3), page, 4, keep_keys=False)
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, dev, ints(lens), 1, page, 4, window))
    assert np.isnan(o[1]).all() and (np.abs(o - want)[[0, 2]] <= bound[[0, 2]]).all()


# ------------------------------------------------------------------------- scores of any size --
#
# One channel of q and k is not zero, so a score is one product of two bf16 values, exact in fp32,
# and the scores of two keys are equal or differ by 2^-8 of their size: 2^10 and more here.  The
# weights are then 0 or equal, whatever the last bits of a score.
#
# From 2^29 in the log2 domain on (power 15: at least 2^30 * 0.7 * 1.44) the largest score's weight
# is exactly 1.  At powers 10 and 13 scores are at most 2^26 * 1.5 * 2 * 0.7 * 1.45 < 2^29: the exact
# product and the maximum, rounded to fp32, differ by r, |r| <= 2^4, and the weight is 2^r.  It
# cancels against the sum of weights, but is rounded to bf16 before the weighted sum (H of it),
# which the sum is not: H times the sum of the weighted magnitudes is added there.

def weight_error(power):
    return M.H if power < 15 else 0.0


def one_channel(t, heads, kv, d, power, seed, rising=False):
    rng = np.random.RandomState(seed)
    q, k = torch.zeros(t, heads, d), torch.zeros(t, kv, d)
    q[:, :, 0] = torch.from_numpy(rng.choice([-1.5, -1.0, 1.0, 1.25], (t, heads))) * 2.0 ** power
    m = 1 + (np.arange(t) % 128) / 128 if rising else 1 + rng.permutation(128 * (1 + t // 128))[:t] % 128 / 128
    k[:, :, 0] = torch.from_numpy(m)[:, None] * 2.0 ** power
    return q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), normal((t, kv, d), seed)


def weights64(q, k, first, window, scale):
    """[m, h, n] softmax weights of rows at positions first.., float64."""
    g = q.shape[1] // k.shape[1]
    s = np.einsum("mhd,nhd->mhn", q, np.repeat(k, g, 1)) * scale
    p, j = first + np.arange(q.shape[0])[:, None], np.arange(k.shape[0])[None]
    s = np.where(((j <= p) & (p - j < window))[:, None], s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    return w / w.sum(-1, keepdims=True)


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("power", [10, 13, 15, 16, 17, 20, 33, 60])
def test_packed_scores_of_any_size(ptb_lib, power, rising):
    t, heads, kv, d, window = 300, 4, 2, 64, 100
    q, k, v = one_channel(t, heads, kv, d, power, 31, rising)
    q[150:] = 0  # rows whose scores are all equal, in tiles of the others
    cu = [0, 200, t]
    o = M.to64(ptb_lib.swa_attention_packed(q, k, v, ints(cu), window, scale=0.7))
    for a, b in zip(cu, cu[1:]):
        w = weights64(M.to64(q)[a:b], M.to64(k)[a:b], 0, window, 0.7)
        v64 = np.repeat(M.to64(v)[a:b], heads // kv, 1)
        want, mag = np.einsum("mhn,nhd->mhd", w, v64), np.einsum("mhn,nhd->mhd", w, np.abs(v64))
        # fp32 sums of at most 100 values
        assert (np.abs(o[a:b] - want) <= M.H * np.abs(want) + 1.01 * (2.0 ** -16 + weight_error(power)) * mag).all()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("heads,rising", [(2, False), (2, True), (24, False)])
@pytest.mark.parametrize("power", [10, 15, 16, 17, 20, 33, 58])
def test_paged_scores_of_any_size(ptb_lib, bits, power, heads, rising):
    n, kv, d, page, window = 300, 2, 64, 16, 250
    q, k, v = one_channel(n, heads, kv, d, power, 41, rising)
    q = torch.cat([q[:2], torch.zeros_like(q[:1])])
    pages = -(-n // page)
    table = ints(range(pages))[None].repeat(3, 1)
    cache = torch.zeros(pages, ptb_lib.kv_page_size(kv, page, d, bits), dtype=torch.uint8, device="cuda")
    ptb_lib.kv_append(None, k, v, cache, table[:1], ints([0, n]), ints([0]), page, bits, keep_keys=False)
    lens = [n, 130, n]
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, table, ints(lens), kv, page, bits, window, scale=0.7))
    host = M.Cache(cache.cpu().numpy(), kv, page, d, bits)
    k64, v64, mag = np.zeros((n, kv, d)), np.zeros((n, kv, d)), np.zeros((n, kv, d))
    for p in range(n):
        for h in range(kv):
            k64[p, h] = host.get(p // page, p % page, h, 0)[0]
            v64[p, h], u, s, z = host.get(p // page, p % page, h, 1)
            # 4 bits: p * scale is rounded before the sum whatever p is, p for the centres as above
            mag[p, h] = (weight_error(power) * np.abs(v64[p, h]) if u is None else
                         M.H * s * np.abs(u - 8) + weight_error(power) * np.abs(z))
    g = heads // kv
    for b, m in enumerate(lens):
        w = weights64(M.to64(q[b:b + 1]), k64[:m], m - 1, window, 0.7)[0]
        want = np.einsum("hn,nhd->hd", w, np.repeat(v64[:m], g, 1))
        err = np.einsum("hn,nhd->hd", w, np.repeat(mag[:m] + 2.0 ** -16 * np.abs(v64[:m]), g, 1))
        assert (np.abs(o[b] - want) <= M.H * np.abs(want) + 1.01 * err).all(), (b, np.abs(o[b] - want).max())


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("heads", [2, 12])
def test_paged_4bit_queries_that_the_scale_takes_out_of_range(ptb_lib, heads, sign):
    """Scale times a query of 2^118 and more: NaN in its row, for scores of either sign (and not the
    zeros of a row without keys); up to 2^116 the row that its neighbours get."""
    n, d, page = 70, 64, 16
    pages = -(-n // page)
    k, v = normal((n, 1, d), 51).abs() + 0.5, normal((n, 1, d), 52)
    table = ints(range(pages))[None].repeat(2, 1)
    cache = torch.zeros(pages, ptb_lib.kv_page_size(1, page, d, 4), dtype=torch.uint8, device="cuda")
    ptb_lib.kv_append(None, k, v, cache, table[:1], ints([0, n]), ints([0]), page, 4, keep_keys=False)
    host = M.Cache(cache.cpu().numpy(), 1, page, d, 4)
    for power, scale in ((118, 1.0), (100, 2.0 ** 18), (0, 2.0 ** 118), (117, 4.0)):
        q = torch.zeros(2, heads, d, dtype=torch.bfloat16, device="cuda")
        q[:, :, 3] = 2.0 ** (power - 130)  # the other heads: scores of 2^-12 and less
        q[0, 1, 3] = sign * 2.0 ** power
        o = M.to64(ptb_lib.swa_attention_paged(q, cache, table, ints([n, n]), 1, page, 4, 1000, scale=scale))
        assert np.isnan(o[0, 1]).all(), (power, scale)
        q[0, 1, 3] = sign * 2.0 ** (power - 130)
        want, bound = M.paged(M.to64(q), host, table.cpu().numpy(), [n, n], 1000, scale)
        o[0, 1] = want[0, 1]
        assert (np.abs(o - want) <= bound).all()
    # scores of 2^115 and more: all the weight on the largest
    q[:, :, 3] = sign * 2.0 ** 115
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, table, ints([n, n]), 1, page, 4, 1000, scale=1.0))
    key = np.array([host.get(p // page, p % page, 0, 0)[0][3] for p in range(n)]) * sign
    w = (key == key.max()) / (key == key.max()).sum()
    got = [host.get(p // page, p % page, 0, 1) for p in range(n)]
    want = w @ np.stack([x[0] for x in got])
    err = w @ np.stack([M.H * x[2] * np.abs(x[1] - 8) + 2.0 ** -16 * np.abs(x[0]) for x in got])
    assert (np.abs(o - want) <= M.H * np.abs(want) + 1.01 * err).all()


# ------------------------------------------------------------------- graphs and other streams --

@pytest.mark.parametrize("bits,inter", [(16, False), (4, True)])
def test_decode_steps_captured_once(ptb_lib, bits, inter):
    """Append, read back and attend in one graph whose lengths move on the device: each replay is the
    next step, bit for bit what the eager calls give; a second graph runs on another stream."""
    prompts, steps, heads, kv, d, page, window = [5, 31, 16, 1], 20, 6, 2, 64, 16, 24
    batch = len(prompts)
    need = [-(-(n + steps) // page) for n in prompts]
    cos = torch.cos(torch.arange(64.0)[:, None] * torch.arange(1, d // 2 + 1) / 50).cuda()
    sin = torch.sin(torch.arange(64.0)[:, None] * torch.arange(1, d // 2 + 1) / 50).cuda()
    cu, one = cumulated(prompts), ints(range(batch + 1))
    q0, k0, v0 = (normal((cu[-1], n, d), 60 + i) for i, n in enumerate((heads, kv, kv)))
    new = [[normal((batch, n, d), 70 + 3 * s + i) for i, n in enumerate((heads, kv, kv))] for s in range(steps)]

    def start():
        order = np.random.RandomState(3).permutation(sum(need))
        table = np.full((batch, max(need)), -1, dtype=np.int32)
        for b, n in enumerate(need):
            table[b, :n], order = order[:n], order[n:]
        cache = torch.full((sum(need), ptb_lib.kv_page_size(kv, page, d, bits)), 0xFF, dtype=torch.uint8, device="cuda")
        s = dict(cache=cache, table=torch.from_numpy(table).cuda(), past=ints([0] * batch), lens=ints(prompts))
        ptb_lib.kv_append(q0, k0, v0, cache, s["table"], ints(cu), s["past"], page, bits, cos=cos, sin=sin, interleaved=inter)
        s["past"].copy_(ints(prompts))
        s["in"] = [t.clone() for t in new[0]]
        return s

    def step(s, stream=None):
        q, k, v = s["in"]
        s["q"], s["k"] = ptb_lib.kv_append(q, k, v, s["cache"], s["table"], one, s["past"], page, bits, cos=cos, sin=sin,
                                           interleaved=inter, stream=stream)
        s["kr"], s["vr"] = ptb_lib.kv_gather(s["cache"], s["table"], one, s["past"], batch, kv, d, page, bits, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            s["lens"].copy_(s["past"] + 1)
        s["o"] = ptb_lib.swa_attention_paged(s["q"], s["cache"], s["table"], s["lens"], kv, page, bits, window, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            s["past"].add_(1)

    want = []
    s = start()
    for x in new:
        for a, b in zip(s["in"], x):
            a.copy_(b)
        step(s)
        want.append([s[n].clone() for n in ("q", "k", "kr", "vr", "o")])
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        s, stream = start(), torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(s)
        runs.append((s, stream, g))
    for x, w in zip(new, want):
        for s, stream, g in runs:
            with torch.cuda.stream(stream):
                for a, b in zip(s["in"], x):
                    a.copy_(b)
                g.replay()
        torch.cuda.synchronize()
        for s, _, _ in runs:
            for n, t in zip(("q", "k", "kr", "vr", "o"), w):
                assert torch.equal(s[n], t), n
    s, stream = start(), torch.cuda.Stream()  # eager, the stream given to each call
    torch.cuda.synchronize()
    for x, w in zip(new, want):
        with torch.cuda.stream(stream):
            for a, b in zip(s["in"], x):
                a.copy_(b)
        step(s, stream)
        stream.synchronize()
        for n, t in zip(("q", "k", "kr", "vr", "o"), w):
            assert torch.equal(s[n], t), n


# A row whose scores are large in one part and ordinary in another: the ordinary part's weights go by
# the ordinary factor, whichever part comes first.

def two_sizes(t, heads, kv, d, order, seed):
    """Scores of -2^30 and less (times 0.7) for some keys and of -3 to 3 for the others, in runs of
    keys as `order` says (0: ordinary), of 2^30 and more for those of order 2; one channel each, in
    groups of their own, so that no score of a kind holds a rounding of the other's size."""
    rng = np.random.RandomState(seed)
    q, k = torch.zeros(t, heads, d), torch.zeros(t, kv, d)
    q[:, :, 0], q[:, :, 32] = 2.0 ** 15, 1.0
    for at, n, kind in order:
        if kind:
            k[at:at + n, :, 0] = torch.from_numpy(rng.randint(128, 256, n) / 128.0)[:, None] * (2.0 ** 15 * (1 if kind == 2 else -1))
        else:
            k[at:at + n, :, 32] = torch.from_numpy(rng.randint(-24, 25, n) / 8.0)[:, None]
    return q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), normal((t, kv, d), seed)


ORDERS = [
    [(0, 150, 1), (150, 150, 0)], [(0, 150, 0), (150, 150, 1)], [(0, 300, 1)], [(0, 40, 1), (40, 3, 0), (43, 257, 1)],
    [(0, 200, 1), (200, 60, 0), (260, 1, 2), (261, 39, 0)], [(0, 64, 0), (64, 64, 1), (128, 64, 0), (192, 108, 1)],
]


@pytest.mark.parametrize("order", range(len(ORDERS)))
@pytest.mark.parametrize("scale", [0.7, 1.2])
def test_packed_scores_large_in_one_part_of_a_row(ptb_lib, order, scale):
    t, heads, kv, d = 300, 2, 1, 64
    q, k, v = two_sizes(t, heads, kv, d, ORDERS[order], 81)
    for window in (1 << 20, 180):
        o = M.to64(ptb_lib.swa_attention_packed(q, k, v, ints([0, t]), window, scale=scale))
        w = weights64(M.to64(q), M.to64(k), 0, window, scale)
        v64 = np.repeat(M.to64(v), heads // kv, 1)
        want, mag = np.einsum("mhn,nhd->mhd", w, v64), np.einsum("mhn,nhd->mhd", w, np.abs(v64))
        # ordinary scores are exact; weights rounded to bf16 once, sums of at most 300 in fp32
        assert (np.abs(o - want) <= M.H * np.abs(want) + 1.01 * (M.H + 2.0 ** -14) * mag).all(), window


@pytest.mark.parametrize("order", range(len(ORDERS)))
@pytest.mark.parametrize("bits,heads", [(16, 2), (4, 2), (16, 12), (4, 12)])
def test_paged_scores_large_in_one_part_of_a_row(ptb_lib, order, bits, heads):
    """Many copies of the sequence, so that a warp takes its parts one after the other."""
    n, kv, d, page, scale = 300, 1, 64, 64, 0.7
    q, k, v = two_sizes(n, heads, kv, d, ORDERS[order], 91)
    batch = 12 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = -(-n // page)
    cache = torch.zeros(pages, ptb_lib.kv_page_size(kv, page, d, bits), dtype=torch.uint8, device="cuda")
    table = ints(range(pages))[None]
    ptb_lib.kv_append(None, k, v, cache, table, ints([0, n]), ints([0]), page, bits, keep_keys=False)
    host = M.Cache(cache.cpu().numpy(), kv, page, d, bits)
    rows = [[host.get(p // page, p % page, 0, i) for p in range(n)] for i in (0, 1)]
    k64, v64 = (np.stack([x[0] for x in r]) for r in rows)
    mag = np.abs(v64) if bits == 16 else np.stack([s * np.abs(u - 8) + np.abs(z) for _, u, s, z in rows[1]])
    for window in (1 << 20, 180):
        o = ptb_lib.swa_attention_paged(q[:1].repeat(batch, 1, 1), cache, table.repeat(batch, 1), ints([n] * batch), kv, page,
                                        bits, window, scale=scale)
        w = weights64(M.to64(q[:1]), k64[:, None], n - 1, window, scale)[0]
        want, a = w @ v64, w @ mag
        # ordinary scores are off by a few units of 2^-22, sums of at most 300 weights in fp32
        assert (np.abs(M.to64(o) - want) <= M.H * np.abs(want) + 1.01 * (M.H + 2.0 ** -14) * a).all(), window
