"""The serving operators on the GPU against the 64-bit model of tests/serving_model.py, element by
element within the bounds derived there."""
import numpy as np
import pytest
import torch

import oracle
from block_sliding_window_gb300 import workloads
from tests import serving_model as M
from tests.parity import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(ptb_lib):
    ptb_lib.last_device_error()
    yield
    assert ptb_lib.last_device_error() == 0, "a kernel recorded a device-side error"


def cumulated(ls):
    return [0] + list(np.cumsum(ls))


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def normal(shape, seed, std=1.0):
    return workloads.normal_bf16(shape, seed=seed, std=std).cuda()


def held_to(got, want, bound):
    got = M.to64(got)
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} values beyond the bound, by up to {over.max():.3e}"


# ------------------------------------------------------------------ packed attention --

PACKED = [
    # lengths of queries, of keys (None: the same), heads, kv heads, d, window
    ([1], None, 1, 1, 128, 1),
    ([1, 2, 3], None, 2, 2, 64, 2),
    ([64, 65, 63], None, 4, 4, 128, 1000),
    ([127, 128, 129, 1], None, 2, 1, 128, 50),
    ([255, 256, 257], None, 2, 2, 32, 64),
    ([300, 5, 0, 77], None, 4, 2, 96, 33),
    ([0, 0, 40, 0], None, 3, 1, 64, 7),
    ([200, 17], None, 8, 1, 128, 96),
    ([100, 31, 64], None, 10, 2, 16, 40),
    ([90, 33], None, 6, 2, 64, 1 << 30),
    ([70, 50], None, 7, 1, 96, 128),
    ([40, 21], None, 16, 1, 128, 30),
    ([33, 5], None, 32, 1, 64, 12),
    ([9, 20], None, 71, 1, 64, 16),
    ([6, 3], None, 128, 1, 32, 4),
    ([700], None, 2, 1, 128, 600),
    ([5, 64, 1, 130], [300, 64, 129, 200], 4, 2, 128, 77),
    ([1, 1, 1], [1, 64, 500], 8, 2, 64, 1 << 20),
    ([10, 4, 3], [6, 0, 3], 4, 4, 128, 9),       # the first queries have no keys; one sequence none
    ([64, 128], [10, 100], 2, 1, 32, 300),
    (list(range(1, 45)), None, 2, 1, 64, 20),    # more sequences than a warp has lanes
    # more items than SMs: the sorted list
    ([100, 1, 0, 257, 64, 300], None, 40, 40, 32, 60),
    ([3] * 70 + [129, 31], None, 24, 12, 64, 1000),
    ([2, 60, 1], [2, 20, 90], 96, 48, 16, 11),
]


def packed_inputs(lq, lk, heads, kv, d, seed, tail=3):
    lk = lq if lk is None else lk
    tq, tk = sum(lq) + tail, sum(lk) + tail
    return (normal((tq, heads, d), seed), normal((tk, kv, d), seed + 1), normal((tk, kv, d), seed + 2),
            cumulated(lq), cumulated(lk))


@pytest.mark.parametrize("lq,lk,heads,kv,d,window", PACKED)
def test_packed(ptb_lib, lq, lk, heads, kv, d, window):
    q, k, v, cu_q, cu_k = packed_inputs(lq, lk, heads, kv, d, 10)
    o = torch.full_like(q, 77.0)
    ptb_lib.swa_attention_packed(q, k, v, ints(cu_q), window, o=o,
                                 cu_seqlens_k=None if lk is None else ints(cu_k))
    want, bound, written = M.packed(M.to64(q), M.to64(k), M.to64(v), cu_q, cu_k, window, d ** -0.5)
    held_to(o[torch.from_numpy(written)], want[written], bound[written])
    assert (o[torch.from_numpy(~written)] == 77).all()  # rows behind the last sequence


@pytest.mark.parametrize("scale,std", [(0.5, 1.0), (0.01, 8.0), (1.0, 3.0)])
def test_packed_scale_and_peaked_weights(ptb_lib, scale, std):
    q, k, v, cu, _ = packed_inputs([150, 90], None, 4, 2, 64, 20)
    q = (q * std).to(torch.bfloat16)
    o = ptb_lib.swa_attention_packed(q, k, v, ints(cu), 80, scale=scale)
    want, bound, written = M.packed(M.to64(q), M.to64(k), M.to64(v), cu, cu, 80, scale)
    held_to(o[torch.from_numpy(written)], want[written], bound[written])


def views(kind, t, heads, kv, d, seed):
    """q, k, v of one shape in several memory orders."""
    if kind == "fused":  # column blocks of a projection's output
        u = normal((t, (heads + 2 * kv) * d + 24), seed)
        cut = lambda a, n: u[:, a * d:(a + n) * d].unflatten(1, (n, d))  # noqa: E731
        return cut(0, heads), cut(heads, kv), cut(heads + kv, kv)
    if kind == "heads_first":
        return tuple(normal((n, t, d), seed + i).transpose(0, 1) for i, n in enumerate((heads, kv, kv)))
    return tuple(normal((2 * t, n, d + 8), seed + i)[::2, :, :d] for i, n in enumerate((heads, kv, kv)))


@pytest.mark.parametrize("kind", ["fused", "heads_first", "gaps"])
def test_packed_strides(ptb_lib, kind):
    lens, heads, kv, d, w = [130, 40], 4, 2, 96, 70
    q, k, v = views(kind, 175, heads, kv, d, 30)
    o = views(kind, 175, heads, kv, d, 40)[0]
    before = o.clone()
    cu = cumulated(lens)
    ptb_lib.swa_attention_packed(q, k, v, ints(cu), w, o=o)
    want, bound, written = M.packed(M.to64(q), M.to64(k), M.to64(v), cu, cu, w, d ** -0.5)
    held_to(o[:170], want[:170], bound[:170])
    assert torch.equal(o[170:], before[170:])


def test_packed_in_place(ptb_lib):
    q, k, v, cu, _ = packed_inputs([300, 33], None, 8, 2, 64, 50)
    want = ptb_lib.swa_attention_packed(q, k, v, ints(cu), 90)
    tail = q[333:].clone()
    got = ptb_lib.swa_attention_packed(q, k, v, ints(cu), 90, o=q)
    assert got is q and torch.equal(got[:333], want[:333]) and torch.equal(q[333:], tail)


def test_packed_of_one_sequence_equals_swa_attention(ptb_lib):
    q, k, v = (normal((1, 4, 500, 128), 60 + i) for i in range(3))
    want = ptb_lib.swa_attention(q, k, v, 200)
    got = ptb_lib.swa_attention_packed(*(t[0].transpose(0, 1) for t in (q, k, v)), ints([0, 500]), 200)
    assert_close(got.transpose(0, 1)[None].float().cpu().numpy(), M.to64(want), "packed")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads,kv", [(2, 2), (8, 1)])
def test_packed_values_that_no_row_sees(ptb_lib, bad, heads, kv):
    """Non-finite keys and values of other sequences, of rows behind the last sequence, and of
    positions that the mask leaves out reach nothing; rows that see one are not finite."""
    lens, d, w = [70, 100, 30], 64, 40
    q, k, v, cu, _ = packed_inputs(lens, None, heads, kv, d, 70, tail=60)
    k[200:], v[200:], q[200:] = bad, bad, bad
    k[:70], v[:70] = bad, bad                # the whole first sequence
    k[70 + 50], v[70 + 50] = bad, bad        # one position of the second
    o = ptb_lib.swa_attention_packed(q, k, v, ints(cu), w)
    k64, v64 = M.to64(k), M.to64(v)
    k64[~np.isfinite(k64)] = 0
    v64[~np.isfinite(v64)] = 0
    want, bound, _ = M.packed(M.to64(q), k64, v64, cu, cu, w, d ** -0.5)
    sees = np.zeros(200, dtype=bool)
    sees[:70] = True
    sees[70 + 50:70 + 50 + w] = True
    held_to(o[:200][torch.from_numpy(~sees)], want[:200][~sees], bound[:200][~sees])
    assert not np.isfinite(M.to64(o[:200][torch.from_numpy(sees)])).any()


def test_packed_infinite_value_alone(ptb_lib):
    """An infinite value whose key is finite: rows that see it get that infinity, in its channel."""
    q, k, v, cu, _ = packed_inputs([150], None, 2, 1, 64, 80, tail=0)
    v[100, 0, 5] = float("-inf")
    o = M.to64(ptb_lib.swa_attention_packed(q, k, v, ints(cu), 30))
    assert (o[100:130, :, 5] == -np.inf).all()
    o[100:130, :, 5] = 0
    assert np.isfinite(o).all()


def test_scores_of_minus_infinity(ptb_lib):
    """A row whose scores are all minus infinity gets zeros, like one without keys; one other key
    takes all the weight."""
    n, heads, d, page = 70, 4, 64, 16
    q, k, v = normal((n, heads, d), 24), normal((n, heads, d), 25), normal((n, heads, d), 26)
    q[..., 0] = 1.0
    k[..., 0] = float("-inf")
    cu = ints([0, n])
    assert (ptb_lib.swa_attention_packed(q, k, v, cu, 40) == 0).all()
    table = ints(range(5))[None]
    cache = new_cache(ptb_lib, 5, heads, page, d, 16)
    ptb_lib.kv_append(None, k, v, cache, table, cu, ints([0]), page, 16)
    assert (ptb_lib.swa_attention_paged(q[n - 1:], cache, table, ints([n]), heads, page, 16, 40) == 0).all()
    k[50, :, 0] = 0.0
    ptb_lib.kv_append(None, k, v, cache, table, cu, ints([0]), page, 16)
    o = ptb_lib.swa_attention_packed(q, k, v, cu, 40)
    assert (o[:50] == 0).all() and torch.equal(o[50:], v[50:51].expand(n - 50, heads, d))
    o = ptb_lib.swa_attention_paged(q[n - 1:], cache, table, ints([n]), heads, page, 16, 40)
    assert torch.equal(o[0], v[50])


def test_packed_bad_offsets_are_recorded(ptb_lib):
    q, k, v, _, _ = packed_inputs([64, 64], None, 2, 2, 64, 90, tail=0)
    for cu in ([0, 64, 200], [0, 100, 64], [-5, 64, 128]):
        o = torch.full_like(q, 5.0)
        ptb_lib.swa_attention_packed(q, k, v, ints(cu), 16, o=o)
        assert ptb_lib.last_device_error() == 1, cu
    good = ptb_lib.swa_attention_packed(q, k, v, ints([0, 64, 128]), 16)
    o = torch.full_like(q, 5.0)
    ptb_lib.swa_attention_packed(q, k, v, ints([0, 64, 200]), 16, o=o)
    assert ptb_lib.last_device_error() == 1
    assert torch.equal(o[:64], good[:64]) and (o[64:] == 5).all()


def test_packed_empty(ptb_lib):
    q, k, v, _, _ = packed_inputs([8], None, 2, 2, 64, 95, tail=0)
    o = torch.full_like(q, 5.0)
    ptb_lib.swa_attention_packed(q, k, v, ints([0, 0, 0]), 16, o=o)
    assert (o == 5).all()
    assert ptb_lib.swa_attention_packed(q[:0], k[:0], v[:0], ints([0, 0]), 16).shape == (0, 2, 64)
    o = ptb_lib.swa_attention_packed(q, k[:0], v[:0], ints([0, 8]), 16, cu_seqlens_k=ints([0, 0]))
    assert (o == 0).all()


def test_packed_graph_replays_with_other_lengths(ptb_lib):
    q, k, v, _, _ = packed_inputs([200, 100], None, 4, 2, 64, 100, tail=0)
    cu = ints([0, 200, 300])
    o = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        ptb_lib.swa_attention_packed(q, k, v, cu, 64, o=o)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                ptb_lib.swa_attention_packed(q, k, v, cu, 64, o=o)
            graphs.append(g)
    torch.cuda.synchronize()
    for lens in ([0, 200, 300], [0, 3, 300], [0, 0, 0], [0, 150, 299]):
        cu.copy_(ints(lens))
        o.fill_(9)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want, bound, written = M.packed(M.to64(q), M.to64(k), M.to64(v), lens, lens, 64, 64 ** -0.5)
        held_to(o[torch.from_numpy(written)], want[written], bound[written])
        assert (o[torch.from_numpy(~written)] == 9).all()


@pytest.mark.parametrize("heads,kv", [(4, 2), (96, 48)])
def test_packed_workspace_of_the_caller(ptb_lib, heads, kv):
    """A caller's workspace with anything in it, used again and again; the small call needs none."""
    lens, d = [90, 3, 200], 32
    q, k, v, cu, _ = packed_inputs(lens, None, heads, kv, d, 105, tail=0)
    n = ptb_lib.swa_attention_packed_workspace_size(3, 293, heads, kv)
    assert (n > 0) == (kv == 48)
    ws = torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")
    want, bound, _ = M.packed(M.to64(q), M.to64(k), M.to64(v), cu, cu, 50, d ** -0.5)
    for _ in range(3):
        held_to(ptb_lib.swa_attention_packed(q, k, v, ints(cu), 50, workspace=ws), want, bound)
    if n:
        with pytest.raises(ptb_lib.PTBError, match="WORKSPACE"):
            ptb_lib.swa_attention_packed(q, k, v, ints(cu), 50, workspace=ws[:n - 16])


def test_packed_graph_of_a_listed_call(ptb_lib):
    """More items than SMs: the list kernel and the attention kernel in two graphs, with other
    lengths at each replay."""
    heads = kv = 60
    q, k, v, _, _ = packed_inputs([300], None, heads, kv, 32, 106, tail=0)
    cu = ints([0, 300, 300, 300])
    outs = [torch.zeros_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s, o in zip(streams, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ptb_lib.swa_attention_packed(q, k, v, cu, 40, o=o)
        graphs.append(g)
    for lens in ([0, 300, 300, 300], [0, 10, 11, 299], [0, 0, 150, 150]):
        cu.copy_(ints(lens))
        for o in outs:
            o.fill_(9)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want, bound, written = M.packed(M.to64(q), M.to64(k), M.to64(v), lens, lens, 40, 32 ** -0.5)
        for o in outs:
            held_to(o[torch.from_numpy(written)], want[written], bound[written])
            assert (o[torch.from_numpy(~written)] == 9).all()


def test_packed_offsets_that_go_back_stay_inside_the_list(ptb_lib):
    """Sequences that overlap name more query blocks than the list was sized for: recorded, and
    nothing outside o and the list is written."""
    heads = kv = 40
    q, k, v, _, _ = packed_inputs([512], None, heads, kv, 16, 107, tail=0)
    cu = ints([0, 512] * 40)
    n = ptb_lib.swa_attention_packed_workspace_size(79, 512, heads, kv)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    o = ptb_lib.swa_attention_packed(q, k, v, cu, 64, workspace=ws[:n])
    assert ptb_lib.last_device_error() == 1
    assert (ws[n:] == 0x5A).all() and torch.isfinite(o.float()).all()


def test_packed_on_two_streams(ptb_lib):
    sets = [packed_inputs([400, 70, 33], None, 8, 2, 64, 110 + 5 * i, tail=0) for i in range(2)]
    want = [ptb_lib.swa_attention_packed(q, k, v, ints(cu), 128) for q, k, v, cu, _ in sets]
    cus = [ints(s[3]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = []
    for _ in range(20):
        for s, (q, k, v, _, _), cu in zip(streams, sets, cus):
            outs.append(ptb_lib.swa_attention_packed(q, k, v, cu, 128, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


# ------------------------------------------------------------------------------- cache --

def new_cache(ptb_lib, pages, kv, page, d, bits, fill=0xFF):
    """A cache whose rows read as NaN until they are written."""
    n = ptb_lib.kv_page_size(kv, page, d, bits)
    return torch.full((pages, n), fill, dtype=torch.uint8, device="cuda")


def tables(lens, page, seed, spare=2):
    """A page table with the pages of all sequences in a random order, and the page count."""
    need = [-(-n // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def angles(positions, rot):
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


APPEND = [
    # new tokens a sequence, past, heads, kv heads, d, rotated channels, interleaved, page, bits
    ([1], [0], 1, 1, 128, 128, False, 16, 16),
    ([1, 1, 1], [0, 15, 16], 8, 2, 128, 128, False, 16, 4),
    ([3, 0, 40, 1], [14, 3, 100, 0], 6, 3, 96, 96, False, 32, 4),
    ([3, 0, 40, 1], [14, 3, 100, 0], 6, 3, 96, 64, True, 32, 16),
    ([70, 5], [0, 31], 5, 5, 64, 16, False, 64, 4),
    ([70, 5], [0, 31], 5, 5, 64, 32, True, 64, 4),
    ([33], [7], 4, 1, 32, 32, False, 16, 4),
    ([33], [7], 3, 2, 16, 16, False, 16, 16),
    ([20, 9], [0, 300], 2, 2, 128, 0, False, 128, 4),
    ([300, 1, 260], [0, 255, 256], 40, 40, 128, 128, False, 256, 16),
    ([1] * 40, list(range(40)), 16, 8, 128, 128, True, 16, 4),
]


def append_case(ptb_lib, new, past, heads, kv, d, rot, inter, page, bits, seed, tail=2):
    t = sum(new) + tail
    total = [a + n for a, n in zip(past, new)]
    table, pages = tables(total, page, seed)
    c = dict(q=normal((t, heads, d), seed), k=normal((t, kv, d), seed + 1), v=normal((t, kv, d), seed + 2),
             cache=new_cache(ptb_lib, pages, kv, page, d, bits), table=table, cu=cumulated(new), total=total)
    if rot:
        c["cos"], c["sin"] = angles(max(total) + 3, rot)
    return c


def run_append(ptb_lib, c, past, page, bits, inter, **kw):
    rot = {}
    if "cos" in c:
        rot = dict(cos=torch.from_numpy(c["cos"]).cuda(), sin=torch.from_numpy(c["sin"]).cuda())
    return ptb_lib.kv_append(c["q"], c["k"], c["v"], c["cache"], torch.from_numpy(c["table"]).cuda(),
                             ints(c["cu"]), ints(past), page, bits, interleaved=inter, **rot, **kw)


def model_append(c, past, kv, page, d, bits, inter):
    """The expected rotated q and k and the expected bytes of the cache."""
    q, k, v = (t.float().cpu().numpy() for t in (c["q"], c["k"], c["v"]))
    host = M.Cache(c["cache"].cpu().numpy().copy(), kv, page, d, bits)
    for b in range(len(past)):
        for i in range(c["cu"][b + 1] - c["cu"][b]):
            t, p = c["cu"][b] + i, past[b] + i
            if "cos" in c:
                q[t] = M.rotate32(q[t], c["cos"][p], c["sin"][p], inter)
                k[t] = M.rotate32(k[t], c["cos"][p], c["sin"][p], inter)
            for h in range(kv):
                host.put(c["table"][b, p // page], p % page, h, 0, k[t, h])
                host.put(c["table"][b, p // page], p % page, h, 1, v[t, h])
    return q, k, host


@pytest.mark.parametrize("new,past,heads,kv,d,rot,inter,page,bits", APPEND)
def test_append(ptb_lib, new, past, heads, kv, d, rot, inter, page, bits):
    """Bit for bit the definition's fp32 steps, nothing else in the cache touched; the rotation
    also within its 64-bit bound."""
    c = append_case(ptb_lib, new, past, heads, kv, d, rot, inter, page, bits, 200)
    q, k, host = model_append(c, past, kv, page, d, bits, inter)
    qo, ko = torch.full_like(c["q"], 7.0), torch.full_like(c["k"], 7.0)
    run_append(ptb_lib, c, past, page, bits, inter, q_out=qo, k_out=ko)
    n = c["cu"][-1]
    assert np.array_equal(qo[:n].float().cpu().numpy(), q[:n])
    assert np.array_equal(ko[:n].float().cpu().numpy(), k[:n])
    assert (qo[n:] == 7).all() and (ko[n:] == 7).all()
    assert np.array_equal(c["cache"].cpu().numpy(), host.raw)
    if rot:
        x = M.to64(c["q"])[:, :, :rot]
        pos = np.concatenate([np.arange(a, a + m) for a, m in zip(past, new)])
        ang = pos[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        a, b = (x[:n, :, 0::2], x[:n, :, 1::2]) if inter else (x[:n, :, :rot // 2], x[:n, :, rot // 2:])
        co, si = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y = M.to64(qo)[:n, :, :rot]
        ya, yb = (y[:, :, 0::2], y[:, :, 1::2]) if inter else (y[:, :, :rot // 2], y[:, :, rot // 2:])
        # tables and products rounded to fp32 (2^-24 each), the result to bf16
        err = 2.0 ** -22 * (np.abs(a) + np.abs(b)) + 1e-30
        assert (np.abs(ya - (a * co - b * si)) <= M.H * np.abs(a * co - b * si) + err).all()
        assert (np.abs(yb - (b * co + a * si)) <= M.H * np.abs(b * co + a * si) + err).all()


@pytest.mark.parametrize("bits,inter", [(16, False), (4, False), (4, True)])
def test_append_in_place_and_strided(ptb_lib, bits, inter):
    new, past, heads, kv, d, page = [40, 3], [5, 60], 4, 2, 128, 32
    c = append_case(ptb_lib, new, past, heads, kv, d, d, inter, page, bits, 210)
    u = normal((45, (heads + 2 * kv) * d), 211)
    c["q"], c["k"], c["v"] = (u[:, a * d:(a + n) * d].unflatten(1, (n, d))
                              for a, n in ((0, heads), (heads, kv), (heads + kv, kv)))
    before = u.clone()
    q, k, host = model_append(c, past, kv, page, d, bits, inter)
    run_append(ptb_lib, c, past, page, bits, inter, q_out=c["q"], k_out=c["k"])
    assert np.array_equal(c["q"][:43].float().cpu().numpy(), q[:43])
    assert np.array_equal(c["k"][:43].float().cpu().numpy(), k[:43])
    assert np.array_equal(c["cache"].cpu().numpy(), host.raw)
    assert torch.equal(u[43:], before[43:]) and torch.equal(c["v"], before[:, -kv * d:].unflatten(1, (kv, d)))


def test_append_keys_only(ptb_lib):
    c = append_case(ptb_lib, [20], [3], 2, 2, 64, 64, False, 16, 4, 220)
    _, k, host = model_append(c, [3], 2, 16, 64, 4, False)
    c["q"] = None
    q_out, k_out = run_append(ptb_lib, c, [3], 16, 4, False, keep_keys=False)
    assert q_out is None and k_out is None
    assert np.array_equal(c["cache"].cpu().numpy(), host.raw)


def test_append_4bit_special_groups(ptb_lib):
    """Constant groups, tiny and huge ranges, ties, and values that are not finite."""
    d, page = 128, 16
    c = append_case(ptb_lib, [8], [0], 1, 1, d, 0, False, page, 4, 230, tail=0)
    x = c["v"]
    x[0], x[1] = 0, -3.25
    x[2, 0, :64] = torch.linspace(0, 15, 64).to(torch.bfloat16)       # steps of 1/4: ties
    x[3, 0, 5], x[3, 0, 40], x[3, 0, 70] = float("nan"), float("inf"), float("-inf")
    x[4] *= 1e38
    x[4, 0, 0], x[4, 0, 1] = 3e38, -3e38                              # the range overflows
    x[5] *= 1e-39                                                     # subnormals
    x[6] = 1000 + x[6]                                                # a range far from zero
    x[7, 0] = 1.0
    x[7, 0, 3] = 1.0078125
    c["k"].copy_(x)
    _, _, host = model_append(c, [0], 1, page, d, 4, False)
    run_append(ptb_lib, c, [0], page, 4, False)
    assert np.array_equal(c["cache"].cpu().numpy(), host.raw)


def test_append_out_of_range_is_recorded(ptb_lib):
    new, past, page, d = [3, 2], [4, 9], 16, 64
    for what in ("page", "negative page", "table", "positions", "past", "offsets"):
        c = append_case(ptb_lib, new, past, 2, 1, d, d, False, page, 16, 240, tail=0)
        q, k, host = model_append(c, past, 1, page, d, 16, False)
        before = c["cache"].cpu().numpy().copy()
        p = list(past)
        if what == "page":
            c["table"][1, 0] = c["cache"].shape[0]
        elif what == "negative page":
            c["table"][1, 0] = -1
        elif what == "table":
            p[1] = 16 * c["table"].shape[1]
            c["cos"], c["sin"] = angles(p[1] + 5, d)
        elif what == "positions":
            c["cos"], c["sin"] = angles(9, d)
        elif what == "past":
            p[1] = -1
        else:
            c["cu"] = [0, 3, 6]  # past the tensors' five rows
        run_append(ptb_lib, c, p, page, 16, False)
        assert ptb_lib.last_device_error() == 1, what
        got = c["cache"].cpu().numpy()
        # the first sequence is written, the second nowhere
        page0 = c["table"][0, 0]
        assert np.array_equal(got[page0], host.raw[page0])
        rest = np.arange(len(got)) != page0
        assert np.array_equal(got[rest], before[rest]), what


@pytest.mark.parametrize("bits,d,page", [(16, 128, 16), (4, 128, 64), (4, 96, 16), (4, 32, 32), (16, 16, 256),
                                         (4, 64, 128)])
def test_gather_reads_what_append_wrote(ptb_lib, bits, d, page):
    new, past, kv = [70, 0, 1, 20], [0, 5, 33, 250], 3
    c = append_case(ptb_lib, new, past, 3, kv, d, d, False, page, bits, 250)
    _, _, host = model_append(c, past, kv, page, d, bits, False)
    run_append(ptb_lib, c, past, page, bits, False)
    start, lens = [10, 5, 33, 252], [60, 0, 1, 17]
    cu = cumulated(lens)
    k, v = (torch.full((cu[-1] + 4, kv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ptb_lib.kv_gather(c["cache"], torch.from_numpy(c["table"]).cuda(), ints(cu), ints(start), cu[-1] + 4, kv, d,
                      page, bits, k=k, v=v)
    assert (k[cu[-1]:] == 7).all() and (v[cu[-1]:] == 7).all()
    for which, got in ((0, k), (1, v)):
        got = got.float().cpu().numpy()
        for b in range(len(lens)):
            for i in range(lens[b]):
                p = start[b] + i
                for h in range(kv):
                    x = host.get(c["table"][b, p // page], p % page, h, which)[0]
                    # 4 bits: one fp32 rounding of the value, then one to bf16
                    assert np.array_equal(got[cu[b] + i, h], M.bf16_np(np.float32(x))), (which, b, i, h)


def test_gather_out_of_range_is_recorded(ptb_lib):
    c = append_case(ptb_lib, [20], [0], 1, 1, 64, 0, False, 16, 16, 260)
    run_append(ptb_lib, c, [0], 16, 16, False)
    for start, entry in ((-1, None), (1 << 20, None), (0, 99), (0, -7)):
        table = torch.from_numpy(c["table"]).cuda()
        if entry is not None:
            table[0, 0] = entry
        k = torch.full((3, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, 7.0)
        ptb_lib.kv_gather(c["cache"], table, ints([0, 3]), ints([start]), 3, 1, 64, 16, 16, k=k, v=v)
        assert ptb_lib.last_device_error() == 1
        assert (k == 7).all() and (v == 7).all()
    ptb_lib.kv_gather(c["cache"], torch.from_numpy(c["table"]).cuda(), ints([0, 4]), ints([0]), 3, 1, 64, 16, 16, k=k, v=v)
    assert ptb_lib.last_device_error() == 1 and (k == 7).all()


# --------------------------------------------------------------------- paged attention --

PAGED = [
    # cached lengths, heads, kv heads, d, window, page, bits
    ([1], 1, 1, 128, 1, 16, 16),
    ([1], 1, 1, 128, 1, 16, 4),
    ([2, 1, 3], 2, 2, 64, 2, 16, 4),
    ([15, 16, 17, 31, 32, 33], 4, 2, 128, 1 << 30, 16, 16),
    ([15, 16, 17, 31, 32, 33], 4, 2, 128, 1 << 30, 16, 4),
    ([63, 64, 65, 0, 129], 8, 1, 96, 50, 32, 16),
    ([63, 64, 65, 0, 129], 8, 1, 96, 50, 32, 4),
    ([300, 1, 128], 3, 1, 32, 100, 64, 4),
    ([300, 1, 128], 3, 1, 32, 100, 64, 16),
    ([77, 200], 5, 5, 16, 90, 16, 16),
    ([500], 8, 8, 128, 300, 128, 4),
    ([500], 8, 8, 64, 300, 256, 16),
    ([257, 90], 16, 1, 128, 1 << 20, 16, 4),
    ([257, 90], 16, 1, 128, 1 << 20, 16, 16),
    ([100, 40], 12, 1, 64, 64, 16, 4),
    ([60, 33], 40, 2, 96, 48, 32, 4),
    ([60, 33], 71, 1, 64, 48, 32, 16),
    ([2500, 3], 4, 2, 64, 2400, 64, 4),
    ([2500, 3], 4, 2, 64, 2400, 64, 16),
    ([20 + 3 * i for i in range(50)], 2, 1, 64, 33, 16, 4),
]


def filled(ptb_lib, lens, kv, d, page, bits, seed, heads=1):
    """A cache filled by kv_append with `lens` tokens a sequence; unwritten rows read as NaN."""
    c = append_case(ptb_lib, lens, [0] * len(lens), 1, kv, d, 0, False, page, bits, seed)
    c["k"].mul_(1.5)
    run_append(ptb_lib, c, [0] * len(lens), page, bits, False)
    c["host"] = M.Cache(c["cache"].cpu().numpy(), kv, page, d, bits)
    c["q1"] = normal((len(lens), heads, d), seed + 3)
    c["table_d"] = torch.from_numpy(c["table"]).cuda()
    return c


@pytest.mark.parametrize("lens,heads,kv,d,window,page,bits", PAGED)
def test_paged(ptb_lib, lens, heads, kv, d, window, page, bits):
    c = filled(ptb_lib, lens, kv, d, page, bits, 300, heads)
    o = ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], ints(lens), kv, page, bits, window)
    want, bound = M.paged(M.to64(c["q1"]), c["host"], c["table"], lens, window, d ** -0.5)
    held_to(o, want, bound)


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_leaves_old_pages_alone(ptb_lib, bits):
    """Entries of pages that the window has left behind may hold anything."""
    lens, w, page = [200, 97], 40, 16
    c = filled(ptb_lib, lens, 2, 64, page, bits, 310, 4)
    want = ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], ints(lens), 2, page, bits, w)
    for b, n in enumerate(lens):
        c["table_d"][b, :(n - w) // page] = -12345
    got = ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], ints(lens), 2, page, bits, w)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("heads", [2, 16])
def test_paged_rows_that_the_mask_leaves_out(ptb_lib, bits, heads):
    """Rows before the window and past the length hold NaN; a NaN inside the window shows."""
    lens, w, page, d = [45, 70], 20, 32, 64
    c = filled(ptb_lib, lens, 1, d, page, bits, 320, heads)
    want, bound = M.paged(M.to64(c["q1"]), c["host"], c["table"], lens, w, d ** -0.5)
    raw = c["cache"].cpu().numpy().copy()
    host = M.Cache(raw, 1, page, d, bits)
    for b, n in enumerate(lens):
        for p in range(0, n - w):
            for which in (0, 1):
                host.put(c["table"][b, p // page], p % page, 0, which, np.full(d, np.nan, np.float32))
    cache = torch.from_numpy(raw).cuda()
    o = ptb_lib.swa_attention_paged(c["q1"], cache, c["table_d"], ints(lens), 1, page, bits, w)
    held_to(o, want, bound)
    host.put(c["table"][1, 60 // page], 60 % page, 0, 1, np.full(d, np.nan, np.float32))
    cache = torch.from_numpy(raw).cuda()
    o = M.to64(ptb_lib.swa_attention_paged(c["q1"], cache, c["table_d"], ints(lens), 1, page, bits, w))
    assert np.isfinite(o[0]).all() and np.isnan(o[1]).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_strides_scale_and_in_place(ptb_lib, bits):
    lens, page = [33, 80, 5], 16
    c = filled(ptb_lib, lens, 2, 64, page, bits, 330, 6)
    big = normal((3, 20, 64), 331)
    q = big[:, 3:15:2]
    want, bound = M.paged(M.to64(q), c["host"], c["table"], lens, 60, 0.3)
    before = big.clone()
    o = ptb_lib.swa_attention_paged(q, c["cache"], c["table_d"], ints(lens), 2, page, bits, 60, scale=0.3, o=q)
    assert o is q
    held_to(q, want, bound)
    keep = [i for i in range(20) if i not in range(3, 15, 2)]
    assert torch.equal(big[:, keep], before[:, keep])


def test_paged_out_of_range_is_recorded(ptb_lib):
    lens, page = [40, 40], 16
    for bits in (16, 4):
        c = filled(ptb_lib, lens, 1, 64, page, bits, 340, 4)
        good = ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], ints(lens), 1, page, bits, 99)
        for n, what in ((-1, "length"), (10 ** 6, "length"), (40, "page")):
            table = c["table_d"].clone()
            if what == "page":
                table[1, 1] = 1 << 30
            o = ptb_lib.swa_attention_paged(c["q1"], c["cache"], table, ints([40, n]), 1, page, bits, 99)
            assert ptb_lib.last_device_error() == 1, (bits, n, what)
            assert torch.equal(o[0], good[0])
            if what == "length":
                assert (o[1] == 0).all()
            else:  # the keys of the bad page are left out
                assert torch.isfinite(o[1].float()).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_graphs_and_streams(ptb_lib, bits):
    """Captured once, replayed with other lengths; two graphs and two streams side by side."""
    lens, page, kv, d = [700, 64, 300], 16, 2, 64
    c = filled(ptb_lib, lens, kv, d, page, bits, 350, 8)
    n = ints(lens)
    o = [torch.zeros_like(c["q1"]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for s, out in zip(streams, o):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], n, kv, page, bits, 512, o=out)
        graphs.append(g)
    for ls in (lens, [1, 0, 299], [512, 64, 17]):
        n.copy_(ints(ls))
        want, bound = M.paged(M.to64(c["q1"]), c["host"], c["table"], ls, 512, d ** -0.5)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for out in o:
            held_to(out, want, bound)


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_queries_that_are_not_finite_or_zero(ptb_lib, bits):
    """A NaN or an infinity in a query stays in its row; a query of zeros averages the values; tiny
    and huge queries keep their weights."""
    lens, page, d = [70, 40, 33, 90], 16, 64
    c = filled(ptb_lib, lens, 1, d, page, bits, 365, 4)
    q = c["q1"]
    q[0, 1, 3], q[0, 2, 60] = float("nan"), float("inf")
    q[1] = 0
    q[2] *= 1e-20
    q[3] *= 1e4
    o = M.to64(ptb_lib.swa_attention_paged(q, c["cache"], c["table_d"], ints(lens), 1, page, bits, 1000, scale=0.01))
    assert np.isnan(o[0, 1:3]).all()
    q[0, 1:3] = 0
    want, bound = M.paged(M.to64(q), c["host"], c["table"], lens, 1000, 0.01)
    o[0, 1:3] = want[0, 1:3]
    assert (np.abs(o - want) <= bound).all()


@pytest.mark.parametrize("power", [-126, -100, -40, 0, 40, 100, 116])
def test_paged_4bit_query_range(ptb_lib, power):
    """Queries of any magnitude with a scale that makes up for it; beyond 2^119 they give NaN."""
    lens, page, d = [70, 40], 16, 64
    c = filled(ptb_lib, lens, 2, d, page, 4, 369, 4)
    q = c["q1"].clamp(-3.9, 3.9)
    q[1, 1] = 0
    scale = 2.0 ** max(-3 - power, -126)
    q = (q.double() * 2.0 ** power).to(torch.bfloat16)
    o = ptb_lib.swa_attention_paged(q, c["cache"], c["table_d"], ints(lens), 2, page, 4, 1000, scale=scale)
    want, bound = M.paged(M.to64(q), c["host"], c["table"], lens, 1000, scale)
    held_to(o, want, bound)
    q[0, 2, 7] = 2.0 ** 119
    o = ptb_lib.swa_attention_paged(q, c["cache"], c["table_d"], ints(lens), 2, page, 4, 1000, scale=scale)
    assert torch.isnan(o[0, 2]).all() and torch.isfinite(o[0, :2]).all() and torch.isfinite(o[1]).all()


def test_paged_workspace_of_the_caller(ptb_lib):
    c = filled(ptb_lib, [500, 70], 2, 64, 32, 4, 366, 4)
    n = ptb_lib.swa_attention_paged_workspace_size(2, 4, 2, 64)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    args = (c["q1"], c["cache"], c["table_d"], ints([500, 70]), 2, 32, 4, 300)
    want = ptb_lib.swa_attention_paged(*args)
    for _ in range(3):
        assert torch.equal(ptb_lib.swa_attention_paged(*args, workspace=ws), want)
    with pytest.raises(ptb_lib.PTBError, match="WORKSPACE"):
        ptb_lib.swa_attention_paged(*args, workspace=ws[:n - 16])
    with pytest.raises(ValueError, match="workspace"):
        ptb_lib.swa_attention_paged(*args, workspace=ws.cpu())


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_long_tables(ptb_lib, bits):
    """A table with room for long sequences has the join launched early.  Calls one behind the other
    on one stream share a workspace, eager and replayed; one writes over its own queries."""
    lens, page, kv, d, w = [3000, 1, 700], 16, 2, 128, 1 << 20
    c = filled(ptb_lib, lens, kv, d, page, bits, 368, 8)
    wide = torch.full((3, 1 << 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :c["table"].shape[1]] = c["table_d"]
    n = ints(lens)
    want, bound = M.paged(M.to64(c["q1"]), c["host"], c["table"], lens, w, d ** -0.5)
    one = ptb_lib.swa_attention_paged(c["q1"], c["cache"], c["table_d"], n, kv, page, bits, w)
    held_to(one, want, bound)
    ws = torch.empty(ptb_lib.swa_attention_paged_workspace_size(3, 8, kv, d), dtype=torch.uint8, device="cuda")
    qs = [c["q1"] * f for f in (1.0, -1.0, 2.0)]
    alone = [ptb_lib.swa_attention_paged(q, c["cache"], c["table_d"], n, kv, page, bits, w) for q in qs]
    o = [q.clone() for q in qs]

    def calls():
        for q, out in zip(qs, o):
            ptb_lib.swa_attention_paged(q, c["cache"], wide, n, kv, page, bits, w, o=out, workspace=ws)

    for _ in range(20):
        calls()
    for got, other in zip(o, alone):
        assert torch.equal(got, other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for out in o:
        out.zero_()
    for _ in range(5):
        g.replay()
    for got, other in zip(o, alone):
        assert torch.equal(got, other)
    q = qs[0].clone()
    assert torch.equal(ptb_lib.swa_attention_paged(q, c["cache"], wide, n, kv, page, bits, w, o=q), alone[0])


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_sequences_that_share_pages(ptb_lib, bits):
    """Two sequences of one prefix read the same pages."""
    page, d = 16, 64
    c = filled(ptb_lib, [64, 100], 2, d, page, bits, 367, 4)
    c["table"][1, :4] = c["table"][0, :4]
    o = ptb_lib.swa_attention_paged(c["q1"], c["cache"], torch.from_numpy(c["table"]).cuda(), ints([64, 100]), 2, page, bits, 1 << 20)
    want, bound = M.paged(M.to64(c["q1"]), c["host"], c["table"], [64, 100], 1 << 20, d ** -0.5)
    held_to(o, want, bound)


def test_paged_same_bits_every_time(ptb_lib):
    for bits in (16, 4):
        c = filled(ptb_lib, [900, 30], 2, 128, 32, bits, 360, 8)
        args = (c["q1"], c["cache"], c["table_d"], ints([900, 30]), 2, 32, bits, 4096)
        first = ptb_lib.swa_attention_paged(*args)
        for _ in range(5):
            assert torch.equal(ptb_lib.swa_attention_paged(*args), first)


def test_cache_beyond_32_bit_offsets(ptb_lib):
    """Rows whose byte offset in the cache passes 2^32."""
    kv, d, page, bits = 8, 128, 256, 16
    n = ptb_lib.kv_page_size(kv, page, d, bits)
    pages = (1 << 32) // n + 3
    cache = torch.empty(pages, n, dtype=torch.uint8, device="cuda")
    table = ints([pages - 1, pages - 2])[None]
    q, k, v = normal((300, 16, d), 370), normal((300, kv, d), 371), normal((300, kv, d), 372)
    ptb_lib.kv_append(q, k, v, cache, table, ints([0, 300]), ints([0]), page, bits)
    kr, vr = ptb_lib.kv_gather(cache, table, ints([0, 300]), ints([0]), 300, kv, d, page, bits)
    assert torch.equal(kr, k) and torch.equal(vr, v)
    o = ptb_lib.swa_attention_paged(q[299:], cache, table, ints([300]), kv, page, bits, 128)
    want, bound, _ = M.packed(M.to64(q), M.to64(k), M.to64(v), [0, 300], [0, 300], 128, d ** -0.5)
    held_to(o, want[299:], bound[299:])


# ---------------------------------------------------------------- as they would be used --

@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_in_two_chunks(ptb_lib, bits):
    """A later chunk of a prompt attends to the earlier one read back from the cache."""
    first, second, heads, kv, d, page, w = [50, 7], [30, 41], 8, 2, 64, 16, 60
    total = [a + b for a, b in zip(first, second)]
    table, pages = tables(total, page, 400)
    cache = new_cache(ptb_lib, pages, kv, page, d, bits)
    table = torch.from_numpy(table).cuda()
    cos, sin = (torch.from_numpy(t).cuda() for t in angles(200, d))
    parts = []
    for i, (lens, past) in enumerate(((first, [0, 0]), (second, first))):
        t = sum(lens)
        q, k, v = normal((t, heads, d), 401 + 3 * i), normal((t, kv, d), 402 + 3 * i), normal((t, kv, d), 403 + 3 * i)
        q, _ = ptb_lib.kv_append(q, k, v, cache, table, ints(cumulated(lens)), ints(past), page, bits, cos=cos, sin=sin)
        parts.append(q)
    cu_k = cumulated(total)
    k, v = ptb_lib.kv_gather(cache, table, ints(cu_k), ints([0, 0]), cu_k[-1], kv, d, page, bits)
    cu_q = cumulated(second)
    o = ptb_lib.swa_attention_packed(parts[1], k, v, ints(cu_q), w, cu_seqlens_k=ints(cu_k))
    want, bound, _ = M.packed(M.to64(parts[1]), M.to64(k), M.to64(v), cu_q, cu_k, w, d ** -0.5)
    held_to(o, want, bound)
    # the last token once more, as a decode step over the cache
    last = torch.stack([parts[1][cu_q[1] - 1], parts[1][cu_q[2] - 1]])
    o1 = ptb_lib.swa_attention_paged(last, cache, table, ints(total), kv, page, bits, w)
    host = M.Cache(cache.cpu().numpy(), kv, page, d, bits)
    want, bound = M.paged(M.to64(last), host, table.cpu().numpy(), total, w, d ** -0.5)
    held_to(o1, want, bound)


def test_ptb_layer_answers_token_by_token(ptb_lib):
    """The PTB layer on packed prompts, then one token at a time over the cache, against the fp64
    layer on the whole sequences."""
    heads, d, ffn, w, page = 4, 64, 512, 40, 16
    hidden = heads * d
    prompts, steps = [37, 1, 90], 6
    cfg = workloads.small_ptb(1, max(prompts) + steps, hidden, heads, ffn, w, seed=5)
    host = workloads.ptb_inputs(cfg)
    dev = {n: t.cuda() for n, t in host.items()}
    xs = [workloads.normal_bf16((n + steps, hidden), seed=50 + i) for i, n in enumerate(prompts)]
    table, pages = tables([n + steps for n in prompts], page, 410)
    cache, table = new_cache(ptb_lib, pages, heads, page, d, 16), torch.from_numpy(table).cuda()

    def layer(x, attend, cu, past):
        xn = ptb_lib.layernorm(x, dev["ln_gamma"], dev["ln_beta"])
        u = ptb_lib.gemm_qkv_up(xn, dev["w_qkv"], dev["w_up"])
        q, k, v = (u[:, i * hidden:(i + 1) * hidden].unflatten(1, (heads, d)) for i in range(3))
        ptb_lib.kv_append(q, k, v, cache, table, cu, past, page, 16, q_out=q, k_out=k)
        ctx = attend(q, k, v)
        return ptb_lib.gemm_out_down(ctx.flatten(1), u[:, 3 * hidden:], dev["w_o"], dev["w_down"], x)

    cu = ints(cumulated(prompts))
    x = torch.cat([t[:n] for t, n in zip(xs, prompts)]).cuda()
    y = layer(x, lambda q, k, v: ptb_lib.swa_attention_packed(q, k, v, cu, w), cu, ints([0] * 3))
    got = [[y[a:b]] for a, b in zip(cumulated(prompts), cumulated(prompts)[1:])]
    one = ints(range(4))
    for s in range(steps):
        x = torch.stack([t[n + s] for t, n in zip(xs, prompts)]).cuda()
        past = ints([n + s for n in prompts])
        y = layer(x, lambda q, k, v: ptb_lib.swa_attention_paged(q, cache, table, past + 1, heads, page, 16, w), one, past)
        for g, row in zip(got, y):
            g.append(row[None])
    f = {n: t.float().numpy() for n, t in host.items()}
    for x, g in zip(xs, got):
        want = oracle.ptb_forward(x.float().numpy()[None], f["ln_gamma"], f["ln_beta"], f["w_qkv"], f["w_o"],
                                  f["w_up"], f["w_down"], heads, w)
        assert_close(torch.cat(g).float().cpu().numpy()[None], want, "layer")
