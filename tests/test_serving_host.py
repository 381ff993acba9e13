"""Refusals of the serving entry points, on the host: nothing here touches a device, the pointers
are never read."""

import pytest
import torch

FAKE = 1 << 20
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
NO_DEVICE = (5, 7, 8)  # past the host checks


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import block_sliding_window_gb300 as bsw
    return bsw.load()


def past_checks(st):
    return st in NO_DEVICE or (torch.cuda.is_available() and st == 0)


@pytest.mark.parametrize("kv,page,d,bits,want", [
    (8, 64, 128, 16, 2 * 8 * 64 * 256), (8, 64, 128, 4, 2 * 8 * 64 * (64 + 16)), (1, 16, 32, 4, 2 * 16 * 20),
    (3, 256, 16, 16, 2 * 3 * 256 * 32), (2, 16, 96, 4, 2 * 2 * 16 * 60),
    (0, 64, 128, 16, 0), (8, 8, 128, 16, 0), (8, 48, 128, 16, 0), (8, 512, 128, 16, 0), (8, 64, 80, 16, 0),
    (8, 64, 128, 8, 0), (8, 64, 16, 4, 0), (70000, 64, 128, 16, 0),
])
def test_page_size(lib, kv, page, d, bits, want):
    assert lib.ptb_kv_page_size(kv, page, d, bits) == want


def append(lib, **kw):
    a = dict(q=FAKE, q_st=256, q_sh=64, k=FAKE * 2, k_st=128, k_sh=64, v=FAKE * 3, v_st=128, v_sh=64, cos=FAKE, sin=FAKE,
             positions=100, rot=64, inter=0, cu=FAKE, past=FAKE, batch=2, tokens=0, heads=4, kv=2, d=64, qo=FAKE * 4,
             qo_st=256, qo_sh=64, ko=FAKE * 5, ko_st=128, ko_sh=64, cache=FAKE * 6, pages=10, table=FAKE, stride=5, n=5,
             page=16, bits=16)
    a.update(kw)
    return lib.ptb_kv_append(a["q"], a["q_st"], a["q_sh"], a["k"], a["k_st"], a["k_sh"], a["v"], a["v_st"], a["v_sh"],
                             a["cos"], a["sin"], a["positions"], a["rot"], a["inter"], a["cu"], a["past"], a["batch"],
                             a["tokens"], a["heads"], a["kv"], a["d"], a["qo"], a["qo_st"], a["qo_sh"], a["ko"], a["ko_st"],
                             a["ko_sh"], a["cache"], a["pages"], a["table"], a["stride"], a["n"], a["page"], a["bits"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None, tokens=1), ARG), (dict(v=None, tokens=1), ARG), (dict(cu=None), ARG), (dict(past=None), ARG),
    (dict(cache=None), ARG), (dict(table=None), ARG), (dict(batch=0), ARG), (dict(tokens=-1), ARG), (dict(kv=0), ARG),
    (dict(heads=0), ARG), (dict(qo=None), ARG), (dict(q=None), ARG), (dict(cos=None), ARG), (dict(positions=0), ARG),
    (dict(rot=-16), ARG), (dict(inter=2), ARG), (dict(stride=4), ARG), (dict(pages=0), ARG), (dict(n=0), ARG),
    (dict(qo=FAKE, qo_st=512), ARG), (dict(ko=FAKE * 2, ko_sh=128), ARG), (dict(qo=FAKE * 2), ARG), (dict(ko=FAKE * 3), ARG),
    (dict(ko=FAKE * 4), ARG),
    (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(d=80), SHAPE), (dict(page=24), SHAPE), (dict(bits=8), SHAPE),
    (dict(d=16, bits=4, rot=0), SHAPE), (dict(tokens=1 << 40), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(q=FAKE + 8), ALIGN), (dict(k_st=130), ALIGN), (dict(v_sh=60), ALIGN), (dict(v_sh=0), ALIGN), (dict(k_st=-64), ALIGN),
    (dict(cache=FAKE + 8), ALIGN), (dict(cu=FAKE + 2), ALIGN), (dict(cos=FAKE + 4), ALIGN),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_accepts(lib):
    for kw in ({}, dict(qo=FAKE), dict(ko=FAKE * 2), dict(q=None, qo=None), dict(ko=None), dict(rot=0, cos=None, sin=None),
               dict(bits=4), dict(rot=16, inter=1)):
        assert past_checks(append(lib, **kw)), kw


def gather(lib, **kw):
    a = dict(cache=FAKE, pages=10, table=FAKE, stride=5, n=5, cu=FAKE, start=FAKE, batch=2, tokens=0, kv=2, d=64, page=16,
             bits=4, k=FAKE * 2, k_st=128, k_sh=64, v=FAKE * 3, v_st=128, v_sh=64)
    a.update(kw)
    return lib.ptb_kv_gather(a["cache"], a["pages"], a["table"], a["stride"], a["n"], a["cu"], a["start"], a["batch"],
                             a["tokens"], a["kv"], a["d"], a["page"], a["bits"], a["k"], a["k_st"], a["k_sh"], a["v"],
                             a["v_st"], a["v_sh"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), ARG), (dict(cu=None), ARG), (dict(start=None), ARG), (dict(batch=0), ARG), (dict(tokens=-1), ARG),
    (dict(k=None, tokens=4), ARG), (dict(v=FAKE * 2), ARG), (dict(d=48), SHAPE), (dict(page=15), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(k=FAKE + 2), ALIGN), (dict(v_st=7), ALIGN), (dict(table=FAKE + 1), ALIGN),
])
def test_gather_refuses(lib, kw, code):
    assert gather(lib, **kw) == code


def test_gather_accepts(lib):
    assert past_checks(gather(lib)) and past_checks(gather(lib, bits=16, d=16))


def packed(lib, **kw):
    a = dict(q=FAKE, q_st=256, q_sh=64, k=FAKE * 2, k_st=128, k_sh=64, v=FAKE * 3, v_st=128, v_sh=64, cu=FAKE, cuk=None,
             batch=2, tq=0, tk=100, heads=4, kv=2, d=64, window=8, scale=0.0, o=FAKE * 4, o_st=256, o_sh=64, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.swa_attention_packed(a["q"], a["q_st"], a["q_sh"], a["k"], a["k_st"], a["k_sh"], a["v"], a["v_st"], a["v_sh"],
                                    a["cu"], a["cuk"], a["batch"], a["tq"], a["tk"], a["heads"], a["kv"], a["d"],
                                    a["window"], a["scale"], a["o"], a["o_st"], a["o_sh"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, tq=5), ARG), (dict(k=None), ARG), (dict(cu=None), ARG), (dict(batch=0), ARG), (dict(tq=-1), ARG),
    (dict(tk=-1), ARG), (dict(heads=0), ARG), (dict(kv=0), ARG), (dict(window=0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(o=FAKE * 2), ARG), (dict(o=FAKE * 3), ARG),
    (dict(o=FAKE, o_st=512), ARG),
    (dict(heads=3), SHAPE), (dict(heads=258), SHAPE), (dict(d=80), SHAPE), (dict(d=0), SHAPE), (dict(batch=70000), SHAPE),
    (dict(tq=1 << 31), SHAPE), (dict(tk=1 << 31), SHAPE),
    (dict(q=FAKE + 2), ALIGN), (dict(k_st=66), ALIGN), (dict(v_sh=-64), ALIGN), (dict(o_sh=4), ALIGN), (dict(cu=FAKE + 3), ALIGN),
])
def test_packed_refuses(lib, kw, code):
    assert packed(lib, **kw) == code


def test_packed_workspace(lib):
    n = lib.swa_attention_packed_workspace_size(2, 100, 4, 2)
    assert n % 256 == 0
    assert past_checks(packed(lib))
    if n:
        kw = dict(tq=100)
        assert packed(lib, ws=None, **kw) == ARG
        assert packed(lib, wsb=n - 1, **kw) == WORKSPACE
        assert packed(lib, ws=FAKE + 64, **kw) == ALIGN
    for bad in ((0, 100, 4, 2), (2, -1, 4, 2), (2, 100, 3, 2), (2, 100, 4, 0)):
        assert lib.swa_attention_packed_workspace_size(*bad) == 0


def paged(lib, **kw):
    a = dict(q=FAKE, q_sb=256, q_sh=64, cache=FAKE * 2, pages=10, table=FAKE, stride=5, n=5, lens=FAKE, batch=2, heads=4,
             kv=2, d=64, page=16, bits=4, window=8, scale=0.0, o=FAKE * 4, o_sb=256, o_sh=64, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.swa_attention_paged(a["q"], a["q_sb"], a["q_sh"], a["cache"], a["pages"], a["table"], a["stride"], a["n"],
                                   a["lens"], a["batch"], a["heads"], a["kv"], a["d"], a["page"], a["bits"], a["window"],
                                   a["scale"], a["o"], a["o_sb"], a["o_sh"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(cache=None), ARG), (dict(lens=None), ARG), (dict(batch=0), ARG), (dict(heads=0), ARG),
    (dict(kv=0), ARG), (dict(window=0), ARG), (dict(scale=-0.5), ARG), (dict(scale=float("inf")), ARG), (dict(stride=3), ARG),
    (dict(o=FAKE, o_sb=512), ARG), (dict(heads=5), SHAPE), (dict(d=48), SHAPE), (dict(bits=2), SHAPE),
    (dict(d=16), SHAPE), (dict(page=100), SHAPE), (dict(batch=70000), SHAPE), (dict(q=FAKE + 4), ALIGN),
    (dict(o_sh=36), ALIGN), (dict(lens=FAKE + 1), ALIGN), (dict(cache=FAKE * 2 + 4), ALIGN),
])
def test_paged_refuses(lib, kw, code):
    assert paged(lib, **kw) == code


def test_paged_workspace(lib):
    n = lib.swa_attention_paged_workspace_size(2, 4, 2, 64)
    assert n % 256 == 0
    if n:
        assert paged(lib, ws=None) == ARG
        assert paged(lib, wsb=n - 1) == WORKSPACE
        assert paged(lib, ws=FAKE + 128) == ALIGN
    for bad in ((0, 4, 2, 64), (2, 3, 2, 64), (2, 4, 2, 80), (70000, 4, 2, 64)):
        assert lib.swa_attention_paged_workspace_size(*bad) == 0


def test_binding_refuses_cpu_tensors(lib):
    import block_sliding_window_gb300 as bsw
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(2, 2 * 2 * 16 * 128, dtype=torch.uint8)
    for call in (lambda: bsw.swa_attention_packed(x, x, x, i, 4),
                 lambda: bsw.swa_attention_paged(x, cache, i[None], i, 2, 16, 16, 4),
                 lambda: bsw.kv_append(x, x, x, cache, i[None], i, i, 16, 16),
                 lambda: bsw.kv_gather(cache, i[None], i, i, 4, 2, 64, 16, 16, k=x, v=x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    for bad in ((0, 16, 64, 16), (2, 20, 64, 16), (2, 16, 64, 5), (2, 16, 16, 4)):
        with pytest.raises(ValueError):
            bsw.kv_page_size(*bad)


def test_search_for_a_token_of_a_sequence():
    """The warp's 32-way search of a token's sequence, step by step on the host."""
    import random

    def find(cu, batch, t):
        lo, n = 0, batch
        while n > 0:
            step = (n + 31) >> 5
            votes = [(lo + lane * step + step - 1 >= lo + n) or cu[lo + lane * step + step] > t for lane in range(32)]
            if not any(votes):
                return lo + n
            f = votes.index(True)
            if step == 1:
                return min(lo + f, batch)
            if f * step >= n:
                return lo + n
            lo, n = lo + f * step, min(step, n - f * step)
        return lo

    r = random.Random(1)
    for _ in range(3000):
        batch = r.choice([1, 2, 31, 32, 33, 64, 65, 500, 1024, 1025, 3000])
        cu = [0]
        for _ in range(batch):
            cu.append(cu[-1] + r.choice([0, 0, 1, 2, 50]))
        t = r.randint(0, cu[-1] + 2)
        want = next((b for b in range(batch) if cu[b + 1] > t), batch)
        assert find(cu, batch, t) == want, (batch, t)
