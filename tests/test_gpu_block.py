"""The gated feed-forward, the norms around a block and the 8-bit checkpoints on the GPU, element by
element against the 64-bit model and the bounds of tests/block_model.py."""
import ctypes
import math
import threading

import pytest
import torch

from tests import block_model as M

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(ptb_lib):
    ptb_lib.last_device_error()
    yield
    assert ptb_lib.last_device_error() == 0, "a kernel recorded a device-side error"


def normal(*shape, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(torch.bfloat16).cuda()


def padded(t, ld, offset=0):
    """The same values in rows of stride ld that begin at column `offset` of a buffer of NaN."""
    buf = torch.full((t.shape[0], ld), math.nan, dtype=t.dtype, device=t.device)
    v = buf[:, offset:offset + t.shape[1]]
    v.copy_(t)
    return v, buf


# ------------------------------------------------------------------ checkpoints --

@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (2, 2048), (5, 1056), (77, 320), (700, 5120), (40000, 32)])
def test_checkpoint_codes(ptb_lib, rows, cols):
    x = normal(rows, cols, seed=rows + cols) * torch.exp2(torch.randint(-20, 20, (rows, 1)).float()).cuda()
    x = x.to(torch.bfloat16)
    if rows > 2:
        x[0, :32] = 0
        x[1, :16] = 127.5
        x[2, 0] = math.inf
        x[2, 32:64] = math.nan if cols > 32 else 1.0
    codes, exps = ptb_lib.checkpoint_pack(x)
    wc, we = M.pack(M.d(x))
    assert torch.equal(exps.cpu(), we) and torch.equal(codes.cpu(), wc)
    back = ptb_lib.checkpoint_unpack(codes, exps)
    want = M.unpack(wc, we)
    assert torch.equal(torch.nan_to_num(M.d(back), nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_checkpoint_magnitudes(ptb_lib):
    # every exponent that bf16 has, subnormal numbers and the largest among them
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16).reshape(-1, 32).cuda()
    x = torch.cat([x, -x], 1).contiguous()
    codes, exps = ptb_lib.checkpoint_pack(x)
    wc, we = M.pack(M.d(x))
    assert torch.equal(exps.cpu(), we) and torch.equal(codes.cpu(), wc)
    back, want = M.d(ptb_lib.checkpoint_unpack(codes, exps)), M.unpack(wc, we)
    assert torch.equal(torch.nan_to_num(back, nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_checkpoint_strides(ptb_lib):
    x, _ = padded(normal(9, 96, seed=1), 136, 8)
    cbuf = torch.full((9, 160), 99, dtype=torch.int8, device="cuda")
    ebuf = torch.full((9, 7), 99, dtype=torch.uint8, device="cuda")
    codes, exps = ptb_lib.checkpoint_pack(x, codes=cbuf[:, 16:112], exps=ebuf[:, 1:4])
    wc, we = M.pack(M.d(x))
    assert torch.equal(codes.cpu(), wc) and torch.equal(exps.cpu(), we)
    assert (cbuf[:, :16] == 99).all() and (cbuf[:, 112:] == 99).all()
    assert (ebuf[:, :1] == 99).all() and (ebuf[:, 4:] == 99).all()
    out = torch.zeros(9, 128, dtype=torch.bfloat16, device="cuda")
    ptb_lib.checkpoint_unpack(codes, exps, x=out[:, 8:104])
    assert torch.equal(M.d(out[:, 8:104]), M.unpack(wc, we)) and (out[:, :8] == 0).all() and (out[:, 104:] == 0).all()


def test_checkpoint_shapes(ptb_lib):
    x = normal(2, 3, 64, seed=4)
    codes, exps = ptb_lib.checkpoint_pack(x)
    assert codes.shape == (2, 3, 64) and exps.shape == (2, 3, 2)
    assert ptb_lib.checkpoint_unpack(codes, exps).shape == x.shape
    none = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    codes, exps = ptb_lib.checkpoint_pack(none)
    assert codes.shape == (0, 64) and exps.shape == (0, 2) and ptb_lib.checkpoint_unpack(codes, exps).shape == (0, 64)


# --------------------------------------------------------------------- the norms --

NORMS = [
    # rows, hidden, gates, post, pre
    (1, 8, 0, 1, 1), (1, 5120, 1, 1, 1), (2, 24, 2, 1, 1), (3, 64, 1, 1, 1), (5, 256, 0, 0, 1), (6, 264, 3, 1, 0),
    (7, 512, 1, 0, 0), (4, 1024, 2, 1, 1), (9, 1032, 1, 1, 1), (12, 2048, 4, 1, 1), (5, 5120, 0, 1, 1), (300, 320, 3, 1, 1),
    (170, 6144, 2, 1, 1), (10, 6152, 1, 1, 1), (6, 8192, 2, 1, 1), (5, 12288, 5, 1, 1), (3, 12296, 0, 1, 1),
    (4, 16384, 2, 1, 1), (2, 20480, 1, 1, 0), (3, 24584, 1, 1, 1), (2, 32768, 2, 1, 1), (1000, 128, 500, 1, 1),
    (400, 96, 1, 1, 1), (5000, 32, 1, 0, 1),
]


def norm_inputs(rows, n, gates, post, pre, rms, seed=0):
    s = dict(x=normal(rows, n, seed=seed, std=2), o=normal(rows, n, seed=seed + 1, std=0.7, mean=0.2), post_gamma=None,
             post_beta=None, gate=None, pre_gamma=None, pre_beta=None)
    if post:
        s["post_gamma"] = normal(n, seed=seed + 2, std=0.2, mean=1)
        s["post_beta"] = None if rms else normal(n, seed=seed + 3, std=0.3)
    if gates:
        s["gate"] = normal(gates, n, seed=seed + 4, std=0.5)
    if pre:
        s["pre_gamma"] = normal(n, seed=seed + 5, std=0.2, mean=1)
        s["pre_beta"] = None if rms else normal(n, seed=seed + 6, std=0.3)
    return s


def parameters(s):
    return {k: s[k] for k in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")}


def check_norm_forward(s, y, h, stats, alpha, rms, eps=1e-5):
    wy, ey, wh, eh, ws = M.norm_residual(M.d(s["x"]), M.d(s["o"]), M.d(s["post_gamma"]), M.d(s["post_beta"]), M.d(s["gate"]),
                                         alpha, M.d(s["pre_gamma"]), M.d(s["pre_beta"]), rms, eps, M.d(y).reshape(s["x"].shape))
    M.held_to("y", y, wy, ey)
    if wh is not None:
        M.held_to("h", h, wh, eh)
    if stats is not None:
        M.held_to("stats", stats, ws, M.F * (ws.abs() + M.d(s["o"]).abs().mean(1, keepdim=True)
                                             + M.d(y).reshape(s["x"].shape).abs().mean(1, keepdim=True)))


def check_norm_backward(out, s, dy, dh, y, o, alpha, rms, eps=1e-5):
    want = M.norm_backward(M.d(dy), M.d(dh), M.d(y), M.values(o), M.d(s["post_gamma"]), M.d(s["post_beta"]), M.d(s["gate"]),
                           alpha, M.d(s["pre_gamma"]), rms, eps)
    for k, (w, e) in want.items():
        if k in ("dpost_beta", "dpre_beta") and s[k[1:]] is None:
            assert k not in out
            continue
        M.held_to(k, out[k], w, e)


@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("rows,n,gates,post,pre", NORMS)
def test_norm_residual(ptb_lib, rows, n, gates, post, pre, rms):
    s = norm_inputs(rows, n, gates, post, pre, rms, seed=rows + n)
    alpha = 0.75
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], alpha=alpha, rms=bool(rms), **parameters(s))
    check_norm_forward(s, y, h, stats, alpha, rms)
    y2, h2 = ptb_lib.norm_residual(s["x"], s["o"], alpha=alpha, rms=bool(rms), **parameters(s))
    assert torch.equal(y, y2) and (h is None) == (not pre) and (h is None or torch.equal(h, h2))
    dy = normal(rows, n, seed=91, std=0.1)
    dh = normal(rows, n, seed=92, std=0.1) if pre else None
    out = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, alpha=alpha, rms=bool(rms), **parameters(s))
    check_norm_backward(out, s, dy, dh, y, s["o"], alpha, rms)
    again = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, alpha=alpha, rms=bool(rms), **parameters(s))
    assert set(out) == set(again) and all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("rows,n", [(1, 32), (50, 96), (333, 5120), (7, 12288), (4, 32768)])
def test_norm_backward_from_a_checkpoint(ptb_lib, rows, n, rms):
    s = norm_inputs(rows, n, 1, 1, 1, rms, seed=n)
    kept = ptb_lib.checkpoint_pack(s["o"])
    value = ptb_lib.checkpoint_unpack(*kept)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], value, rms=bool(rms), **parameters(s))
    dy, dh = normal(rows, n, seed=1), normal(rows, n, seed=2)
    out = ptb_lib.norm_residual_backward(dy, dh, y, kept, stats, rms=bool(rms), **parameters(s))
    check_norm_backward(out, s, dy, dh, y, kept, 1.0, rms)
    same = ptb_lib.norm_residual_backward(dy, dh, y, value, stats, rms=bool(rms), **parameters(s))
    assert all(torch.equal(out[k], same[k]) for k in out)


def test_norm_backward_from_a_checkpoint_of_any_magnitude(ptb_lib):
    # scales from 2^-126 to beyond 2^104, without a norm that would take them away
    rows, n = 40, 320
    o = normal(rows, n, seed=1) * torch.exp2(torch.linspace(-130, 118, rows)).unsqueeze(1).cuda()
    o = o.to(torch.bfloat16)
    kept = ptb_lib.checkpoint_pack(o)
    value = ptb_lib.checkpoint_unpack(*kept)
    gate = normal(rows, n, seed=2)
    dy = normal(rows, n, seed=3)
    stats = torch.zeros(rows, 4, device="cuda")
    for rms in (False, True):
        out = ptb_lib.norm_residual_backward(dy, None, None, kept, stats, gate=gate, rms=rms)
        M.held_to("dgate", out["dgate"], M.d(dy) * M.values(kept), M.F * (M.d(dy) * M.values(kept)).abs())
        same = ptb_lib.norm_residual_backward(dy, None, None, value, stats, gate=gate, rms=rms)
        assert all(torch.equal(out[k], same[k]) for k in out)


def test_norm_backward_without_a_norm_ignores_its_statistics(ptb_lib):
    s = norm_inputs(9, 256, 1, 1, 0, 0, seed=11)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    dy = normal(9, 256, seed=12)
    want = ptb_lib.norm_residual_backward(dy, None, y, s["o"], stats, **parameters(s))
    stats[:, 2:] = math.nan
    got = ptb_lib.norm_residual_backward(dy, None, y, s["o"], stats, **parameters(s))
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("n,rms", [(14400, False), (20480, False), (26000, False), (26000, True), (13312, True)])
def test_norm_backward_of_a_cluster_captured_first(ptb_lib, n, rms):
    # sizes that no other test calls: the launch's own set-up happens under capture
    s = norm_inputs(64, n, 2, 1, 1, rms, seed=n)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], rms=rms, **parameters(s))
    dy, dh = normal(64, n, seed=1), normal(64, n, seed=2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, rms=rms, **parameters(s))
    g.replay()
    torch.cuda.synchronize()
    check_norm_backward(out, s, dy, dh, y, s["o"], 1.0, rms)


@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("rows,n", [(701, 4104), (700, 5128), (701, 6144), (701, 6152), (702, 8200), (533, 12296),
                                    (401, 16392), (300, 20488), (250, 24584), (200, 28680)])
def test_norm_backward_of_many_wide_rows(ptb_lib, rows, n, rms):
    # every way of cutting a row, each block with several rounds and gates that end inside its run
    gates = 1 if rows % 2 else 2
    s = norm_inputs(rows, n, gates, 1, 1, rms, seed=n)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], rms=bool(rms), **parameters(s))
    dy, dh = normal(rows, n, seed=1), normal(rows, n, seed=2)
    out = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, rms=bool(rms), **parameters(s))
    check_norm_backward(out, s, dy, dh, y, s["o"], 1.0, rms)
    again = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, rms=bool(rms), **parameters(s))
    assert all(torch.equal(out[k], again[k]) for k in out)


def test_norm_without_the_streams_gradient(ptb_lib):
    s = norm_inputs(20, 256, 1, 1, 1, 0, seed=3)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    dh = normal(20, 256, seed=4)
    out = ptb_lib.norm_residual_backward(None, dh, y, s["o"], stats, **parameters(s))
    check_norm_backward(out, s, None, dh, y, s["o"], 1.0, 0)


@pytest.mark.parametrize("n", [192, 2048, 12288])
def test_norm_strides_and_in_place(ptb_lib, n):
    rows = 11
    s = norm_inputs(rows, n, 1, 1, 1, 0, seed=5)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    x2, bx = padded(s["x"], n + 24, 8)
    o2, bo = padded(s["o"], n + 40, 16)
    y2, h2, st2 = ptb_lib.norm_residual_train(x2, o2, y=x2, h=o2, **parameters(s))
    assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(st2, stats)
    assert torch.isnan(bx[:, :8]).all() and torch.isnan(bx[:, n + 8:]).all()
    assert torch.isnan(bo[:, :16]).all() and torch.isnan(bo[:, n + 16:]).all()
    dy, dh = normal(rows, n, seed=6), normal(rows, n, seed=7)
    want = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, **parameters(s))
    dy2, b1 = padded(dy, n + 8, 8)
    dh2, b2 = padded(dh, n + 16, 8)
    yy, _ = padded(y, n + 32, 16)
    oo, _ = padded(s["o"], n + 48, 8)
    grads = dict(want, dx=dy2, do=dh2)
    grads = {k: v if k in ("dx", "do") else torch.full_like(v, math.nan) for k, v in grads.items()}
    got = ptb_lib.norm_residual_backward(dy2, dh2, yy, oo, stats, grads=grads, **parameters(s))
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert torch.isnan(b1[:, :8]).all() and torch.isnan(b2[:, :8]).all() and torch.isnan(b2[:, n + 8:]).all()


@pytest.mark.parametrize("n", [192, 12288])
def test_norm_of_one_row_uses_no_stride(ptb_lib, n):
    lib = ptb_lib.load()
    s = norm_inputs(1, n, 1, 1, 1, 0, seed=5)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    dy, dh = normal(1, n, seed=6), normal(1, n, seed=7)
    want = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, **parameters(s))
    p = {k: s[k].data_ptr() for k in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")}
    x2, o2 = s["x"].clone(), s["o"].clone()
    assert lib.ptb_norm_residual(x2.data_ptr(), 0, o2.data_ptr(), 8, p["post_gamma"], p["post_beta"], p["gate"], 1, 1.0,
                                 p["pre_gamma"], p["pre_beta"], 0, 1e-5, 1, n, x2.data_ptr(), 1 << 40, o2.data_ptr(), 16,
                                 None, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(o2, h)
    ws = torch.empty(ptb_lib.norm_residual_backward_workspace_size(1, n), dtype=torch.uint8, device="cuda")
    got = {k: v.clone() for k, v in want.items() if k not in ("dx", "do")}
    o2 = s["o"].clone()
    assert lib.ptb_norm_residual_backward(dy.data_ptr(), 0, dh.data_ptr(), 8, y.data_ptr(), 0, o2.data_ptr(), 16, None, 0,
                                          stats.data_ptr(), p["post_gamma"], p["post_beta"], p["gate"], 1, 1.0,
                                          p["pre_gamma"], 0, 1, n, dy.data_ptr(), 1 << 40, o2.data_ptr(), 24,
                                          got["dpost_gamma"].data_ptr(), got["dpost_beta"].data_ptr(),
                                          got["dgate"].data_ptr(), got["dpre_gamma"].data_ptr(),
                                          got["dpre_beta"].data_ptr(), ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    got.update(dx=dy, do=o2)
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("post,pre", [(1, 1), (1, 0), (0, 1)])
@pytest.mark.parametrize("rows,n,gates", [(4, 64, 2), (300, 320, 3), (12, 12288, 12), (700, 5120, 700)])
def test_norm_without_a_gate_uses_no_count_of_gates(ptb_lib, rows, n, gates, post, pre, rms):
    """A caller may pass its number of sequences whether there is a gate or not."""
    lib = ptb_lib.load()
    s = norm_inputs(rows, n, 0, post, pre, rms, seed=rows)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], rms=bool(rms), **parameters(s))
    dy, dh = normal(rows, n, seed=1), normal(rows, n, seed=2) if pre else None
    want = ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, rms=bool(rms), **parameters(s))
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    y2, h2 = torch.empty_like(y), torch.empty_like(y) if pre else None
    assert lib.ptb_norm_residual(p(s["x"]), n, p(s["o"]), n, p(s["post_gamma"]), p(s["post_beta"]), None, gates, 1.0,
                                 p(s["pre_gamma"]), p(s["pre_beta"]), rms, 1e-5, rows, n, p(y2), n, p(h2), n, None, None) == 0
    ws = torch.empty(ptb_lib.norm_residual_backward_workspace_size(rows, n, gates), dtype=torch.uint8, device="cuda")
    got = {k: torch.full_like(v, math.nan) for k, v in want.items()}
    g = lambda k: p(got.get(k))  # noqa: E731
    assert lib.ptb_norm_residual_backward(p(dy), n, p(dh), n, p(y), n, p(s["o"]), n, None, 0, p(stats), p(s["post_gamma"]),
                                          p(s["post_beta"]), None, gates, 1.0, p(s["pre_gamma"]), rms, rows, n, g("dx"), n,
                                          g("do"), n, g("dpost_gamma"), g("dpost_beta"), None, g("dpre_gamma"),
                                          g("dpre_beta"), p(ws), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and (h is None or torch.equal(h2, h))
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("ld", [3, -8, 1 << 40])
@pytest.mark.parametrize("n", [192, 12288])
def test_one_row_of_any_stride(ptb_lib, n, ld):
    """A single row's stride need not be one that several rows could have."""
    lib = ptb_lib.load()
    s = norm_inputs(1, n, 1, 1, 1, 0, seed=6)
    p = lambda t: t.data_ptr()  # noqa: E731
    w = [p(s[k]) for k in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")]
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    got = [torch.full_like(t, math.nan) for t in (y, h, stats)]
    assert lib.ptb_norm_residual(p(s["x"]), ld, p(s["o"]), ld, *w[:3], 1, 1.0, *w[3:], 0, 1e-5, 1, n, p(got[0]), ld,
                                 p(got[1]), ld, p(got[2]), None) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, h, stats)))
    kept = ptb_lib.checkpoint_pack(s["o"])
    codes, exps, back = torch.zeros_like(kept[0]), torch.zeros_like(kept[1]), torch.empty_like(y)
    assert lib.ptb_checkpoint_pack(p(s["o"]), ld, 1, n, p(codes), ld, p(exps), ld, None) == 0
    assert lib.ptb_checkpoint_unpack(p(codes), ld, p(exps), ld, 1, n, p(back), ld, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(codes, kept[0]) and torch.equal(exps, kept[1])
    assert torch.equal(back, ptb_lib.checkpoint_unpack(*kept))
    dy, dh = normal(1, n, seed=1), normal(1, n, seed=2)
    ws = torch.empty(ptb_lib.norm_residual_backward_workspace_size(1, n), dtype=torch.uint8, device="cuda")
    for o, oe in ((s["o"], None), kept):
        want = ptb_lib.norm_residual_backward(dy, dh, y, o if oe is None else kept, stats, **parameters(s))
        out = {k: torch.full_like(v, math.nan) for k, v in want.items()}
        assert lib.ptb_norm_residual_backward(
            p(dy), ld, p(dh), ld, p(y), ld, p(o), ld, None if oe is None else p(oe), ld, p(stats), *w[:3], 1, 1.0, w[3], 0, 1,
            n, p(out["dx"]), ld, p(out["do"]), ld, p(out["dpost_gamma"]), p(out["dpost_beta"]), p(out["dgate"]),
            p(out["dpre_gamma"]), p(out["dpre_beta"]), p(ws), ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)


@pytest.mark.parametrize("ld", [3, -8])
@pytest.mark.parametrize("h,f", [(128, 192), (2048, 512)])
def test_gated_ffn_of_one_token_of_any_stride(ptb_lib, h, f, ld):
    lib = ptb_lib.load()
    s = ffn_inputs(1, h, f, seed=9)
    y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), residual=s["resid"])
    plain = ptb_lib.gated_ffn(s["x"], *weights(s), residual=s["resid"])
    x8 = ptb_lib.checkpoint_pack(s["x"])
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    wp = [p(t) for t in weights(s)]
    ws = torch.empty(max(ptb_lib.gated_ffn_workspace_size(1, h, f), ptb_lib.gated_ffn_backward_workspace_size(1, h, f, 8)),
                     dtype=torch.uint8, device="cuda")
    for k, want in ((None, plain), (torch.empty_like(kept), y)):
        got = torch.empty_like(y)
        assert lib.ptb_gated_ffn(p(s["x"]), ld, *wp, p(s["resid"]), ld, 1, h, f, 0, p(got), ld, p(k), None, p(ws), ws.numel(),
                                 None) == 0
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (k is None or torch.equal(k, kept))
    for x, xe in ((s["x"], None), x8):
        want = ptb_lib.gated_ffn_backward(s["dy"], x if xe is None else x8, *weights(s), kept)
        got = {k: torch.empty_like(v) for k, v in want.items()}
        assert lib.ptb_gated_ffn_backward(p(s["dy"]), ld, p(x), ld, p(xe), ld, *wp, p(kept), None, 1, h, f, 0, p(got["dx"]), ld,
                                          p(got["dw_gate"]), p(got["dw_up"]), p(got["dw_down"]), 16, p(ws), ws.numel(),
                                          None) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_norm_rows_of_nan_stay_their_own(ptb_lib):
    s = norm_inputs(40, 512, 1, 1, 1, 0, seed=8)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    bad = s["o"].clone()
    bad[7, 100] = math.inf
    bad[8, 0] = math.nan
    y2, h2, st2 = ptb_lib.norm_residual_train(s["x"], bad, **parameters(s))
    rest = [r for r in range(40) if r not in (7, 8)]
    assert torch.equal(y2[rest], y[rest]) and torch.equal(h2[rest], h[rest])
    assert torch.isnan(h2[7]).any() and torch.isnan(h2[8]).all()


def test_norm_of_constant_rows_and_no_rows(ptb_lib):
    s = norm_inputs(4, 512, 0, 1, 1, 0, seed=9)
    s["x"] = torch.zeros_like(s["x"])
    s["o"] = torch.full_like(s["o"], 3.0)
    s["post_beta"] = None
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    assert (y == 0).all() and torch.equal(h, s["pre_beta"].expand(4, -1))
    none = torch.zeros(0, 512, dtype=torch.bfloat16, device="cuda")
    y, h, stats = ptb_lib.norm_residual_train(none, none, **parameters(s))
    assert y.shape == (0, 512) and stats.shape == (0, 4)
    out = ptb_lib.norm_residual_backward(none, none, none, none, stats, **parameters(s))
    assert (out["dpost_gamma"] == 0).all() and (out["dpre_beta"] == 0).all() and out["dx"].shape == (0, 512)


def test_norm_binding_refusals(ptb_lib):
    s = norm_inputs(4, 64, 0, 1, 1, 0, seed=1)
    x, o = s["x"], s["o"]
    for kw in (dict(gate=normal(3, 64, seed=1)), dict(gate=normal(32, seed=1)), dict(post_gamma=normal(32, seed=1)),
               dict(post_gamma=normal(2, 64, seed=1)[:, ::1][0:1])):
        with pytest.raises(ValueError):
            ptb_lib.norm_residual(x, o, **kw)
    with pytest.raises(ValueError):
        ptb_lib.norm_residual(x, o[:2])
    with pytest.raises(TypeError):
        ptb_lib.norm_residual(x, o.float())
    with pytest.raises(ValueError):
        ptb_lib.norm_residual(x, o.t().contiguous().t())
    with pytest.raises(ptb_lib.PTBError):
        ptb_lib.norm_residual(x, o, post_gamma=s["post_gamma"], post_beta=s["post_beta"], rms=True)


# --------------------------------------------------------------- gated feed-forward --

FFNS = [
    # tokens, hidden, ffn
    (1, 64, 64), (2, 64, 128), (3, 128, 64), (1, 1024, 2752), (7, 192, 320), (8, 256, 512), (9, 64, 192), (16, 512, 192),
    (17, 320, 128), (33, 256, 448), (64, 128, 1024), (127, 128, 192), (128, 256, 256), (129, 256, 320), (130, 192, 384),
    (200, 1088, 256), (257, 512, 640), (300, 64, 1088), (513, 256, 256), (24, 1024, 1024),
    # the border between the kernels of few tokens and the others, and wide outputs of few tokens
    (31, 192, 256), (32, 256, 192), (20, 5120, 64), (11, 4928, 128), (32, 4864, 64),
    # N tiles that reach past the width, K split over the SMs
    (260, 1088, 832), (140, 2112, 704), (700, 576, 1344),
]


def ffn_inputs(t, h, f, seed=0):
    return dict(x=normal(t, h, seed=seed), wg=normal(f, h, seed=seed + 1, std=1.2 / math.sqrt(h)),
                wu=normal(f, h, seed=seed + 2, std=1.2 / math.sqrt(h)), wd=normal(h, f, seed=seed + 3, std=1 / math.sqrt(f)),
                dy=normal(t, h, seed=seed + 4, std=0.1), resid=normal(t, h, seed=seed + 5, std=2))


def weights(s):
    return s["wg"], s["wu"], s["wd"]


def model_weights(s):
    return M.d(s["wg"]), M.d(s["wu"]), M.d(s["wd"])


def check_ffn(s, act, y, kept=None, resid=None):
    g, eg, u, eu, wy, ey = M.ffn(M.d(s["x"]), *model_weights(s), act, M.d(resid))
    M.held_to("y", y, wy, ey)
    if kept is not None:
        both, err = torch.cat([g, u], 1), torch.cat([eg, eu], 1)
        bound = M.kept_bound(both, err, kept)
        over = (M.values(kept) - both).abs() - bound
        assert (over <= 0).all(), f"kept: {int((over > 0).sum())} beyond the bound, by up to {over.max():.3e}"


def check_ffn_backward(out, s, act, x, kept, rounding=M.U16):
    f = s["wg"].shape[0]
    v = M.values(kept)
    want = M.ffn_backward(M.d(s["dy"]), M.values(x), *model_weights(s), v[:, :f], v[:, f:], act, rounding)
    for k, (w, e) in want.items():
        M.held_to(k, out[k], w, e)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("t,h,f", FFNS)
def test_gated_ffn(ptb_lib, t, h, f, pairs, act):
    s = ffn_inputs(t, h, f, seed=t + h + f)
    was = ptb_lib.set_gemm_pairs(pairs)
    try:
        y = ptb_lib.gated_ffn(s["x"], *weights(s), activation=act)
        check_ffn(s, act, y)
        y = ptb_lib.gated_ffn(s["x"], *weights(s), activation=act, residual=s["resid"])
        check_ffn(s, act, y, resid=s["resid"])
        for bits in (16, 8):
            y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), activation=act, bits=bits)
            check_ffn(s, act, y, kept)
            x = s["x"] if bits == 16 else ptb_lib.checkpoint_pack(s["x"])
            out = ptb_lib.gated_ffn_backward(s["dy"], x, *weights(s), kept, activation=act)
            check_ffn_backward(out, s, act, x, kept)
    finally:
        ptb_lib.set_gemm_pairs(was)


# Every tile (256 wide on pairs of CTAs, 256, 128 and 64 on one), whole and in pieces of K, that a
# GEMM of the call can be given.
TILES = [
    (32, 576, 1088), (129, 4928, 64), (37, 3712, 4928), (32, 64, 9984), (2959, 1088, 192), (644, 4864, 64),
    (131, 5056, 3456), (551, 3968, 2240), (35, 5056, 10048), (259, 64, 9984), (2765, 192, 10816), (4040, 192, 2560),
    (133, 2240, 11008), (129, 4928, 6976), (158, 5888, 6528), (777, 2048, 5440),
]

# Long and narrow: one tile of a weight gradient in dozens of pieces, rows of one tile's columns.
LONG = [(100003, 64, 64), (20000, 128, 64), (3, 64, 39936), (65, 10240, 128)]

# Few tokens and so many weights that the kernels of few tokens end at 16.
MANY_WEIGHTS = [(16, 4160, 9664), (17, 4160, 9664), (32, 9664, 4160)]


@pytest.mark.parametrize("t,h,f", TILES)
def test_gated_ffn_of_every_tile(ptb_lib, t, h, f):
    s = ffn_inputs(t, h, f, seed=t + h + f)
    act, bits = ("silu", 16) if t % 2 else ("gelu", 8)
    y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), activation=act, bits=bits, residual=s["resid"])
    check_ffn(s, act, y, kept, resid=s["resid"])
    x = s["x"] if bits == 16 else ptb_lib.checkpoint_pack(s["x"])
    out = ptb_lib.gated_ffn_backward(s["dy"], x, *weights(s), kept, activation=act)
    check_ffn_backward(out, s, act, x, kept)
    again = ptb_lib.gated_ffn_backward(s["dy"], x, *weights(s), kept, activation=act)
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("t,h,f", LONG)
def test_gated_ffn_long_and_narrow(ptb_lib, t, h, f):
    s = ffn_inputs(t, h, f, seed=t)
    check_ffn(s, "silu", ptb_lib.gated_ffn(s["x"], *weights(s)))
    y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), bits=8)
    check_ffn(s, "silu", y, kept)
    out = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept)
    check_ffn_backward(out, s, "silu", s["x"], kept)
    again = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept)
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("t,h,f", [(777, 2048, 5440), (131, 5056, 3456)])
def test_gated_ffn_without_pairs(ptb_lib, t, h, f):
    # the workspace of a size serves either way, and a call after the switch
    s = ffn_inputs(t, h, f, seed=3)
    ws = torch.empty(max(ptb_lib.gated_ffn_workspace_size(t, h, f), ptb_lib.gated_ffn_backward_workspace_size(t, h, f)),
                     dtype=torch.uint8, device="cuda")
    was = ptb_lib.set_gemm_pairs(0)
    try:
        y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), workspace=ws)
        check_ffn(s, "silu", y, kept)
        ptb_lib.set_gemm_pairs(1)
        out = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept, workspace=ws)
        check_ffn_backward(out, s, "silu", s["x"], kept)
        ptb_lib.set_gemm_pairs(0)
        out = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept, workspace=ws)
        check_ffn_backward(out, s, "silu", s["x"], kept)
    finally:
        ptb_lib.set_gemm_pairs(was)


@pytest.mark.parametrize("t,h,f", MANY_WEIGHTS)
def test_gated_ffn_of_few_tokens_and_many_weights(ptb_lib, t, h, f):
    s = ffn_inputs(t, h, f, seed=t)
    check_ffn(s, "silu", ptb_lib.gated_ffn(s["x"], *weights(s)))
    check_ffn(s, "silu", ptb_lib.gated_ffn(s["x"], *weights(s), residual=s["resid"]), resid=s["resid"])


@pytest.mark.parametrize("t,h,f", [(2959, 1088, 192), (4040, 192, 2560), (2765, 192, 10816), (777, 2048, 5440)])
def test_gated_ffn_fp32_gradients_of_every_tile(ptb_lib, t, h, f):
    s = ffn_inputs(t, h, f, seed=2)
    _, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s))
    out = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept, grad_dtype=torch.float32)
    check_ffn_backward(out, s, "silu", s["x"], kept, M.U32)


@pytest.mark.parametrize("t,h,f", [(5, 128, 192), (260, 256, 384), (40, 1024, 256)])
def test_gated_ffn_fp32_gradients(ptb_lib, t, h, f):
    s = ffn_inputs(t, h, f, seed=1)
    _, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s))
    out = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept, grad_dtype=torch.float32)
    assert out["dw_up"].dtype == torch.float32
    check_ffn_backward(out, s, "silu", s["x"], kept, M.U32)
    again = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept, grad_dtype=torch.float32)
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("ld", [0, 8, 1 << 40])
@pytest.mark.parametrize("h,f", [(128, 192), (2048, 512)])
def test_gated_ffn_of_one_token_uses_no_stride(ptb_lib, h, f, ld):
    lib = ptb_lib.load()
    s = ffn_inputs(1, h, f, seed=9)
    y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), residual=s["resid"])
    plain = ptb_lib.gated_ffn(s["x"], *weights(s), residual=s["resid"])
    want = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept)
    ptr = {k: v.data_ptr() for k, v in s.items()}
    wp = ptr["wg"], ptr["wu"], ptr["wd"]
    ws = torch.empty(max(ptb_lib.gated_ffn_workspace_size(1, h, f), ptb_lib.gated_ffn_backward_workspace_size(1, h, f)),
                     dtype=torch.uint8, device="cuda")
    for k, w in ((None, plain), (torch.empty_like(kept), y)):
        got = torch.empty_like(y)
        assert lib.ptb_gated_ffn(ptr["x"], ld, *wp, ptr["resid"], ld, 1, h, f, 0, got.data_ptr(), ld,
                                 None if k is None else k.data_ptr(), None, ws.data_ptr(), ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(got, w) and (k is None or torch.equal(k, kept))
    got = {k: torch.empty_like(v) for k, v in want.items()}
    assert lib.ptb_gated_ffn_backward(ptr["dy"], ld, ptr["x"], ld, None, 0, *wp, kept.data_ptr(), None, 1, h, f, 0,
                                      got["dx"].data_ptr(), ld, got["dw_gate"].data_ptr(), got["dw_up"].data_ptr(),
                                      got["dw_down"].data_ptr(), 16, ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("t", [4, 150, 300])
def test_gated_ffn_strides_and_in_place(ptb_lib, t):
    h, f = 192, 256
    s = ffn_inputs(t, h, f, seed=2)
    y = ptb_lib.gated_ffn(s["x"], *weights(s), residual=s["resid"])
    x2, bx = padded(s["x"], h + 24, 8)
    r2, br = padded(s["resid"], h + 16, 8)
    assert torch.equal(ptb_lib.gated_ffn(x2, *weights(s), residual=r2, y=r2), y)
    assert torch.isnan(br[:, :8]).all() and torch.isnan(br[:, h + 8:]).all()
    assert torch.equal(ptb_lib.gated_ffn(x2, *weights(s), residual=s["resid"], y=x2), y)
    assert torch.isnan(bx[:, :8]).all() and torch.isnan(bx[:, h + 8:]).all()
    _, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), bits=8)
    want = ptb_lib.gated_ffn_backward(s["dy"], s["x"], *weights(s), kept)
    dy2, bd = padded(s["dy"], h + 8, 8)
    x3, _ = padded(s["x"], h + 40, 16)
    grads = {k: torch.full_like(v, math.nan) for k, v in want.items()}
    grads["dx"] = dy2
    got = ptb_lib.gated_ffn_backward(dy2, x3, *weights(s), kept, grads=grads)
    assert all(torch.equal(got[k], want[k]) for k in want) and torch.isnan(bd[:, :8]).all()


def test_gated_ffn_shapes(ptb_lib):
    s = ffn_inputs(6, 64, 128, seed=3)
    y = ptb_lib.gated_ffn(s["x"], *weights(s))
    y3 = ptb_lib.gated_ffn(s["x"].view(2, 3, 64), *weights(s))
    assert y3.shape == (2, 3, 64) and torch.equal(y3.view(6, 64), y)
    none = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    for bits in (16, 8):
        y, kept = ptb_lib.gated_ffn_train(none, *weights(s), bits=bits)
        out = ptb_lib.gated_ffn_backward(none, none, *weights(s), kept)
        assert y.shape == (0, 64) and all((out[k] == 0).all() for k in ("dw_gate", "dw_up", "dw_down"))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_extreme_gates(ptb_lib, act):
    """Gates far out on both sides: act and its derivative reach their limits without NaN."""
    h = f = 64
    x = torch.zeros(4, h, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([1.0, -1.0, 30.0, -30.0])
    wg = torch.zeros(f, h, dtype=torch.bfloat16, device="cuda")
    wg[:, 0] = torch.linspace(-2000, 2000, f)
    s = dict(x=x, wg=wg, wu=normal(f, h, seed=1), wd=normal(h, f, seed=2, std=0.1), dy=normal(4, h, seed=3))
    for bits in (16, 8):
        y, kept = ptb_lib.gated_ffn_train(x, *weights(s), activation=act, bits=bits)
        check_ffn(s, act, y, kept)
        out = ptb_lib.gated_ffn_backward(s["dy"], x, *weights(s), kept, activation=act)
        check_ffn_backward(out, s, act, x, kept)


def test_gated_ffn_rows_of_nan_stay_their_own(ptb_lib):
    s = ffn_inputs(140, 128, 192, seed=6)
    y, kept = ptb_lib.gated_ffn_train(s["x"], *weights(s), bits=8)
    bad = s["x"].clone()
    bad[3, 5] = math.nan
    bad[130, 0] = math.inf
    y2, kept2 = ptb_lib.gated_ffn_train(bad, *weights(s), bits=8)
    rest = [r for r in range(140) if r not in (3, 130)]
    assert torch.equal(y2[rest], y[rest]) and torch.equal(kept2[0][rest], kept[0][rest])
    assert torch.isnan(y2[3]).all() and (kept2[1][3] == 255).all()


def test_gated_ffn_binding_refusals(ptb_lib):
    s = ffn_inputs(4, 64, 128, seed=1)
    x, w = s["x"], weights(s)
    with pytest.raises(ValueError):  # rows at two strides
        ptb_lib.gated_ffn(normal(4, 6, 64, seed=1)[:, :3], *w)
    with pytest.raises(ptb_lib.PTBError):  # rows on top of each other
        ptb_lib.gated_ffn(x[:1].expand(3, 64), *w)
    with pytest.raises(ValueError):
        ptb_lib.gated_ffn(x, *w, activation="relu")
    with pytest.raises(ValueError):
        ptb_lib.gated_ffn(x, w[0], w[1][:64], w[2])
    with pytest.raises(ValueError):
        ptb_lib.gated_ffn(x, w[0].t().contiguous().t(), w[1], w[2])
    with pytest.raises(ValueError):
        ptb_lib.gated_ffn(x, *w, residual=x[:2])
    with pytest.raises(TypeError):
        ptb_lib.gated_ffn(x.float(), *w)
    _, kept = ptb_lib.gated_ffn_train(x, *w)
    with pytest.raises(ValueError):
        ptb_lib.gated_ffn_backward(x, x, *w, kept[:, :128].contiguous())
    with pytest.raises(TypeError):
        ptb_lib.gated_ffn_backward(x, x, *w, kept.float())
    with pytest.raises(ptb_lib.PTBError):
        ptb_lib.gated_ffn(normal(4, 96, seed=1), normal(128, 96, seed=1), normal(128, 96, seed=2), normal(96, 128, seed=3))
    with pytest.raises(ptb_lib.PTBError):
        ptb_lib.gated_ffn(x, *w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------- a block, as it is used --

def block_inputs(rows, h, f, seqs):
    s = norm_inputs(rows, h, seqs, 1, 1, 0, seed=20)
    s.update({k: v for k, v in ffn_inputs(rows, h, f, seed=30).items() if k.startswith("w")})
    s["first"] = normal(h, seed=40, std=0.2, mean=1)
    s["dy"], s["dh"] = normal(rows, h, seed=41, std=0.1), normal(rows, h, seed=42, std=0.1)
    return s


def block_step(lib, s, stream=None):
    """Norm, gated feed-forward, norm with gate and residual, and back, activations in 8 bits."""
    x0 = s["x"]
    zero = torch.zeros_like(x0)
    y0, h0, st0 = lib.norm_residual_train(x0, zero, pre_gamma=s["first"], rms=True, stream=stream)
    o, kept = lib.gated_ffn_train(h0, *weights(s), bits=8, stream=stream)
    h8, o8 = lib.checkpoint_pack(h0, stream=stream), lib.checkpoint_pack(o, stream=stream)
    ov = lib.checkpoint_unpack(*o8, stream=stream)
    y1, h1, st1 = lib.norm_residual_train(y0, ov, stream=stream, **parameters(s))
    b1 = lib.norm_residual_backward(s["dy"], s["dh"], y1, o8, st1, stream=stream, **parameters(s))
    fb = lib.gated_ffn_backward(b1["do"], h8, *weights(s), kept, stream=stream)
    b0 = lib.norm_residual_backward(b1["dx"], fb["dx"], y0, zero, st0, pre_gamma=s["first"], rms=True, stream=stream)
    return dict(y=y1, h=h1, dx=b0["dx"], dfirst=b0["dpre_gamma"], kept=kept, h0=h0, h8=h8, o8=o8, y0=y0, o=o, st1=st1,
                b1=b1, fb=fb)


def test_block_step(ptb_lib):
    s = block_inputs(264, 256, 448, 4)
    r = block_step(ptb_lib, s)
    f = dict(s, x=r["h0"])
    check_ffn(f, "silu", r["o"], r["kept"])
    v = dict(s, x=r["y0"], o=ptb_lib.checkpoint_unpack(*r["o8"]))
    check_norm_forward(v, r["y"], r["h"], r["st1"], 1.0, 0)
    check_norm_backward(r["b1"], v, s["dy"], s["dh"], r["y"], r["o8"], 1.0, 0)
    check_ffn_backward(r["fb"], dict(s, dy=r["b1"]["do"]), "silu", r["h8"], r["kept"])
    # the whole step, against torch's gradients of the block in 64 bits on the unrounded function
    leaves = {k: M.d(s[k]).requires_grad_() for k in ("x", "first", "wg", "wu", "wd", "post_gamma", "post_beta", "gate",
                                                      "pre_gamma", "pre_beta")}
    rms = leaves["x"] * (leaves["x"].square().mean(1, keepdim=True) + 1e-5).rsqrt() * leaves["first"]
    o = (torch.nn.functional.silu(rms @ leaves["wg"].t()) * (rms @ leaves["wu"].t())) @ leaves["wd"].t()
    ln = lambda t, g, b: torch.nn.functional.layer_norm(t, (256,), g, b, 1e-5)  # noqa: E731
    p = ln(o, leaves["post_gamma"], leaves["post_beta"])
    y = leaves["x"] + leaves["gate"].repeat_interleave(66, 0) * p
    h = ln(y, leaves["pre_gamma"], leaves["pre_beta"])
    ((y * M.d(s["dy"])).sum() + (h * M.d(s["dh"])).sum()).backward()
    # Uniform codes of 32 values of a normal group are off by a step / sqrt(12), a step of at most
    # m / 63.75 with m about 2.1 (at most 3) of the group's deviation: 0.014 relative.  Two of them
    # (gate and up) meet in each product, o's and x's add one each, and bf16's add 2^-8 / sqrt(3)
    # five times: 0.03 in all; half as much again for the derivatives' slopes.
    got = dict(x=r["dx"], first=r["dfirst"], wg=r["fb"]["dw_gate"], wu=r["fb"]["dw_up"], wd=r["fb"]["dw_down"],
               **{k: r["b1"]["d" + k] for k in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")})
    for k, t in got.items():
        want = leaves[k].grad
        rel = ((M.d(t).reshape(want.shape) - want).norm() / want.norm()).item()
        assert rel < 0.045, f"{k}: {rel:.4f}"


def flat(r):
    for v in r.values():
        if isinstance(v, dict):
            yield from flat(v)
        elif isinstance(v, tuple):
            yield from v
        else:
            yield v


def test_block_step_on_a_stream_and_in_two_graphs(ptb_lib):
    one, two = block_inputs(200, 256, 320, 2), block_inputs(70, 1024, 192, 1)
    want = [list(flat(block_step(ptb_lib, s))) for s in (one, two)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = list(flat(block_step(ptb_lib, one, stream=side)))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs, outs = [], []
    for s in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(list(flat(block_step(ptb_lib, s))))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    # other inputs in the same buffers
    fresh = block_inputs(200, 256, 320, 2)
    fresh["x"] = normal(200, 256, seed=77)
    one["x"].copy_(fresh["x"])
    graphs[0].replay()
    want0 = list(flat(block_step(ptb_lib, fresh)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want0))


@pytest.mark.parametrize("t", [8, 192])
def test_weights_that_the_call_in_front_wrote(ptb_lib, t):
    """Kernels start while those in front of them end: none may read before what it reads is there."""
    h = 256
    s = ffn_inputs(h, h, h, seed=8)
    x = normal(t, h, seed=9)
    outs, want = [], []
    for wait in (True, False):
        for k in range(12):
            first = ptb_lib.gated_ffn(s["x"] * (k + 1), *weights(s))  # [h, h]: the next call's weights
            if wait:
                torch.cuda.synchronize()
            second = ptb_lib.gated_ffn(x, first, s["wu"], first)
            if wait:
                torch.cuda.synchronize()
            y, kept = ptb_lib.gated_ffn_train(second, s["wg"], first, first)
            if wait:
                torch.cuda.synchronize()
            g = ptb_lib.gated_ffn_backward(y, second, s["wg"], first, first, kept)
            (want if wait else outs).append([first, second, y, kept] + list(g.values()))
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(u.nan_to_num(), v.nan_to_num()) for u, v in zip(a, b))


def test_two_calls_at_once(ptb_lib):
    """Two streams, each with its own workspace, interleaved."""
    s = [ffn_inputs(180, 256, 512, seed=1), ffn_inputs(33, 512, 256, seed=2)]
    want = [ptb_lib.gated_ffn(v["x"], *weights(v)) for v in s]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for k in (0, 1):
            got[k].append(ptb_lib.gated_ffn(s[k]["x"], *weights(s[k]), stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(v, want[k]) for v in got[k])


@pytest.mark.parametrize("rms,widths", [(0, (1024, 4096)), (1, (2048, 4096)), (0, (8200, 16384))])
def test_norm_backward_of_two_widths_from_two_threads(ptb_lib, rms, widths):
    """Kernels of one kind serve many widths, with as much shared memory as each needs: what one thread asks
    for is not to reach another's launch."""
    lib = ptb_lib.load()
    rows, calls, kept, want, got = 4, 4000, [], [], []
    for n in widths:
        s = norm_inputs(rows, n, 1, 1, 1, rms, seed=n)
        y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], rms=bool(rms), **parameters(s))
        dy, dh = normal(rows, n, seed=1), normal(rows, n, seed=2)
        want.append(ptb_lib.norm_residual_backward(dy, dh, y, s["o"], stats, rms=bool(rms), **parameters(s)))
        got.append({k: torch.full_like(v, math.nan) for k, v in want[-1].items()})
        ws = torch.empty(ptb_lib.norm_residual_backward_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        g = lambda k: p(got[-1].get(k))  # noqa: E731
        kept.append(((dy, dh, y, s, stats, ws, stream), (
            p(dy), n, p(dh), n, p(y), n, p(s["o"]), n, None, 0, p(stats), p(s["post_gamma"]), p(s["post_beta"]),
            p(s["gate"]), 1, 1.0, p(s["pre_gamma"]), rms, rows, n, g("dx"), n, g("do"), n, g("dpost_gamma"),
            g("dpost_beta"), g("dgate"), g("dpre_gamma"), g("dpre_beta"), p(ws), ws.numel(), stream.cuda_stream)))
    torch.cuda.synchronize()
    device, start, failed = torch.cuda.current_device(), threading.Barrier(2), [-1, -1]

    def work(k):
        torch.cuda.set_device(device)
        start.wait()
        failed[k] = sum(lib.ptb_norm_residual_backward(*kept[k][1]) != 0 for _ in range(calls))

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0], f"{failed} of {calls} calls failed"
    for k in (0, 1):
        assert all(torch.equal(got[k][key], want[k][key]) for key in want[k])


@pytest.mark.parametrize("refused", ["few tokens", "many tokens", "norm backward", "checkpoint"])
def test_a_failed_launch_is_not_reported_by_the_next_call(ptb_lib, refused):
    """While a stream that waits for the legacy stream is being captured, work on the legacy stream is an error:
    that call's, and not the next one's."""
    lib, cu = ptb_lib.load(), ctypes.CDLL("libcuda.so.1")
    f, s = ffn_inputs(200, 128, 192, seed=1), norm_inputs(6, 64, 1, 1, 1, 0, seed=2)
    y, h, stats = ptb_lib.norm_residual_train(s["x"], s["o"], **parameters(s))
    x = normal(3, 64, seed=3)
    codes, exps = ptb_lib.checkpoint_pack(x)
    want = [t.clone() for t in (codes, exps)]
    ws = torch.empty(max(ptb_lib.gated_ffn_workspace_size(200, 128, 192),
                         ptb_lib.norm_residual_backward_workspace_size(6, 64)), dtype=torch.uint8, device="cuda")
    out = torch.empty(200, 128, dtype=torch.bfloat16, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    pack = lambda: lib.ptb_checkpoint_pack(p(x), 64, 3, 64, p(codes), 64, p(exps), 2, None)  # noqa: E731
    ffn = lambda t: lib.ptb_gated_ffn(p(f["x"]), 128, p(f["wg"]), p(f["wu"]), p(f["wd"]), None, 0, t, 128, 192, 0,  # noqa: E731
                                      p(out), 128, None, None, p(ws), ws.numel(), None)
    norm = lambda: lib.ptb_norm_residual_backward(  # noqa: E731
        p(s["x"]), 64, p(s["x"]), 64, p(y), 64, p(s["o"]), 64, None, 0, p(stats), p(s["post_gamma"]), p(s["post_beta"]),
        p(s["gate"]), 1, 1.0, p(s["pre_gamma"]), 0, 6, 64, p(out), 64, p(out[100:]), 64, None, None, None, None, None,
        p(ws), ws.numel(), None)
    call = {"few tokens": lambda: ffn(8), "many tokens": lambda: ffn(200), "norm backward": norm, "checkpoint": pack}[refused]
    assert call() == 0
    torch.cuda.synchronize()
    codes.zero_(), exps.zero_()
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert cu.cuStreamBeginCapture_v2(stream, 1) == 0  # of this thread's calls
    st = call()
    cu.cuStreamEndCapture(stream, ctypes.byref(graph))
    if graph:
        cu.cuGraphDestroy(graph)
    assert cu.cuStreamDestroy_v2(stream) == 0
    assert st == 5  # PTB_ERR_LAUNCH
    assert pack() == 0
    torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(exps, want[1])
