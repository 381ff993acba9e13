"""Refusals and sizes of the gated feed-forward, the norms around a block and the checkpoints, on the
host: nothing here touches a device, the pointers are never read."""
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


def ffn(lib, **kw):
    a = dict(x=FAKE, ldx=128, wg=FAKE, wu=FAKE, wd=FAKE, r=None, ldr=0, t=0, h=128, f=192, act=0, y=FAKE * 2, ldy=128,
             kept=None, exps=None, ws=FAKE * 8, wsb=1 << 40)
    a.update(kw)
    return lib.ptb_gated_ffn(a["x"], a["ldx"], a["wg"], a["wu"], a["wd"], a["r"], a["ldr"], a["t"], a["h"], a["f"], a["act"],
                             a["y"], a["ldy"], a["kept"], a["exps"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(wg=None), ARG), (dict(wu=None), ARG), (dict(wd=None), ARG), (dict(t=-1), ARG), (dict(act=2), ARG),
    (dict(act=-1), ARG), (dict(exps=FAKE), ARG), (dict(x=None, t=1), ARG), (dict(y=None, t=1), ARG),
    (dict(t=2, ldx=120), ARG), (dict(t=2, ldy=64), ARG), (dict(t=2, r=FAKE, ldr=64), ARG),
    (dict(t=2, r=FAKE * 2, ldr=256), ARG), (dict(t=1, ws=None), ARG), (dict(h=0), ARG), (dict(f=0), ARG),
    (dict(h=96), SHAPE), (dict(f=100), SHAPE), (dict(t=1 << 40), SHAPE), (dict(f=1 << 30), SHAPE),
    (dict(wg=FAKE + 8), ALIGN), (dict(t=1, x=FAKE + 2), ALIGN), (dict(t=2, ldx=132), ALIGN), (dict(kept=FAKE + 8), ALIGN),
    (dict(t=1, ws=FAKE * 8 + 16), ALIGN), (dict(t=1, wsb=100), WORKSPACE),
])
def test_gated_ffn_refuses(lib, kw, code):
    assert ffn(lib, **kw) == code


def ffn_bwd(lib, **kw):
    a = dict(dy=FAKE, lddy=128, x=FAKE, ldx=128, xe=None, ldxe=0, wg=FAKE, wu=FAKE, wd=FAKE, kept=FAKE, exps=None, t=0,
             h=128, f=192, act=0, dx=FAKE * 2, lddx=128, dwg=FAKE * 3, dwu=FAKE * 4, dwd=FAKE * 5, gb=16, ws=FAKE * 8,
             wsb=1 << 40)
    a.update(kw)
    return lib.ptb_gated_ffn_backward(a["dy"], a["lddy"], a["x"], a["ldx"], a["xe"], a["ldxe"], a["wg"], a["wu"], a["wd"],
                                      a["kept"], a["exps"], a["t"], a["h"], a["f"], a["act"], a["dx"], a["lddx"], a["dwg"],
                                      a["dwu"], a["dwd"], a["gb"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(wg=None), ARG), (dict(dwg=None), ARG), (dict(dwd=None), ARG), (dict(kept=None, t=1), ARG), (dict(gb=8), ARG),
    (dict(t=-1), ARG), (dict(act=5), ARG), (dict(dy=None, t=1), ARG), (dict(dx=None, t=1), ARG), (dict(x=None, t=1), ARG),
    (dict(t=2, xe=FAKE, ldxe=3), ARG), (dict(t=2, lddy=64), ARG), (dict(t=1, ws=None), ARG),
    (dict(h=72), SHAPE), (dict(f=72), SHAPE),
    (dict(dwu=FAKE + 4), ALIGN), (dict(t=1, dy=FAKE + 2), ALIGN), (dict(t=2, xe=FAKE, ldxe=4, ldx=136), ALIGN),
    (dict(t=1, wsb=64), WORKSPACE),
])
def test_gated_ffn_backward_refuses(lib, kw, code):
    assert ffn_bwd(lib, **kw) == code


def norm(lib, **kw):
    a = dict(x=FAKE, ldx=64, o=FAKE * 2, ldo=64, pg=FAKE, pb=FAKE, gate=FAKE, gates=2, alpha=1.0, ng=FAKE, nb=FAKE, rms=0,
             eps=1e-5, rows=0, h=64, y=FAKE * 3, ldy=64, out=FAKE * 4, ldh=64, stats=FAKE)
    a.update(kw)
    return lib.ptb_norm_residual(a["x"], a["ldx"], a["o"], a["ldo"], a["pg"], a["pb"], a["gate"], a["gates"], a["alpha"],
                                 a["ng"], a["nb"], a["rms"], a["eps"], a["rows"], a["h"], a["y"], a["ldy"], a["out"],
                                 a["ldh"], a["stats"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ARG), (dict(h=0), ARG), (dict(gates=0), ARG), (dict(rms=2), ARG), (dict(pg=None), ARG),
    (dict(ng=None), ARG), (dict(rms=1), ARG), (dict(rows=2, ng=None, nb=None), ARG), (dict(rows=2, out=None), ARG),
    (dict(alpha=float("inf")), ARG), (dict(alpha=float("nan")), ARG), (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(rows=2, x=None), ARG), (dict(rows=2, o=None), ARG), (dict(rows=2, y=None), ARG),
    (dict(rows=2, ldx=56), ARG), (dict(rows=2, y=FAKE * 4), ARG), (dict(rows=2, y=FAKE, ldy=128), ARG),
    (dict(rows=2, out=FAKE * 2, ldh=72), ARG),
    (dict(h=12), SHAPE), (dict(h=32776), SHAPE), (dict(rows=3), SHAPE), (dict(gates=70000, rows=140000), SHAPE),
    (dict(rows=2, x=FAKE + 8), ALIGN), (dict(rows=2, ldo=68), ALIGN), (dict(pg=FAKE + 2), ALIGN), (dict(gate=FAKE + 8), ALIGN),
    (dict(stats=FAKE + 8), ALIGN),
])
def test_norm_residual_refuses(lib, kw, code):
    assert norm(lib, **kw) == code


def norm_bwd(lib, **kw):
    a = dict(dy=FAKE, lddy=64, dh=FAKE * 2, lddh=64, y=FAKE * 3, ldy=64, o=FAKE * 4, ldo=64, oe=None, ldoe=0, stats=FAKE,
             pg=FAKE, pb=FAKE, gate=FAKE, gates=2, alpha=1.0, ng=FAKE, rms=0, rows=0, h=64, dx=FAKE * 5, lddx=64, do=FAKE * 6,
             lddo=64, dpg=FAKE, dpb=FAKE, dg=FAKE, dng=FAKE, dnb=FAKE, ws=FAKE * 8, wsb=1 << 40)
    a.update(kw)
    return lib.ptb_norm_residual_backward(a["dy"], a["lddy"], a["dh"], a["lddh"], a["y"], a["ldy"], a["o"], a["ldo"], a["oe"],
                                          a["ldoe"], a["stats"], a["pg"], a["pb"], a["gate"], a["gates"], a["alpha"], a["ng"],
                                          a["rms"], a["rows"], a["h"], a["dx"], a["lddx"], a["do"], a["lddo"], a["dpg"],
                                          a["dpb"], a["dg"], a["dng"], a["dnb"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-2), ARG), (dict(gates=0), ARG), (dict(rms=1), ARG), (dict(pg=None), ARG), (dict(gate=None), ARG),
    (dict(ng=None), ARG), (dict(rows=2, dh=None), ARG), (dict(rows=2, dh=None, ng=None, dng=None, dnb=None, dy=None), ARG),
    (dict(rows=2, stats=None), ARG), (dict(alpha=float("nan")), ARG), (dict(rows=2, y=None), ARG), (dict(rows=2, o=None), ARG),
    (dict(rows=2, dx=FAKE * 6), ARG), (dict(rows=2, dx=FAKE, lddx=128), ARG), (dict(rows=2, do=FAKE * 4, lddo=72), ARG),
    (dict(rows=2, oe=FAKE, ldoe=2, do=FAKE * 4), ARG), (dict(rows=2, oe=FAKE, ldoe=1), ARG), (dict(rows=2, ws=None), ARG),
    (dict(pb=None, pg=None, dpg=FAKE, dpb=None), ARG),
    (dict(h=12), SHAPE), (dict(h=40000), SHAPE), (dict(rows=3), SHAPE), (dict(h=40, oe=FAKE), SHAPE),
    (dict(rows=2, dy=FAKE + 8), ALIGN), (dict(rows=2, lddh=68), ALIGN), (dict(dpg=FAKE + 2), ALIGN),
    (dict(rows=2, oe=FAKE, ldoe=2, ldo=72), ALIGN), (dict(rows=2, wsb=16), WORKSPACE),
])
def test_norm_residual_backward_refuses(lib, kw, code):
    assert norm_bwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ARG), (dict(cols=0), ARG), (dict(x=None, rows=1), ARG), (dict(codes=None, rows=1), ARG),
    (dict(exps=None, rows=1), ARG), (dict(rows=2, lde=1), ARG), (dict(rows=2, ldx=32), ARG), (dict(rows=1, codes=FAKE), ARG),
    (dict(cols=48), SHAPE), (dict(rows=1 << 40), SHAPE), (dict(rows=1, x=FAKE + 4), ALIGN), (dict(rows=2, ldx=68), ALIGN),
    (dict(rows=2, ldc=72), ALIGN), (dict(rows=1, codes=FAKE * 2 + 8), ALIGN),
])
def test_checkpoints_refuse(lib, kw, code):
    a = dict(x=FAKE, ldx=64, rows=0, cols=64, codes=FAKE * 2, ldc=64, exps=FAKE * 3, lde=2)
    a.update(kw)
    assert lib.ptb_checkpoint_pack(a["x"], a["ldx"], a["rows"], a["cols"], a["codes"], a["ldc"], a["exps"], a["lde"],
                                   None) == code
    assert lib.ptb_checkpoint_unpack(a["codes"], a["ldc"], a["exps"], a["lde"], a["rows"], a["cols"], a["x"], a["ldx"],
                                     None) == code


ONE_ROW = [3, 4, -8, -1, 1 << 40]


@pytest.mark.parametrize("ld", ONE_ROW)
def test_the_stride_of_a_single_row_is_not_looked_at(lib, ld):
    """Every call is refused, for something that is checked behind the strides."""
    assert ffn(lib, t=1, ldx=ld, ldy=ld, r=FAKE * 4, ldr=ld, wsb=100) == WORKSPACE
    assert ffn_bwd(lib, t=1, lddy=ld, ldx=ld, lddx=ld, wsb=64) == WORKSPACE
    assert ffn_bwd(lib, t=1, lddy=ld, ldx=ld, xe=FAKE, ldxe=ld, lddx=ld, wsb=64) == WORKSPACE
    assert norm(lib, rows=1, gates=1, ldx=ld, ldo=ld, ldy=ld, ldh=ld, y=FAKE * 4) == ARG  # y is h
    assert norm(lib, rows=1, gates=1, ldx=ld, ldo=ld, ldy=ld, ldh=ld, y=FAKE * 4, stats=FAKE + 8) == ALIGN
    one = dict(rows=1, gates=1, lddy=ld, lddh=ld, ldy=ld, ldo=ld, lddx=ld, lddo=ld, wsb=16)
    assert norm_bwd(lib, **one) == WORKSPACE
    assert norm_bwd(lib, oe=FAKE, ldoe=ld, **one) == WORKSPACE
    for call in (lambda x: lib.ptb_checkpoint_pack(x, ld, 1, 64, FAKE * 2, ld, FAKE * 3, ld, None),
                 lambda x: lib.ptb_checkpoint_unpack(FAKE * 2, ld, FAKE * 3, ld, 1, 64, x, ld, None)):
        assert call(FAKE * 2) == ARG and call(FAKE + 4) == ALIGN  # x is the codes


def test_calls_without_rows_pass_the_checks(lib):
    assert past_checks(ffn(lib)) and past_checks(norm(lib))
    assert past_checks(ffn(lib, x=None, y=None, ws=None, wsb=0))


def test_workspace_sizes(lib):
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    t, h, f = 300, 256, 704
    assert lib.ptb_gated_ffn_workspace_size(t, h, f) >= up(t * f * 2)
    b16 = lib.ptb_gated_ffn_backward_workspace_size(t, h, f, 16)
    assert b16 >= up(t * f * 2) + up(t * f * 4)
    assert lib.ptb_gated_ffn_backward_workspace_size(t, h, f, 8) == b16 + up(t * h * 2)
    for bad in ((0, h, f), (t, 100, f), (t, h, 100), (-1, h, f)):
        assert lib.ptb_gated_ffn_workspace_size(*bad) == 0
        assert lib.ptb_gated_ffn_backward_workspace_size(*bad, 16) == 0
    assert lib.ptb_gated_ffn_backward_workspace_size(t, h, f, 4) == 0
    assert lib.ptb_norm_residual_backward_workspace_size(100, 64, 4) >= 4 * 2 * 64 * 4
    for bad in ((0, 64, 1), (100, 12, 1), (100, 64, 3), (100, 40000, 1), (100, 64, 0)):
        assert lib.ptb_norm_residual_backward_workspace_size(*bad) == 0


def test_binding_refuses_host_tensors_and_wrong_pairs():
    import block_sliding_window_gb300 as bsw
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    for call in (lambda: bsw.gated_ffn(x, w, w, w), lambda: bsw.checkpoint_pack(x),
                 lambda: bsw.norm_residual(x, x), lambda: bsw.gated_ffn_backward(x, x, w, w, w, x),
                 lambda: bsw.norm_residual_backward(x, None, x, x, x)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        bsw.gated_ffn_train(x, w, w, w, bits=4)
