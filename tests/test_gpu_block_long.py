"""The gated feed-forward, the norms around a block and the checkpoints where offsets pass 32 bits: tensors of
more than 2^32 elements (the norms' of more than 2^31), checked from the first row to the last."""
import pytest
import torch

from tests import block_exact as X
from tests import block_model as M

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean(ptb_lib):
    ptb_lib.last_device_error()
    yield
    torch.cuda.empty_cache()
    assert ptb_lib.last_device_error() == 0, "a kernel recorded a device-side error"


def filled(rows, cols, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, 16384):
        part = t[at:at + 16384]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
    return t


@pytest.mark.parametrize("bits", [16, 8])
def test_gated_ffn_long(ptb_lib, bits):
    t, h, f, step = 140001, 64, 16384, 8192
    x, wg, wu, wd, _ = (v.cuda() for v in X.forward_inputs(t, h, f, 1))
    g = torch.Generator().manual_seed(2)
    dy = torch.zeros(t, h, dtype=torch.float64)
    dy[torch.arange(t), torch.randint(0, h, (t,), generator=g)] = X.signs(g, t)
    dy = dy.cuda()
    wd2 = X.signs(g, h, f, density=0.25).cuda()  # (of few terms for dx)
    low = lambda v: v.to(torch.bfloat16)  # noqa: E731
    y, kept = ptb_lib.gated_ffn_train(low(x), low(wg), low(wu), low(wd), bits=bits)
    out = ptb_lib.gated_ffn_backward(low(dy), low(x), low(wg), low(wu), low(wd2), kept, grad_dtype=torch.float32)
    sums = {k: torch.zeros(f, h, dtype=torch.float64, device="cuda") for k in ("dw_gate", "dw_up", "dw_down")}
    size = {k: torch.zeros_like(v) for k, v in sums.items()}
    for at in range(0, t, step):
        r = slice(at, min(at + step, t))
        gate, up, a, want = X.forward(x[r], wg, wu, wd)
        both = kept[r] if bits == 16 else ptb_lib.checkpoint_unpack(kept[0][r], kept[1][r])
        assert torch.equal(both, low(torch.cat([gate, up], 1))), at
        assert torch.equal(y[r], X.bf16(want)), at
        da = X.product(dy[r], wd2.t())
        dg, du = X.held(da * up), X.held(da * gate)
        dx = X.product(torch.cat([dg, du], 1), torch.cat([wg, wu], 0).t())
        assert torch.equal(out["dx"][r], X.bf16(dx)), at
        for k, p, q in (("dw_gate", dg, x[r]), ("dw_up", du / 32, x[r]), ("dw_down", a / 32, dy[r])):
            sums[k] += p.t() @ q
            size[k] += p.abs().t() @ q.abs()
    assert all(v.max() < X.EXACT for v in size.values())
    assert torch.equal(out["dw_gate"], sums["dw_gate"].float())
    assert torch.equal(out["dw_up"], (32 * sums["dw_up"]).float())
    assert torch.equal(out["dw_down"], (32 * sums["dw_down"]).float().t())


@pytest.mark.parametrize("rms", [0, 1])
def test_norms_long(ptb_lib, rms):
    rows, n, gates = 70002, 32768, 3
    x, o = filled(rows, n, 1, 2.0), filled(rows, n, 2)
    p = dict(post_gamma=filled(1, n, 3)[0], gate=filled(gates, n, 4), pre_gamma=filled(1, n, 5)[0],
             post_beta=None if rms else filled(1, n, 6)[0], pre_beta=None if rms else filled(1, n, 7)[0])
    y, h, stats = ptb_lib.norm_residual_train(x, o, rms=bool(rms), **p)
    dy, dh = x.mul_(0.05), filled(rows, n, 8, 0.1)
    kept = ptb_lib.checkpoint_pack(o)
    out = ptb_lib.norm_residual_backward(dy, dh, y, o, stats, rms=bool(rms), **p)
    d = {k: M.d(v) for k, v in p.items()}
    for at in (0, rows // 3 - 2, rows // 3 - 1, rows // 3, rows // 2, 65535, 65536, rows - 2):
        r = slice(at, at + 2)
        gate = d["gate"][[k * gates // rows for k in range(at, at + 2)]]
        xs = M.d(dy[r]) * 20  # within half a step of x, which the stream's gradient took the place of
        wy, ey, wh, eh, _ = M.norm_residual(xs, M.d(o[r]), d["post_gamma"], d["post_beta"], gate, 1.0, d["pre_gamma"],
                                            d["pre_beta"], rms, 1e-5, M.d(y[r]))
        M.held_to(f"y at {at}", y[r], wy, ey + 2 * M.U16 * xs.abs())
        M.held_to(f"h at {at}", h[r], wh, eh)
        want = M.norm_backward(M.d(dy[r]), M.d(dh[r]), M.d(y[r]), M.d(o[r]), d["post_gamma"], d["post_beta"], gate, 1.0,
                               d["pre_gamma"], rms, 1e-5)
        M.held_to(f"dx at {at}", out["dx"][r], *want["dx"])
        M.held_to(f"do at {at}", out["do"][r], *want["do"])
        codes, exps = M.pack(M.d(o[r]))
        assert torch.equal(kept[0][r].cpu(), codes) and torch.equal(kept[1][r].cpu(), exps), at
    if not rms:
        total, size = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
        for at in range(0, rows, 4096):
            part = dh[at:at + 4096].double()
            total += part.sum(0)
            size += part.abs().sum(0)
        M.held_to("dpre_beta", out["dpre_beta"], total.cpu(), (rows * 2 * M.U32 * size).cpu())


def test_checkpoint_long(ptb_lib):
    for rows, cols in ((2100003, 2048), (1, (1 << 30) - 32), (3, 1 << 30)):
        base = filled(4096, 2048, 1).reshape(-1)
        x = base.repeat(rows * cols // base.numel() + 1)[:rows * cols].view(rows, cols)
        codes, exps = ptb_lib.checkpoint_pack(x)
        want = ptb_lib.checkpoint_pack(base.view(1, -1))
        assert torch.equal(want[0].cpu(), M.pack(M.d(base.view(1, -1)))[0])
        flat, back = codes.view(-1), ptb_lib.checkpoint_unpack(codes, exps).view(-1)
        value = ptb_lib.checkpoint_unpack(*want).view(-1)
        for at in range(0, rows * cols, base.numel()):
            k = min(base.numel(), rows * cols - at)
            assert torch.equal(flat[at:at + k], want[0].view(-1)[:k]), at
            assert torch.equal(back[at:at + k], value[:k]), at
            assert torch.equal(exps.view(-1)[at // 32:(at + k) // 32], want[1].view(-1)[:k // 32]), at
        del x, codes, exps, flat, back
