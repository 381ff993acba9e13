"""Pins of the 64-bit model that the gated feed-forward, the norms around a block and the checkpoints
are tested against: gradients against differences and torch's own, codes against their definition."""
import math

import pytest
import torch

from tests import block_model as M


def rnd(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64) * std


def differences(f, t, seed):
    """(numerical, index) pairs of df/dt at a few places; f is a scalar."""
    g = torch.Generator().manual_seed(seed)
    flat = t.reshape(-1)
    for i in torch.randint(0, flat.numel(), (6,), generator=g).tolist():
        was, h = flat[i].item(), 1e-5
        flat[i] = was + h
        up = f()
        flat[i] = was - h
        down = f()
        flat[i] = was
        yield (up - down) / (2 * h), i


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_ffn_gradients_against_differences(name):
    x, wg, wu, wd = rnd(5, 8, seed=1), rnd(12, 8, seed=2), rnd(12, 8, seed=3), rnd(8, 12, seed=4)
    dy = rnd(5, 8, seed=5)
    g, _, u, _, _, _ = M.ffn(x, wg, wu, wd, name)
    out = M.ffn_backward(dy, x, wg, wu, wd, g, u, name, M.U16)
    f = lambda: float((M.ffn(x, wg, wu, wd, name)[4] * dy).sum())  # noqa: E731
    for key, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd)):
        for num, i in differences(f, t, 7):
            assert abs(out[key][0].reshape(-1)[i].item() - num) < 1e-6 * max(1, abs(num)), key


@pytest.mark.parametrize("name,ref", [("silu", torch.nn.functional.silu),
                                      ("gelu", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))])
def test_activations_against_torch(name, ref):
    z = torch.linspace(-12, 12, 4001, dtype=torch.float64, requires_grad=True)
    ref(z).sum().backward()
    v, s = M.act(z.detach(), name)
    assert torch.allclose(v, ref(z.detach()), atol=1e-12) and torch.allclose(s, z.grad, atol=1e-12)
    assert s.abs().max() < M.SLOPE


CASES = [dict(post=p, pre=n, gates=k, rms=r) for p in (0, 1) for n in (0, 1) for k in (0, 1, 3) for r in (0, 1)]


@pytest.mark.parametrize("c", CASES)
def test_norm_gradients_against_differences(c):
    rows, n, eps, alpha = 6, 10, 1e-2, 0.7
    x, o, dy, dh = (rnd(rows, n, seed=s) for s in (1, 2, 3, 4))
    pg, pb = (rnd(n, seed=5) + 1, rnd(n, seed=6)) if c["post"] else (None, None)
    ng, nb = (rnd(n, seed=7) + 1, rnd(n, seed=8)) if c["pre"] else (None, None)
    if c["rms"]:
        pb = nb = None
    gate = rnd(c["gates"], n, seed=9) if c["gates"] else None
    if not c["pre"]:
        dh = None

    def f():
        y, _, h, _, _ = M.norm_residual(x, o, pg, pb, gate, alpha, ng, nb, c["rms"], eps)
        return float((y * dy).sum() + (0 if h is None else (h * dh).sum()))

    y = M.norm_residual(x, o, pg, pb, gate, alpha, ng, nb, c["rms"], eps)[0]
    out = M.norm_backward(dy, dh, y, o, pg, pb, gate, alpha, ng, c["rms"], eps)
    for key, t in (("dx", x), ("do", o), ("dpost_gamma", pg), ("dpost_beta", pb), ("dgate", gate),
                   ("dpre_gamma", ng), ("dpre_beta", nb)):
        if t is not None:
            for num, i in differences(f, t, 3):
                assert abs(out[key][0].reshape(-1)[i].item() - num) < 1e-6 * max(1, abs(num)), key


def test_norm_without_gate_or_post_is_layer_norm():
    x, o = rnd(4, 16, seed=1), rnd(4, 16, seed=2)
    g, b = rnd(16, seed=3), rnd(16, seed=4)
    y, _, h, _, _ = M.norm_residual(x, o, None, None, None, 1.0, g, b, 0, 1e-5)
    assert torch.equal(y, x + o)
    assert torch.allclose(h, torch.nn.functional.layer_norm(x + o, (16,), g, b, 1e-5), atol=1e-12)


def test_checkpoint_definition():
    x = rnd(40, 96, seed=3).to(torch.bfloat16).double()
    x[0, :32] = 0
    x[1, :32] = 127.5                   # the border: a scale of 2, codes of 64 (63.75)
    x[2, :32] = 127.0
    x[3, 0] = 2.0 ** -133               # bf16's smallest
    x[3, 1:32] = 0
    codes, exps = M.pack(x)
    v = M.unpack(codes, exps)
    step = torch.ldexp(torch.ones(exps.shape, dtype=torch.float64), exps.long() - 127)
    m = x.abs().reshape(40, 3, 32).amax(2)
    assert (m < 127.5 * step).all()
    assert ((m >= 127.5 * step / 2) | (exps == 1)).all()
    assert ((v - x).abs() <= step.repeat_interleave(32, 1) / 2).all()
    assert (codes.abs() <= 127).all()
    assert torch.equal(v, v.to(torch.bfloat16).double())
    assert exps[0, 0] == 1 and exps[1, 0] == 128 and exps[2, 0] == 127 and exps[3, 0] == 1


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan, 255 * 2.0 ** 120])
def test_checkpoint_of_what_has_no_code(bad):
    x = rnd(2, 64, seed=1)
    x[1, 40] = bad
    codes, exps = M.pack(x)
    v = M.unpack(codes, exps)
    assert exps[1, 1] == 255 and torch.isnan(v[1, 32:]).all() and torch.isfinite(v[0]).all()
    assert torch.isfinite(v[1, :32]).all()
