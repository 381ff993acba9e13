"""Inputs of the gated feed-forward whose results are known to the bit, whatever the order of the sums.

All operands are whole numbers (times a power of two), small enough that the magnitudes of a sum's terms
add up to less than 2^24 units: every partial sum is then an fp32 number.  Gates are 32 or 64, where both
activations are the identity to fp32's last bit and their derivative is 1 (e^-32 < 2^-46), and the values
that are rounded to bf16 between the products are whole numbers up to 256 (times 32 or 64), which bf16
holds.  So outputs have to be equal, and a K piece that is lost or added twice shows in nearly all of
them, where the general bounds grow with K and the sums only with its root."""
import torch

EXACT = 2.0 ** 24


def whole(g, *shape, most, density=1.0):
    """Whole numbers from -most to most, zero but for a share `density`."""
    v = torch.randint(-most, most + 1, shape, generator=g).double()
    return v if density >= 1 else v * (torch.rand(shape, generator=g) < density)


def signs(g, *shape, density=1.0):
    v = torch.randint(0, 2, shape, generator=g).double() * 2 - 1
    return v if density >= 1 else v * (torch.rand(shape, generator=g) < density)


def product(a, b, unit=1.0):
    """a b^T, checked to be exact in fp32 in any order."""
    assert ((a.abs() @ b.abs().t()) / unit).max() < EXACT
    return a @ b.t()


def bf16(t):
    return t.to(torch.float32).to(torch.bfloat16)


def held(t):
    """t, which bf16 holds."""
    assert torch.equal(bf16(t).double(), t)
    return t


def forward_inputs(t, h, f, seed):
    """x, w_gate, w_up, w_down, residual: gates of 32 and 64, from one of several columns of x each."""
    g = torch.Generator().manual_seed(seed)
    x = whole(g, t, h, most=2)
    ones = torch.arange(0, h, 64)
    x[:, ones] = 8
    wg = torch.zeros(f, h, dtype=torch.float64)
    at = ones[torch.randint(0, len(ones), (f,), generator=g)]
    wg[torch.arange(f), at] = 4.0 * torch.randint(1, 3, (f,), generator=g).double()
    wu = signs(g, f, h, density=min(1, 24 / h))
    wu[:, ones] = 0
    wd = signs(g, h, f, density=min(1, 4096 / f))
    return x, wg, wu, wd, whole(g, t, h, most=100)


def forward(x, wg, wu, wd, resid=None):
    """(gate, up, act(gate) up, y before it is rounded)"""
    gate, up = product(x, wg), product(x, wu)
    assert ((gate == 32) | (gate == 64)).all() and up.abs().max() < 127.5
    a = held(gate * up)
    y = product(a, wd, 32.0)
    if resid is not None:
        y = y + resid
        assert y.abs().max() < EXACT
    return gate, up, a, y


def backward_inputs(t, h, f, seed):
    """dy, x, w_gate, w_up, w_down, gate, up"""
    g = torch.Generator().manual_seed(seed)
    few = min(1, 2048 / f)
    gate = 32.0 * torch.randint(1, 3, (t, f), generator=g).double()
    return (whole(g, t, h, most=2), whole(g, t, h, most=2), signs(g, f, h, density=few), signs(g, f, h, density=few),
            signs(g, h, f, density=min(1, 96 / h)), gate, signs(g, t, f) * torch.randint(1, 3, (t, f), generator=g))


def backward_operands(dy, x, wg, wu, wd, gate, up):
    """The operands of the products behind da: a, dg, du."""
    da = product(dy, wd.t())
    assert (da * up).abs().max() <= 256
    return held(gate * up), held(da * up), held(da * gate)


def backward(dy, x, wg, wu, wd, gate, up):
    """The gradients before they are rounded."""
    a, dg, du = backward_operands(dy, x, wg, wu, wd, gate, up)
    both, w = torch.cat([dg, du], 1), torch.cat([wg, wu], 0)
    return dict(dx=product(both, w.t()), dw_gate=product(dg.t(), x.t()), dw_up=product(du.t(), x.t(), 32.0),
                dw_down=product(dy.t(), a.t(), 32.0))
