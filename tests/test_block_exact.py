"""Pins of tests/block_exact.py: its inputs are exact at the sizes that the GPU tests use, and a K piece that
is lost or added twice is seen, which the general bounds of tests/block_model.py do not at these sizes."""
import pytest
import torch

from tests import block_exact as X
from tests import block_model as M

LONG = [(100003, 64, 64), (20000, 128, 64), (3, 64, 39936), (65, 10240, 128)]


def pieces(a, b, n):
    """(without, twice): a b^T less a middle one of n pieces of K, and with it twice."""
    k = a.shape[1]
    lo, hi = n // 2 * k // n, (n // 2 + 1) * k // n
    piece = a[:, lo:hi] @ b[:, lo:hi].t()
    return a @ b.t() - piece, a @ b.t() + piece


@pytest.mark.parametrize("n", [12, 32])
@pytest.mark.parametrize("t,h,f", LONG)
def test_a_lost_or_doubled_piece_is_seen(t, h, f, n):
    s = X.backward_inputs(t, h, f, seed=t + h + f)
    dy, x, wg, wu, wd, gate, up = s
    want = X.backward(*s)
    a, dg, du = X.backward_operands(*s)
    operands = dict(dx=(torch.cat([dg, du], 1), torch.cat([wg, wu], 0).t()), dw_gate=(dg.t(), x.t()),
                    dw_up=(du.t(), x.t()), dw_down=(dy.t(), a.t()))
    checked = 0
    for k, (p, q) in operands.items():
        if p.shape[1] >= 512 * n:  # a piece has 8 blocks of 64 at least
            for wrong in pieces(p, q, n):
                assert (X.bf16(wrong) != X.bf16(want[k])).double().mean() > 0.8, k
                assert (wrong.float() != want[k].float()).double().mean() > 0.8, k
                checked += 1
    sparse = [(dy, wd.t())]  # products over hidden: few terms, so that what they give fits bf16
    x, wg, wu, wd, resid = X.forward_inputs(t, h, f, seed=t)
    _, _, a, y = X.forward(x, wg, wu, wd, resid)
    sparse.append((x, wu))
    if f >= 512 * n:
        for wrong in pieces(a, wd, n):
            assert (X.bf16(wrong + resid) != X.bf16(y)).double().mean() > 0.8
            checked += 1
    if h >= 512 * n:
        for p, q in sparse:
            for wrong in pieces(p, q, n):
                assert (wrong != p @ q.t()).double().mean() > 0.5
                checked += 1
    assert checked or n * 512 > max(t, h, f)


@pytest.mark.parametrize("t,h,f", [(300, 192, 128), (40, 2048, 320), (1, 64, 64)])
def test_the_model_agrees(t, h, f):
    """The 64-bit model on the same inputs: the activations' tails and nothing else apart."""
    x, wg, wu, wd, resid = X.forward_inputs(t, h, f, seed=1)
    gate, up, _, y = X.forward(x, wg, wu, wd, resid)
    g, _, u, _, my, _ = M.ffn(x, wg, wu, wd, "silu", resid)
    assert torch.equal(g, gate) and torch.equal(u, up) and torch.allclose(my, y, rtol=0, atol=1e-6)
    s = X.backward_inputs(t, h, f, seed=2)
    want = X.backward(*s)
    for name in ("silu", "gelu"):
        got = M.ffn_backward(*s, name, M.U32)
        for k in want:
            assert torch.allclose(got[k][0], want[k], rtol=1e-10, atol=1e-6), k
