"""The gated feed-forward on inputs whose results are known to the bit (tests/block_exact.py): every tile, the
joins of K pieces and the forms of what is kept have to give exactly them."""
import pytest
import torch

from tests import block_exact as X
from tests.test_gpu_block import FFNS, LONG, MANY_WEIGHTS, TILES

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(ptb_lib):
    ptb_lib.last_device_error()
    yield
    assert ptb_lib.last_device_error() == 0, "a kernel recorded a device-side error"


def on_device(ts):
    """The same numbers in bf16, all of which it holds, and in 64 bits for the products."""
    return [X.held(t).to(torch.bfloat16).cuda() for t in ts], [t.cuda() for t in ts]


def check_forward(lib, t, h, f, seed):
    (x, wg, wu, wd, resid), wide = on_device(X.forward_inputs(t, h, f, seed))
    for r, wr in ((None, None), (resid, wide[4])):
        gate, up, _, y = X.forward(*wide[:4], wr)
        y = X.bf16(y)
        for act in ("silu", "gelu"):
            assert torch.equal(lib.gated_ffn(x, wg, wu, wd, activation=act, residual=r), y)
        for bits in (16, 8):
            got, kept = lib.gated_ffn_train(x, wg, wu, wd, bits=bits, residual=r)
            kept = kept if bits == 16 else lib.checkpoint_unpack(*kept)
            assert torch.equal(got, y) and torch.equal(kept.double(), torch.cat([gate, up], 1))


def check_backward(lib, t, h, f, seed):
    (dy, x, wg, wu, wd, gate, up), wide = on_device(X.backward_inputs(t, h, f, seed))
    want = X.backward(*wide)
    both = torch.cat([gate, up], 1)
    for act, x_in, kept, dtype in (("silu", x, both, torch.bfloat16), ("gelu", x, both, torch.float32),
                                   ("silu", lib.checkpoint_pack(x), lib.checkpoint_pack(both), torch.bfloat16)):
        got = lib.gated_ffn_backward(dy, x_in, wg, wu, wd, kept, activation=act, grad_dtype=dtype)
        for k, w in want.items():
            assert torch.equal(got[k], X.bf16(w) if got[k].dtype == torch.bfloat16 else w.float()), k


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("t,h,f", LONG + TILES + MANY_WEIGHTS)
def test_exact(ptb_lib, t, h, f, pairs):
    was = ptb_lib.set_gemm_pairs(pairs)
    try:
        check_forward(ptb_lib, t, h, f, t + h)
        check_backward(ptb_lib, t, h, f, t + f)
    finally:
        ptb_lib.set_gemm_pairs(was)


@pytest.mark.parametrize("t,h,f", FFNS)
def test_exact_small(ptb_lib, t, h, f):
    check_forward(ptb_lib, t, h, f, t + h)
    check_backward(ptb_lib, t, h, f, t + f)
