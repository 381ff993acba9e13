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
