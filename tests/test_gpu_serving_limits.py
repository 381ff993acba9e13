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


@pytest.mark.parametrize("heads", [3, 11])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_paged_4bit_rows_that_hold_nan_in_one_group(ptb_lib, heads, d):
    """Every number of groups a row: NaN in one group of keys or values that the window has left
    reaches nothing, and in a key inside the window it reaches its sequence alone."""
    lens, window, page = [75, 64, 33], 30, 16
    pages = sum(-(-n // page) for n in lens)
    table = np.full((3, 5), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = range(at, at + need)
        at += need
    cache = torch.full((pages, ptb_lib.kv_page_size(1, page, d, 4)), 0xFF, dtype=torch.uint8, device="cuda")
    cu = cumulated(lens)
    k, v, q = normal((cu[-1], 1, d), 21), normal((cu[-1], 1, d), 22), normal((3, heads, d), 23)
    first, last = 0, d // 32 - 1
    for b, n in enumerate(lens):
        for p in range(n - window):
            k[cu[b] + p, 0, 32 * (first if p % 2 else last)] = float("nan")
            v[cu[b] + p, 0, 32 * (last if p % 2 else first)] = float("nan")
    dev = torch.from_numpy(table).cuda()
    ptb_lib.kv_append(None, k, v, cache, dev, ints(cu), ints([0] * 3), page, 4, keep_keys=False)
    host = M.Cache(cache.cpu().numpy(), 1, page, d, 4)
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, dev, ints(lens), 1, page, 4, window))
    want, bound = M.paged(M.to64(q), host, table, lens, window, d ** -0.5)
    assert (np.abs(o - want) <= bound).all()
    k[cu[1] + 50, 0, 32 * last] = float("nan")
    ptb_lib.kv_append(None, k, v, cache, dev, ints(cu), ints([0] * 3), page, 4, keep_keys=False)
    o = M.to64(ptb_lib.swa_attention_paged(q, cache, dev, ints(lens), 1, page, 4, window))
    assert np.isnan(o[1]).all() and (np.abs(o - want)[[0, 2]] <= bound[[0, 2]]).all()
