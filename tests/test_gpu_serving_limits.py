"""The serving operators on the GPU at the limits of what they document: refusals through the
binding, partly filled tiles, values of extreme size, calls of many items and long shares."""
import pytest
import torch

from block_sliding_window_gb300 import workloads

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
