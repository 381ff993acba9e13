"""Limits of the serving entry points, on the host: sizes asked for shapes that are refused.  Nothing
here touches a device."""

import subprocess
import sys

import pytest

SHAPE = 2

SIZES = """
import block_sliding_window_gb300 as bsw
lib = bsw.load()
for a in {cases!r}:
    print(lib.swa_attention_packed_workspace_size(*a), flush=True)
"""


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import block_sliding_window_gb300 as bsw
    return bsw.load()


def test_packed_workspace_of_groups_beyond_a_tile(lib):
    """More than 128 query heads of one kv head: size 0, like every refused shape.  In a process of
    its own: dividing by a tile of no tokens would end it."""
    cases = [(2, 100, 256, 1), (1, 0, 129, 1), (3, 5000, 65535, 1), (2, 100, 1290, 10)]
    r = subprocess.run([sys.executable, "-c", SIZES.format(cases=cases)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert r.stdout.split() == ["0"] * len(cases)
    # 128 is served; a call of any length is refused beyond it
    assert lib.swa_attention_packed_workspace_size(2, 10 ** 6, 128, 1) > 0
    p = 1 << 20
    for heads in (129, 256):
        st = lib.swa_attention_packed(p, heads * 64, 64, 2 * p, 64, 64, 3 * p, 64, 64, p, None, 2, 100, 100, heads, 1, 64,
                                      8, 0.0, 4 * p, heads * 64, 64, p, 1 << 40, None)
        assert st == SHAPE


@pytest.mark.parametrize("scale", [2.0 ** 126 * 1.0001, 3e38, -1e-30, float("nan"), float("inf")])
def test_attention_refuses_scales_whose_factor_overflows(lib, scale):
    """scale * log2(e) has to be a number below 2^127 (2^126 is the last power of two that is)."""
    p, arg, align = 1 << 20, 1, 3
    # lens and cu_seqlens are misaligned, so that no scale gets as far as a launch
    packed = lambda s: lib.swa_attention_packed(p, 256, 64, 2 * p, 128, 64, 3 * p, 128, 64, p + 1, None, 2, 100, 100, 4, 2,  # noqa: E731
                                                64, 8, s, 4 * p, 256, 64, p, 1 << 40, None)
    paged = lambda s: lib.swa_attention_paged(p, 256, 64, 2 * p, 10, p, 5, 5, p + 1, 2, 4, 2, 64, 16, 4, 8, s, 4 * p, 256, 64,  # noqa: E731
                                              p, 1 << 40, None)
    for call in (packed, paged):
        assert call(scale) == arg
        assert call(2.0 ** 126) == align and call(0.0) == align


@pytest.mark.parametrize("high", [1 << 32, -(1 << 32), 1 << 40])
def test_sizes_refuse_numbers_beyond_32_bits(lib, high):
    """Not the answer for their low 32 bits."""
    import block_sliding_window_gb300 as bsw
    for f, args in ((bsw.kv_page_size, (8, 64, 128, 16)), (bsw.swa_attention_paged_workspace_size, (2, 4, 2, 64)),
                    (bsw.swa_attention_packed_workspace_size, (2, 10 ** 6, 4, 2))):
        assert f(*args) > 0
        for i in range(4):
            if args[i] == 10 ** 6:  # tokens: 64 bits
                continue
            with pytest.raises(ValueError, match="32 bits"):
                f(*(a + high if i == j else a for j, a in enumerate(args)))
