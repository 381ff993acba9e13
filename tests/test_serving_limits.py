"""Limits of the serving entry points, on the host: sizes asked for shapes that are refused.  Nothing
here touches a device."""

import subprocess
import sys

import pytest
import torch

from tests import serving_exact as X

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


@pytest.mark.parametrize("bits", [16, 4])
def test_limits_of_long_rows_show_a_lost_key(bits):
    """Mistakes planted in the 64-bit model pass the limits that GPU rows are held to: a block of 32
    keys left out, one key left out, a page taken twice, a row of codes that reads another's pair."""
    n, heads, kv, d, page = 1500, 4, 2, 64, 16
    gen = torch.Generator().manual_seed(5)
    pages = -(-n // page)
    cache = torch.zeros(pages, 2, kv, page * (2 * d if bits == 16 else d // 2 + d // 8), dtype=torch.uint8)
    x = torch.randn(pages, 2, kv, page, d, generator=gen)
    if bits == 16:
        cache[:] = x.to(torch.bfloat16).flatten(-2).view(torch.uint8)
    else:
        cache[..., :page * d // 2] = torch.randint(0, 256, (pages, 2, kv, page * d // 2), generator=gen, dtype=torch.uint8)
        pair = torch.rand(pages, 2, kv, page * d // 32, 2, generator=gen) * torch.tensor([0.2, 0.1]) + torch.tensor([0.1, -0.05])
        cache[..., page * d // 2:] = pair.to(torch.bfloat16).flatten(-2).view(torch.uint8)
    cache = cache.flatten(1)
    q = torch.randn(1, heads, d, generator=gen).to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32)[None]
    args = (kv, page, bits)
    want, bound = X.paged(q, cache, table, [n], *args, 1 << 20, d ** -0.5)
    assert X.row_error(want.bfloat16().double(), want) <= X.ROW_LIMIT / 3  # the output's rounding alone
    assert torch.isfinite(want).all() and (bound > 0).all()
    twice = table.clone()
    twice[0, 10] = 11
    moved = cache.clone()
    at = page * d // 2 if bits == 4 else 0
    moved.view(pages, 2, kv, -1)[3, 1, :, at:] = moved.view(pages, 2, kv, -1)[3, 1, :, at:].roll(d // 8 if bits == 4 else 2 * d, -1)
    for c, t, m, w in ((cache, table, n, n - 32), (cache, table, n, n - 1), (cache, twice, n, n), (moved, table, n, n)):
        other, _ = X.paged(q, c, t, [m], *args, w, d ** -0.5)
        assert X.row_error(other, want) > X.ROW_LIMIT, (w, X.row_error(other, want))
