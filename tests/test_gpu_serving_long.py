"""The serving attention kernels where they run as they do in service: every warp of the paged kernel
streams many units of many sequences, every CTA of the packed kernel takes many items; against
64-bit models (tests/serving_exact.py, tests/serving_model.py)."""
import numpy as np
import pytest
import torch

from block_sliding_window_gb300 import workloads
from tests import serving_exact as X
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


def cumulated(ls):
    out = [0]
    for n in ls:
        out.append(out[-1] + n)
    return out


def table_of(lens, page, seed):
    """Pages in a random order; entries behind a sequence's last page are out of range."""
    need = [-(-n // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(need) + 1)
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), sum(need) + 1


RAGGED = [1, 4000, 31, 900, 2500, 33, 0, 3999, 64, 1700, 3000, 100, 3500, 2049, 3333, 8, 2900, 1024, 3100, 400, 2222, 3700,
          1500, 3456]
SHORT = [15, 16, 17, 31, 32, 33, 0, 129, 1]


def filled(ptb_lib, lens, heads, kv, d, page, bits, seed, spikes):
    """A cache filled by kv_append (unwritten rows read as NaN), and queries.  With spikes, every
    sequence has two keys, somewhere behind its middle, whose scores pass all earlier ones by 2^9.5
    and 2^19 (log2 domain): the reference maximum is raised over sums that count."""
    rng = np.random.RandomState(seed)
    t, cu = sum(lens), cumulated(lens)
    q, k, v = normal((len(lens), heads, d), seed), normal((t, kv, d), seed + 1), normal((t, kv, d), seed + 2)
    if spikes:
        q[:, :, 0], k[:, :, 0] = 4.0, 0.0
        step = 9.5 * np.log(2) / (4 * d ** -0.5)
        for b, n in enumerate(lens):
            if n > 8:
                first = rng.randint(n // 2, n - 2)
                second = rng.randint(first + 1, n)
                k[cu[b] + first, :, 0] = step
                if b % 2:
                    k[cu[b] + second, :, 0] = 2 * step
    table, pages = table_of(lens, page, seed)
    cache = torch.full((pages, ptb_lib.kv_page_size(kv, page, d, bits)), 0xFF, dtype=torch.uint8, device="cuda")
    ptb_lib.kv_append(None, k, v, cache, table, ints(cu), ints([0] * len(lens)), page, bits, keep_keys=False)
    return q, cache, table


def units(lens, window, kv, heads):
    """32-key blocks of all (sequence, kv head, up to 8 or 16 query heads)."""
    g = heads // kv
    blocks = -(-g // (16 if g > 8 else 8))
    return kv * blocks * sum((n - 1) // 32 - max(0, n - window) // 32 + 1 for n in lens if n)


def held_to(o, want, bound):
    o = o.double()
    assert torch.isfinite(o).all()
    over = (o - want).abs() - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} values beyond the bound, by up to {over.max():.3e}"
    off = X.row_error(o, want)
    assert off <= X.ROW_LIMIT, f"a row is off by {off:.3e} of its length"


LONG = [
    # heads, kv heads, d, page, window
    (64, 8, 128, 16, 1 << 20),
    (64, 8, 128, 64, 1000),
    (96, 8, 128, 64, 1 << 20),     # groups of 12: 16 query heads a block
    (80, 4, 96, 16, 1 << 20),      # groups of 20: two blocks of query heads
    (48, 8, 96, 32, 1 << 20),
    (16, 8, 64, 128, 1 << 20),
    (16, 16, 32, 256, 3000),
    (72, 8, 64, 16, 1 << 20),
    (16, 4, 16, 32, 1 << 20),
]


@pytest.mark.parametrize("spikes", [False, True])
@pytest.mark.parametrize("heads,kv,d,page,window,bits",
                         [c + (bits,) for c in LONG for bits in (16, 4) if c[2] % 32 == 0 or bits == 16])
def test_paged_many_units_a_warp(ptb_lib, heads, kv, d, page, window, bits, spikes):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = list(RAGGED)
    # more than twice the stages (at most 3) of the most warps that a block has (12)
    while units(lens, window, kv, heads) < 2 * 3 * 12 * sms:
        lens += RAGGED
    q, cache, table = filled(ptb_lib, lens, heads, kv, d, page, bits, 500, spikes)
    o = ptb_lib.swa_attention_paged(q, cache, table, ints(lens), kv, page, bits, window)
    want, bound = X.paged(q, cache, table, lens, kv, page, bits, window, d ** -0.5)
    held_to(o, want, bound)
    assert torch.equal(o, ptb_lib.swa_attention_paged(q, cache, table, ints(lens), kv, page, bits, window))


@pytest.mark.parametrize("bits", [16, 4])
def test_paged_many_units_of_one_sequence(ptb_lib, bits):
    """One segment a kv head, cut between most blocks and between their warps."""
    lens, heads, kv, d, page = [60001], 16, 2, 128, 64
    q, cache, table = filled(ptb_lib, lens, heads, kv, d, page, bits, 520, True)
    o = ptb_lib.swa_attention_paged(q, cache, table, ints(lens), kv, page, bits, 1 << 20)
    held_to(o, *X.paged(q, cache, table, lens, kv, page, bits, 1 << 20, d ** -0.5))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("heads,kv,d", [(16, 8, 64), (96, 8, 128), (8, 8, 32), (24, 8, 96)])
def test_paged_one_heavy_key(ptb_lib, heads, kv, d, bits):
    """A key with most of the weight that comes after the reference of its part was set, by less than 2^8
    over it, is not rounded on its way into the output: within the bound, which leaves its weight out,
    and on the average no further from 64 bits than the output's own rounding and a tenth.  So many
    sequences that a warp holds whole ones."""
    page, sms = 16, torch.cuda.get_device_properties(0).multi_processor_count
    lens = [33 + b % 17 for b in range(6 * 12 * sms // (2 * kv))]
    q, cache, table = filled(ptb_lib, lens, heads, kv, d, page, bits, 700, False)
    k, v, cu = normal((sum(lens), kv, d), 701, std=0.02), normal((sum(lens), kv, d), 702), cumulated(lens)
    q[:, :, 0], k[:, :, 0] = 4.0, 0.0
    for b, n in enumerate(lens):
        k[cu[b] + 32 + b % (n - 32), :, 0] = (7 + b % 31 / 32) * np.log(2) / (4 * d ** -0.5)
    ptb_lib.kv_append(None, k, v, cache, table, ints(cu), ints([0] * len(lens)), page, bits, keep_keys=False)
    o = ptb_lib.swa_attention_paged(q, cache, table, ints(lens), kv, page, bits, 1 << 20)
    want, bound = X.paged(q, cache, table, lens, kv, page, bits, 1 << 20, d ** -0.5)
    assert ((o.double() - want).abs() <= bound).all()
    err, own = (o.double() - want).norm(), (want.bfloat16().double() - want).norm()
    assert err <= 1.1 * own, err / own


@pytest.mark.parametrize("heads,kv,d,page,window", [(8, 2, 128, 16, 1 << 20), (24, 2, 64, 32, 40), (6, 2, 96, 16, 1 << 20),
                                                    (40, 2, 96, 32, 48), (3, 3, 32, 64, 100)])
def test_paged_4bit_short_sequences(ptb_lib, heads, kv, d, page, window):
    """The 4-bit scores and weights within the bound of the arithmetic that the kernel does."""
    q, cache, table = filled(ptb_lib, SHORT, heads, kv, d, page, 4, 540, False)
    q[:, ::2] *= 3
    o = ptb_lib.swa_attention_paged(q, cache, table, ints(SHORT), kv, page, 4, window)
    want, bound = X.paged(q, cache, table, SHORT, kv, page, 4, window, d ** -0.5)
    assert ((o.double() - want).abs() <= bound).all()


def test_the_two_models_agree(ptb_lib):
    """tests/serving_model.py and tests/serving_exact.py, written apart, on one cache."""
    for bits in (16, 4):
        q, cache, table = filled(ptb_lib, SHORT, 8, 2, 96, 32, bits, 550, False)
        o, _ = X.paged(q, cache, table, SHORT, 2, 32, bits, 50, 96 ** -0.5)
        host = M.Cache(cache.cpu().numpy(), 2, 32, 96, bits)
        want, _ = M.paged(M.to64(q), host, table.cpu().numpy(), SHORT, 50, 96 ** -0.5)
        assert np.abs(o.cpu().numpy() - want).max() < 1e-12


# -------------------------------------------------------------------------- packed attention --

def run_packed(ptb_lib, lq, lk, heads, kv, d, window, seed):
    cu_q, cu_k = cumulated(lq), cumulated(lk or lq)
    q = normal((cu_q[-1] + 2, heads, d), seed)
    k, v = (normal((cu_k[-1] + 2, kv, d), seed + i) for i in (1, 2))
    o = torch.full_like(q, 77.0)
    ptb_lib.swa_attention_packed(q, k, v, ints(cu_q), window, cu_seqlens_k=ints(cu_k) if lk else None, o=o)
    want, bound, written = X.packed(q, k, v, cu_q, cu_k, window, d ** -0.5)
    assert (o[~written] == 77).all()
    held_to(o[written], want[written], bound[written])


def test_packed_more_items_than_a_cta_holds(ptb_lib):
    """Sequences beyond those whose offsets the list kernel holds (1024), and more than 64 items a
    CTA, the later ones read from the list in global memory."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.RandomState(7)
    lens = list(rng.randint(0, 4, 1100))
    for b in (3, 500, 1023, 1024, 1050, 1098):
        lens[b] = 257 + b % 50  # two query blocks each
    heads = 66 * sms // sum(1 for n in lens if n) + 1
    assert heads * sum(-(-n // 256) for n in lens) > 64 * sms
    run_packed(ptb_lib, [int(n) for n in lens], None, heads, heads, 16, 100, 600)


def test_packed_more_items_than_a_cta_holds_grouped(ptb_lib):
    """The same with query blocks of two tokens and 128 heads to a kv head."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.RandomState(8)
    lens = [int(n) for n in rng.randint(1, 24, 1200)]
    assert sum(-(-n // 2) for n in lens) * 2 > 64 * sms
    run_packed(ptb_lib, lens, None, 256, 2, 32, 9, 610)


@pytest.mark.parametrize("window", [1 << 20, 66000, 50])
def test_packed_bands_of_more_tiles_than_classes(ptb_lib, window):
    """Bands that may have more than 1023 key tiles share classes in the list's order."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lq, lk = [2, 40, 0, 5, 3], [70000, 300, 10, 5, 20000]
    kv = sms // 5 + 1  # more items than SMs
    run_packed(ptb_lib, lq, lk, 2 * kv, kv, 32, window, 620)
