"""Chunk and windowed attention and the page operators where their arithmetic, their sizes or what they share could go wrong."""
import math

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, on_device, queries, run_chunk
from paged_ref import DTYPES, VARLEN, Paged

pytestmark = pytest.mark.gpu
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.load()


def run_window(q, paged, Tq, window, sinks, expect=0):
    """q [B * Tq, Hq, D]"""
    cache, B, (_, Hq, D) = on_device(paged), len(paged.lens), q.shape
    ws = da.alloc_paged_workspace(Tq, Hq, cache.Hkv, D)
    out, lse = torch.full((B, Tq, Hq, D), 7.0, dtype=q.dtype, device="cuda"), torch.full((B, Tq, Hq), 7.0, device="cuda")
    da.decode_attn_paged_window(q.view(B, Tq, Hq, D).cuda(), cache, ints(paged.lens), paged.table.cuda(), out, ws, window=window,
                                sinks=sinks, lse=lse)
    assert da.decode_attn_splitkv_get_error(ws) == expect
    return out.view(-1, Hq, D), lse.view(-1, Hq)


# ------------------------------------------------------------ values that count for nothing
# of the pages without a value scale, or out of the cache: the first key, and the first one behind them
SPANS = [(128, 256), (512, 640), (400, 416), (0, 512), (256, 720)]


def zero_scales(span, D, G, seed):
    lens, new = [720, 300], [310, 300]
    paged = Paged(lens, 1, D, "e4m3", 16, VARLEN, seed=seed, scale_spread=2)
    for b, n in enumerate(lens):
        for i in range(-(-n // 16)):
            if span[0] <= 16 * i < span[1]:
                paged.v_scale[int(paged.table[b, i])] = 0.0
    return paged, new


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 4), (128, 1), (128, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 3), (100, 0), (130, 0), (130, 1)])
def test_chunk_zero_value_scales_behind_a_window(window, sinks, D, G, dtype):
    """Rows that see nothing of a piece's first tile, and no value of the second that counts."""
    for span in SPANS:
        paged, new = zero_scales(span, D, G, 90)
        q = queries(sum(new), G, D, dtype, 91)
        want = chunk64(q, paged, new, None, window, sinks)
        assert torch.isfinite(want[0]).all()
        out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
        assert check(out, lse, want, DTYPES[dtype]) is None, span


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Tq,G", [(1, 1), (4, 1), (16, 1), (4, 7)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (70, 0), (70, 3), (200, 0)])
def test_window_zero_value_scales(window, sinks, Tq, G, dtype):
    for D in (64, 128):
        for span in [(400, 704), (640, 704), (704, 720), (0, 720)]:
            paged, _ = zero_scales(span, D, G, 92)
            q = queries(2 * Tq, G, D, dtype, 93)
            want = chunk64(q, paged, [Tq, Tq], None, window, sinks)
            out, lse = run_window(q, paged, Tq, window, sinks)
            assert check(out, lse, want, DTYPES[dtype]) is None, (D, span)


def gone_pages(span, kv, D, seed):
    """(pages with entries outside the cache, the same with pages of zeros there)"""
    bad, zero = (Paged([720, 300], 1, D, kv, 16, VARLEN, seed=seed, scale_spread=2) for _ in range(2))
    for b, n in enumerate(bad.lens):
        for i in range(-(-n // 16)):
            if span[0] <= 16 * i < span[1]:
                for x in (zero.k, zero.v):
                    x.view(torch.uint8)[int(bad.table[b, i])] = 0
                bad.table[b, i] = -1 if i % 2 else len(bad.k)
    return bad, zero


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 3), (130, 0)])
def test_entries_outside_the_cache_behind_a_window(window, sinks, D, G, kv, dtype):
    for span in SPANS:
        bad, zero = gone_pages(span, kv, D, 94)
        new = [310, 300]
        q = queries(sum(new), G, D, dtype, 95)
        want = chunk64(q, zero, new, None, window, sinks)
        out, lse = run_chunk(q, bad, new, window=window, sinks=sinks, expect=da.DA_DEVERR_PAGE)
        assert check(out, lse, want, DTYPES[dtype]) is None, span
    bad, zero = gone_pages((640, 704), kv, D, 96)
    bad.lens[1] = zero.lens[1] = 0
    q = queries(8, G, D, dtype, 97)
    want = chunk64(q, zero, [4, 4], None, 70, sinks)
    out, lse = run_window(q, bad, 4, 70, sinks, expect=da.DA_DEVERR_PAGE)
    assert check(out, lse, want, DTYPES[dtype]) is None


# ------------------------------------------------------------ sizes
def test_a_length_that_cannot_be_and_the_widest_window():
    """Many rows of a sequence that counts as empty lie far below position 0."""
    paged = Paged([2000, 3], 1, 64, "f16", 16, VARLEN, seed=98)
    new = [1500, 3]
    q = queries(1503, 2, 64, "f16", 99)
    for sinks in (0, 0x7FFFFFFF):
        out, lse = run_chunk(q, paged, new, window=0x7FFFFFFF, sinks=sinks, lens=[1 << 30, 3], expect=da.DA_DEVERR_SEQLENS)
        assert (out[:1500] == 0).all() and torch.isneginf(lse[:1500]).all()
        want = chunk64(q, paged, new)
        assert check(out[1500:], lse[1500:], tuple(x[1500:] for x in want), torch.float16) is None


@pytest.mark.parametrize("page", [304, 976, 16])
def test_free_pages_of_a_sequence_as_long_as_can_be(page):
    """Length and page size add up to more than 32 bits hold."""
    num_pages = 0x7FFFFF00 // page
    table = torch.arange(num_pages, dtype=torch.int32, device="cuda").flip(0).view(1, -1)
    ws = da.alloc_paged_pages_workspace(num_pages)
    free, count = torch.full((num_pages,), -9, dtype=torch.int32, device="cuda"), ints([-1])
    for length, left in ((num_pages * page, 0), (num_pages * page - page + 1, 0), (num_pages * page - 3 * page, 3)):
        free.fill_(-9)
        da.decode_attn_paged_free_pages(ints([length]), table, free, count, ws, page_size=page)
        assert da.decode_attn_splitkv_get_error(ws) == 0
        assert count.item() == left
        assert free[:left].tolist() == list(range(left)) and (free[left:] == -9).all()


# ------------------------------------------------------------ pages
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_fork_of_a_row_whose_last_entry_is_outside_the_cache(kv):
    """There is nothing to copy: the entry stays what it is, and the new page is not taken into use as it lies."""
    paged = Paged([40, 37], 2, 64, kv, 16, VARLEN, seed=30, extra_pages=4)
    cache = on_device(paged)
    n = cache.num_pages
    unused = [i for i in range(n) if i not in set(paged.table.flatten().tolist())][:2]
    table = paged.table.clone()
    table[0, 2], before = n + 5, [x.view(torch.uint8).clone() for x in (cache.k, cache.v)]
    lens, out, ws = ints([0, 0]), torch.full((2, 3), -9, dtype=torch.int32, device="cuda"), da.alloc_paged_pages_workspace(n)
    da.decode_attn_paged_fork(cache, ints(paged.lens), table.cuda(), ints([0, 1]), ints(unused), lens, out, ws)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_PAGE
    assert lens.tolist() == paged.lens
    assert out.tolist() == [table[0].tolist(), [*table[1, :2].tolist(), unused[1]]]
    after = [x.view(torch.uint8) for x in (cache.k, cache.v)]
    for x, y in zip(before, after):
        x[unused[1], :5] = x[int(table[1, 2]), :5]
        assert torch.equal(x, y)


# ------------------------------------------------------------ refusals of the binding
def test_windows_and_sinks_are_whole_numbers():
    import numpy as np
    paged = Paged([100], 1, 64, "f16", 16, VARLEN, seed=31)
    q = queries(3, 2, 64, "f16", 32)
    for bad in (True, 1.5, "4", 1 << 31, math.nan):
        with pytest.raises(ValueError):
            run_chunk(q, paged, [3], window=bad)
        with pytest.raises(ValueError):
            run_chunk(q, paged, [3], window=5, sinks=bad)
        with pytest.raises(ValueError):
            run_window(q, paged, 3, bad, 0)
    want = chunk64(q, paged, [3], None, 5, 2)
    for out, lse in (run_chunk(q, paged, [3], window=np.int64(5), sinks=np.int32(2)), run_window(q, paged, 3, np.int64(5), np.int32(2))):
        assert check(out, lse, want, torch.float16) is None


def test_tensors_without_a_dimension_are_refused():
    paged = Paged([100], 1, 64, "f16", 16, VARLEN, seed=33)
    cache, ws = on_device(paged), da.alloc_paged_pages_workspace(len(paged.k))
    lens, table, one = ints([100]), paged.table.cuda(), ints(1)
    with pytest.raises(ValueError):
        da.decode_attn_paged_fork(cache, lens, table, one, ints([-1]), ints([0]), table.clone(), ws)
    with pytest.raises(ValueError):
        da.decode_attn_paged_free_pages(lens, table, one, ints([0]), ws, page_size=16)
    with pytest.raises(ValueError):
        da.decode_attn_paged_append(None, cache.k.flatten()[0], cache.v.flatten()[0], cache, ints([0, 1]), lens, table, ws)
