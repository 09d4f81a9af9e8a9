"""Windowed decode attention over a paged cache against float64 references."""
import math

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, on_device, queries, unseen_entries
from paged_ref import BHSD, DTYPES, VARLEN, Paged, token_view

pytestmark = pytest.mark.gpu
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.load()


def run(q, paged, Tq, window, sinks, cache=None, scale=None, ws=None, expect=0):
    """q [B * Tq, Hq, D]"""
    cache = on_device(paged) if cache is None else cache
    B, (_, Hq, D) = len(paged.lens), q.shape
    ws = da.alloc_paged_workspace(Tq, Hq, cache.Hkv, D) if ws is None else ws
    out = torch.full((B, Tq, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B, Tq, Hq), 7.0, device="cuda")
    da.decode_attn_paged_window(q.view(B, Tq, Hq, D).cuda(), cache, ints(paged.lens), paged.table.cuda(), out, ws, window=window,
                                sinks=sinks, scale=scale, lse=lse)
    assert da.decode_attn_splitkv_get_error(ws) == expect
    return out.view(-1, Hq, D), lse.view(-1, Hq)


def compare(lens, Tq, Hq, Hkv, D, kv, dtype, page, layout, window, sinks, seed=0, spread=0, scale=None):
    paged = Paged(lens, Hkv, D, kv, page, layout, seed=seed, scale_spread=spread)
    q = queries(len(lens) * Tq, Hq, D, dtype, seed + 1)
    want = chunk64(q, paged, [Tq] * len(lens), scale, window, sinks)
    out, lse = run(q, paged, Tq, window, sinks, scale=scale)
    assert check(out, lse, want, DTYPES[dtype]) is None
    return paged, q, out, lse


LENS = [1, 2, 63, 64, 65, 500, 127, 128, 129, 1111, 3000, 17, 256]
WINDOWS = [(1, 0), (1, 1), (3, 2), (64, 0), (65, 4), (127, 129), (128, 64), (200, 63), (1000, 1000), (4000, 1), (0x7FFFFFFF, 0), (5, 0x7FFFFFFF)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("Tq", [1, 4])
def test_windows(Tq, kv, dtype, window, sinks):
    compare(LENS, Tq, 4, 2, 128, kv, dtype, 16, VARLEN, window, sinks, seed=Tq, spread=2)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Tq", [(1, 1, 1), (7, 1, 1), (8, 1, 3), (28, 4, 5), (5, 5, 16), (20, 1, 2)])
def test_heads(Hq, Hkv, Tq, D, kv, dtype):
    compare([900, 2, 0, 77, 400], Tq, Hq, Hkv, D, kv, dtype, 64, BHSD, 150, 9, seed=Hq + Tq, spread=1)


@pytest.mark.parametrize("page", [16, 48, 80, 128, 256, 1024])
@pytest.mark.parametrize("kv,dtype", [("bf16", "bf16"), ("e4m3", "f16")])
def test_page_sizes(page, kv, dtype):
    compare([1, page, page + 1, 2500, 700], 2, 8, 2, 128, kv, dtype, page, VARLEN, 300, 33, seed=page, spread=2)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 4), (130, 17), (300, 260), (2000, 4)])
@pytest.mark.parametrize("Tq", [1, 3])
def test_pages_outside_the_window_are_not_read(Tq, window, sinks, kv, dtype):
    paged = Paged([900, 5000, 17, 2600], 2, 128, kv, 32, VARLEN, seed=3)
    q = queries(4 * Tq, 8, 128, dtype, 4)
    want = chunk64(q, paged, [Tq] * 4, None, window, sinks)
    assert unseen_entries(paged, [Tq] * 4, window, sinks)
    out, lse = run(q, paged, Tq, window, sinks)
    assert check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_a_window_over_all_keys_is_plain_attention(kv, dtype):
    paged, q, out, lse = compare([700, 4000, 1], 2, 8, 2, 64, kv, dtype, 64, BHSD, 4000, 0, seed=5)
    ws = da.alloc_paged_workspace(2, 8, 2, 64)
    o, l = torch.empty(3, 2, 8, 64, dtype=q.dtype, device="cuda"), torch.empty(3, 2, 8, device="cuda")
    da.decode_attn_paged(q.view(3, 2, 8, 64).cuda(), on_device(paged), ints(paged.lens), paged.table.cuda(), o, ws, lse=l)
    assert torch.equal(o.view_as(out), out) and torch.equal(l.view_as(lse), lse)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite_reach_the_tokens_that_see_them(bad, kv, dtype):
    if kv == "e4m3" and math.isinf(bad):
        pytest.skip("no infinity in e4m3")
    Tq, window, sinks = 4, 100, 20
    q = queries(Tq, 4, 64, dtype, 7)
    # below the window, at each token's edge of it, among the sinks and behind them, at the newest tokens
    for spot in (3, 19, 20, 300, 596, 597, 598, 599, 600, 601, 690, 697, 698, 699):
        paged = Paged([700], 2, 64, kv, 16, VARLEN, seed=6)
        token_view(paged.v, VARLEN)[int(paged.table[0, spot // 16]), spot % 16, 1, 9] = bad
        want = chunk64(q, paged, [Tq], None, window, sinks)
        out, lse = run(q, paged, Tq, window, sinks)
        assert check(out, lse, want, DTYPES[dtype]) is None, spot


def test_many_sequences_and_a_long_one():
    compare([i % 350 for i in range(1024)], 1, 4, 1, 64, "f16", "f16", 16, VARLEN, 60, 5, seed=8)
    compare([60000, 1, 30000], 1, 8, 2, 128, "bf16", "bf16", 64, BHSD, 20000, 3000, seed=9)


def test_bad_lengths_and_pages():
    paged = Paged([700, 300], 2, 64, "f16", 16, VARLEN, seed=10)
    q = queries(2, 4, 64, "f16", 11)
    out, lse = run(q, paged, 1, 50, 4)
    good = list(paged.lens)
    paged.lens = [700, 1 << 20]
    got, got_l = run(q, paged, 1, 50, 4, expect=da.DA_DEVERR_SEQLENS)
    assert torch.equal(got[0], out[0]) and (got[1] == 0).all() and torch.isneginf(got_l[1]).all()
    paged.lens = good
    paged.table[0, 699 // 16] = -1
    run(q, paged, 1, 50, 4, expect=da.DA_DEVERR_PAGE)


def test_graph_and_chunk_agree():
    paged, q, out, lse = compare([3000, 70], 1, 8, 2, 128, "bf16", "bf16", 64, BHSD, 500, 4, seed=12)
    cache, ws = on_device(paged), da.alloc_paged_workspace(1, 8, 2, 128)
    qd, lens, table = q.cuda(), ints(paged.lens), paged.table.cuda()
    o = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_paged_window(qd, cache, lens, table, o, ws, window=500, sinks=4)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out)
