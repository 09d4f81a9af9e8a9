"""Chunk and windowed attention and the page operators where their arithmetic, their sizes or what they share could go wrong."""
import math

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, on_device, queries, run_chunk, starts
from paged_ref import BHSD, DTYPES, VARLEN, Paged

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


# ------------------------------------------------------------ long calls
@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D,window", [(128, 0), (64, 0), (128, 3000), (64, 3000)])
def test_long_calls_against_the_definition(D, window, kv, dtype):
    """Every block walks through many key tiles: rows at the edges of items, each over its whole history."""
    g = torch.Generator().manual_seed(51)
    lens, new, pages = [16384, 5000], [2048, 700], 400
    shape = (pages, 8, 64, D)
    k, v = (torch.randn(shape, generator=g).to(DTYPES[kv]) for _ in range(2))
    scales = [torch.exp2(torch.randint(-3, 3, (pages, 8), generator=g).float()) for _ in range(2)] if kv == "e4m3" else [None, None]
    order = torch.randperm(pages, generator=g).to(torch.int32)[:358]
    table = torch.stack([order[:256], torch.cat([order[256:], order.new_zeros(154)])])
    q = torch.randn(2748, 32, D, generator=g).to(DTYPES[dtype])
    cache = da.PagedCache(k.cuda(), v.cuda(), *(s if s is None else s.cuda() for s in scales), layout=BHSD)
    ws = da.alloc_paged_chunk_workspace(32, 8, D)
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(2748, 32, device="cuda")
    da.decode_attn_paged_chunk(q.cuda(), cache, ints(starts(new)), ints(lens), table.cuda(), out, ws, window=window, sinks=5, lse=lse)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    # (sequence, new token): of items of 64 tokens
    picked = [(0, 0), (0, 63), (0, 64), (0, 1055), (0, 2047), (1, 0), (1, 351), (1, 699)]
    rows = [t + (2048 if b else 0) for b, t in picked]
    heads = [0, 1, 2, 3, 28, 29, 30, 31]
    some = object.__new__(Paged)       # two of the KV heads
    some.Hkv, some.D, some.kv, some.page, some.layout = 2, D, kv, 64, BHSD
    raw = lambda x: x.view(torch.uint8 if kv == "e4m3" else torch.int16)[:, [0, 7]].contiguous().view(x.dtype)
    some.k, some.v = raw(k), raw(v)
    some.k_scale, some.v_scale = (s if s is None else s[:, [0, 7]] for s in scales)
    some.table = table[[b for b, _ in picked]]
    some.lens = [lens[b] - new[b] + t + 1 for b, t in picked]
    want = chunk64(q[rows][:, heads], some, [1] * len(picked), None, window, 5)
    assert check(out[rows][:, heads], lse[rows][:, heads], want, DTYPES[dtype]) is None


# ------------------------------------------------------------ together
def test_a_window_of_single_tokens_by_either_call():
    paged = Paged([3000, 70, 1], 2, 128, "bf16", 64, BHSD, seed=12)
    q = queries(3, 8, 128, "bf16", 13)
    want = chunk64(q, paged, [1, 1, 1], None, 500, 4)
    for out, lse in (run_chunk(q, paged, [1, 1, 1], window=500, sinks=4), run_window(q, paged, 1, 500, 4)):
        assert check(out, lse, want, torch.bfloat16) is None


@pytest.mark.parametrize("D", [64, 128])
def test_decode_steps_beside_chunks(D):
    """A chunk call and windowed decode steps over the same pages, on two streams."""
    paged = Paged([900, 64, 10, 2000], 2, D, "bf16", 16, VARLEN, seed=60)
    new = [300, 64, 0, 1]
    q, dq = queries(sum(new), 8, D, "bf16", 62), queries(4, 8, D, "bf16", 70)
    want, dwant = chunk64(q, paged, new), chunk64(dq, paged, [1] * 4, None, 100, 4)
    cache, table, lens, cu = on_device(paged), paged.table.cuda(), ints(paged.lens), ints(starts(new))
    ws, dec = da.alloc_paged_chunk_workspace(8, 2, D), da.alloc_paged_workspace(1, 8, 2, D)
    qd, dqd = q.cuda(), dq.cuda()
    out, lse, dout, dlse = torch.empty_like(qd), torch.empty(len(q), 8, device="cuda"), torch.empty_like(dqd), torch.empty(4, 8, device="cuda")
    one, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        da.decode_attn_paged_chunk(qd, cache, cu, lens, table, out, ws, lse=lse, stream=one)
        da.decode_attn_paged_window(dqd, cache, lens, table, dout, dec, window=100, sinks=4, lse=dlse, stream=other)
    torch.cuda.synchronize()
    assert da.decode_attn_splitkv_get_error(ws) == 0 and da.decode_attn_splitkv_get_error(dec) == 0
    assert check(out, lse, want, torch.bfloat16) is None and check(dout, dlse, dwant, torch.bfloat16) is None


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_one_workspace_for_attention_append_and_pages(kv):
    """Every call of the paged cache in turn on one workspace, nothing waited for in between."""
    Hq, Hkv, D, P, Tq = 8, 2, 128, 16, 4
    paged = Paged([6005, 900, 33], Hkv, D, kv, P, VARLEN, seed=21, extra_pages=60)
    cache, B = on_device(paged), 3
    n = cache.num_pages
    size = max(da.paged_workspace_size(Tq, Hq, Hkv, D), da.paged_chunk_workspace_size(Hq, Hkv, D), da.paged_pages_workspace_size(n))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xA5)
    assert da.load().decode_attn_paged_workspace_init(ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == 0
    q = queries(B * Tq, Hq, D, "f16", 22).cuda()
    want, windowed = chunk64(q.cpu(), paged, [Tq] * B), chunk64(q.cpu(), paged, [Tq] * B, None, 700, 20)
    lens, cu = ints(paged.lens), ints(starts([Tq] * B))
    width = paged.table.shape[1] + 2
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    table[:, :width - 2] = paged.table.cuda()
    used = sum(-(-m // P) for m in paged.lens)
    # the last token's own key and value, appended again (16-bit pages; into 8-bit ones a page that no row uses)
    rows = [paged.sequence(b) for b in range(B)]
    newest = [torch.stack([r[i][-1] for r in rows]).half().cuda() for i in range(2)]
    free, count, moved = torch.empty(n, dtype=torch.int32, device="cuda"), ints([0]), ints([0])
    parents, fresh = ints([0, 1, 2]), ints([0] * B)
    got, results = {}, []
    for turn in range(4):
        table2, table3, lens2 = torch.zeros_like(table), torch.zeros_like(table), torch.zeros_like(lens)
        for name in ("chunk", "window", "decode"):
            got[name] = (torch.full_like(q, 7.0), torch.full((B * Tq, Hq), 7.0, device="cuda"))
        o, l = got["chunk"]
        da.decode_attn_paged_chunk(q, cache, cu, lens, table, o, ws, lse=l)
        da.decode_attn_paged_free_pages(lens, table, free, count, ws, page_size=P)
        o, l = got["decode"]
        da.decode_attn_paged(q.view(B, Tq, Hq, D), cache, lens, table, o.view(B, Tq, Hq, D), ws, lse=l.view(B, Tq, Hq))
        fresh.copy_(free[:B])
        da.decode_attn_paged_fork(cache, lens, table, parents, fresh, lens2, table2, ws)
        if kv == "f16":
            da.decode_attn_paged_append(None, *newest, cache, ints(list(range(B + 1))), lens2, table2, ws)
        else:
            da.decode_attn_paged_append(None, *newest, cache, ints(list(range(B + 1))), ints([1] * B), free[B:2 * B].view(B, 1), ws)
        o, l = got["window"]
        da.decode_attn_paged_window(q.view(B, Tq, Hq, D), cache, lens2, table2, o.view(B, Tq, Hq, D), ws, window=700, sinks=20,
                                    lse=l.view(B, Tq, Hq))
        da.decode_attn_paged_compact(cache, lens2, table2, table3, moved, ws)
        results.append({k: (a.clone(), b.clone()) for k, (a, b) in got.items()} | dict(
            free=free[:n - used].clone(), count=count.clone(), moved=moved.clone(), before=table, after=table3, lens=lens2))
        table, lens = table3, lens2
    assert da.decode_attn_splitkv_get_error(ws) == 0
    need = [-(-m // P) for m in paged.lens]
    for r in results:
        for name, ref in (("chunk", want), ("decode", want), ("window", windowed)):
            assert check(*r[name], ref, torch.float16) is None, name
        in_use = {x for row, m in zip(r["before"].tolist(), need) for x in row[:m]}
        assert r["free"].tolist() == [x for x in range(n) if x not in in_use] and r["count"].item() == n - used
        assert r["moved"].item() == used and r["lens"].tolist() == paged.lens
        assert sorted(x for row, m in zip(r["after"].tolist(), need) for x in row[:m]) == list(range(used))


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
