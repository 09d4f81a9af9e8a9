"""Attention of chunks of new tokens over a paged cache against float64 references."""
import math

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, on_device, queries, run_chunk, starts, unseen_entries
from paged_ref import BHSD, DTYPES, VARLEN, Paged, token_view

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.load()


def compare(lens, new, Hq, Hkv, D, kv, dtype, page, layout, window=0, sinks=0, scale=None, seed=0, spread=0, mean=0.0, q_mean=0.0):
    paged = Paged(lens, Hkv, D, kv, page, layout, seed=seed, scale_spread=spread, mean=mean)
    q = queries(sum(new), Hq, D, dtype, seed + 1, q_mean)
    want = chunk64(q, paged, new, scale, window, sinks)
    out, lse = run_chunk(q, paged, new, scale=scale, window=window, sinks=sinks)
    assert check(out, lse, want, DTYPES[dtype]) is None
    return paged, q, out, lse


TYPES = [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]
LENGTHS = {
    "one_token": ([1], [1]),
    "one_of_many": ([300], [1]),
    "whole_prompt": ([200], [200]),
    "part": ([777], [130]),
    "mixed": ([129, 0, 1, 500, 64, 127, 16], [129, 0, 1, 1, 0, 33, 16]),
    "tile_edges": ([128, 256, 384, 255, 257], [64, 65, 63, 255, 1]),
    "no_history": ([5, 3, 40], [9, 3, 50]),
    "several_tiles": ([1500, 1029], [700, 1029]),
}


@pytest.mark.parametrize("layout", [VARLEN, BHSD])
@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths(lengths, kv, dtype, layout):
    lens, new = LENGTHS[lengths]
    page = {VARLEN: 16, BHSD: 64}[layout]
    compare(lens, new, 4, 2, 128, kv, dtype, page, layout, seed=len(lengths), spread=3)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (14, 2), (8, 1), (24, 1), (130, 1), (300, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(Hq, Hkv, D, kv, dtype):
    compare([203, 40], [37, 20], Hq, Hkv, D, kv, dtype, 32, VARLEN, seed=Hq, spread=1)


@pytest.mark.parametrize("kv,dtype", [("bf16", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("page", [16, 48, 80, 96, 128, 256, 1024])
@pytest.mark.parametrize("layout", [VARLEN, BHSD])
def test_page_sizes(page, layout, kv, dtype):
    compare([1, page - 1, page, page + 1, 700], [1, 5, 16, 17, 300], 4, 1, 64, kv, dtype, page, layout, seed=page, spread=2)


WINDOWS = [(1, 0), (1, 1), (2, 5), (16, 0), (100, 4), (128, 128), (129, 130), (333, 200), (5000, 7), (0x7FFFFFFF, 0), (40, 0x7FFFFFFF)]


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, kv, dtype):
    lens, new = [900, 3, 1300, 131, 64], [300, 3, 1, 131, 70]
    compare(lens, new, 4, 2, 64, kv, dtype, 16, BHSD, window, sinks, seed=window % 97, spread=2)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 4), (130, 17), (300, 260)])
def test_pages_outside_the_window_are_not_read(window, sinks, kv, dtype):
    paged = Paged([900, 2000, 17], 2, 128, kv, 32, VARLEN, seed=3)
    new = [60, 1, 17]
    q = queries(sum(new), 8, 128, dtype, 4)
    want = chunk64(q, paged, new, None, window, sinks)
    assert unseen_entries(paged, new, window, sinks)
    out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
    assert check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-6, 4.0, 1e-30])
@pytest.mark.parametrize("kv,dtype", TYPES)
def test_scales(scale, kv, dtype):
    compare([260, 30], [140, 30], 4, 1, 64, kv, dtype, 16, VARLEN, scale=scale, seed=5)


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_scale_zero_keeps_what_is_not_finite(kv, dtype):
    """0 times a score that is not a number is none."""
    paged = Paged([200], 1, 64, kv, 16, VARLEN, seed=40)
    q = queries(200, 2, 64, dtype, 41)
    q[7, 1, 3], q[100, 0, 5] = math.nan, math.inf
    want = chunk64(q, paged, [200], 0.0)
    out, lse = run_chunk(q, paged, [200], scale=0.0)
    bad = torch.zeros(200, 2, dtype=torch.bool)
    bad[7, 1] = bad[100, 0] = True
    assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    good = tuple(x[:, 0][~bad[:, 0]] for x in want)
    assert check(out[:, 0].cpu()[~bad[:, 0]], lse[:, 0].cpu()[~bad[:, 0]], good, DTYPES[dtype]) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_growing_scores(kv, dtype):
    """Every key's score above the last one's by more than any headroom, and one far above the rest."""
    paged = Paged([700], 1, 64, kv, 16, VARLEN, seed=6)
    ramp = (torch.arange(700).float() / 4 + 1) if kv != "e4m3" else torch.exp2(torch.arange(700).float() / 80 - 3)
    for p in range(700):
        paged.k[int(paged.table[0, p // 16]), p % 16] = (ramp[p] * torch.ones(64)).to(paged.k.dtype)
    new = [150]
    q = torch.full((150, 2, 64), 0.5).to(DTYPES[dtype])
    q[:, 1] *= -1
    want = chunk64(q, paged, new, 1.0)
    out, lse = run_chunk(q, paged, new, scale=1.0)
    assert check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("kv,dtype", [("e4m3", "f16"), ("e4m3", "bf16")])
def test_unequal_page_scales(kv, dtype):
    compare([1000, 400], [333, 400], 4, 1, 128, kv, dtype, 16, BHSD, seed=8, spread=12)
    compare([1000, 400], [333, 400], 4, 1, 64, kv, dtype, 48, VARLEN, seed=9, spread=20, window=100, sinks=3, scale=1e-3)


def test_zero_scales_and_tiny_scales():
    paged = Paged([400], 1, 64, "e4m3", 16, VARLEN, seed=10)
    for i in range(25):
        if i % 3 == 0:
            paged.k_scale[int(paged.table[0, i])] = 0.0
        if i % 3 == 1:
            paged.v_scale[int(paged.table[0, i])] = 0.0 if i % 2 else 2.0 ** -100
    new = [200]
    q = queries(200, 4, 64, "f16", 11)
    want = chunk64(q, paged, new)
    out, lse = run_chunk(q, paged, new)
    assert check(out, lse, want, torch.float16) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(bad, window, sinks, kv, dtype):
    if kv == "e4m3" and not math.isnan(bad):
        pytest.skip("no infinity in e4m3")
    paged = Paged([700, 90], 2, 64, kv, 16, VARLEN, seed=12)
    new = [300, 90]
    q = queries(390, 4, 64, dtype, 13)
    spots = [(0, 5, 3), (0, 19, 0), (0, 20, 63), (0, 350, 7), (0, 420, 9), (0, 555, 1), (0, 698, 30), (0, 699, 31), (1, 40, 2)]
    for b, p, d in spots:
        page = int(paged.table[b, p // 16])
        token_view(paged.v, VARLEN)[page, p % 16, 1, d] = bad
    want = chunk64(q, paged, new, None, window, sinks)
    assert torch.isfinite(want[0][:, :2]).all() and not torch.isfinite(want[0][:, 2:]).all()
    out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
    assert check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_values_that_are_not_finite_among_many_first_tokens(kv, dtype):
    """Whole tiles of first tokens, seen by all rows, beside those that the window cuts."""
    paged = Paged([4000], 1, 128, kv, 64, BHSD, seed=42)
    new, window, sinks = [300], 500, 1500
    q = queries(300, 2, 128, dtype, 43)
    for p, d in ((100, 1), (1407, 2), (1408, 3), (1499, 4), (1500, 5), (3300, 6), (3999, 7)):
        token_view(paged.v, BHSD)[int(paged.table[0, p // 64]), p % 64, 0, d] = math.nan
    want = chunk64(q, paged, new, None, window, sinks)
    out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
    assert torch.isnan(want[0][:, :, 1:5]).all() and torch.isfinite(want[0][:, :, 5]).all()
    assert check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_keys_and_queries_that_are_not_finite(kv, dtype):
    paged = Paged([500], 2, 64, kv, 16, VARLEN, seed=14)
    for p in (300, 420):
        paged.k[int(paged.table[0, p // 16]), p % 16, 0, 5] = math.nan
    new = [200]
    q = queries(200, 4, 64, dtype, 15)
    q[150, 2] = math.nan
    want = chunk64(q, paged, new)
    out, lse = run_chunk(q, paged, new)
    assert torch.isnan(out[:, :2]).all() and torch.isnan(lse[:, :2]).all()          # key 300 is seen by all of them
    assert torch.isnan(out[150, 2]).all() and torch.isfinite(out[150, 3]).all()
    keep = torch.ones(200, 4, dtype=torch.bool)
    keep[:, :2] = False
    keep[150, 2] = False
    assert check(out[:, 3:], lse[:, 3:], tuple(x[:, 3:] for x in want), DTYPES[dtype]) is None
    assert torch.isfinite(out.cpu()[keep]).all()
    # seen by some: only the later key is not finite
    paged.k[int(paged.table[0, 300 // 16]), 300 % 16, 0, 5] = 1.0
    want = chunk64(q, paged, new)
    out, lse = run_chunk(q, paged, new)
    assert torch.isfinite(out[:120, :2]).all() and torch.isnan(out[120:, :2]).all()
    assert check(out[:120, :2], lse[:120, :2], tuple(x[:120, :2] for x in want), DTYPES[dtype]) is None


def test_strided_rows_in_and_out():
    paged = Paged([333, 90], 2, 128, "bf16", 16, VARLEN, seed=16)
    new = [100, 90]
    q = queries(190, 4, 128, "bf16", 17)
    want = chunk64(q, paged, new)
    cache, ws = on_device(paged), da.alloc_paged_chunk_workspace(4, 2, 128)
    qkv = torch.full((190, 4 + 2 + 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :4] = q.cuda()
    wide = torch.full((190, 6, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(190, 4, device="cuda")
    da.decode_attn_paged_chunk(qkv[:, :4], cache, ints(starts(new)), ints(paged.lens), paged.table.cuda(), wide[:, 1:5], ws, lse=lse)
    assert check(wide[:, 1:5], lse, want, torch.bfloat16) is None
    assert (wide[:, 0] == 3.0).all() and (wide[:, 5] == 3.0).all()
    out = torch.empty(190, 4, 128, dtype=torch.bfloat16, device="cuda")
    da.decode_attn_paged_chunk(qkv[:, :4], cache, ints(starts(new)), ints(paged.lens), paged.table.cuda(), out, ws)   # without lse
    assert torch.equal(out, wide[:, 1:5])


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_bad_sequences_and_pages(kv, dtype):
    """What cannot be is flagged, and the other sequences keep their results to the bit."""
    new = [30, 40, 50, 7]
    paged = Paged([100, 200, 150, 7], 2, 64, kv, 16, VARLEN, seed=18)
    q = queries(127, 4, 64, dtype, 19)
    out, lse = run_chunk(q, paged, new)
    lens = [100, 100000, 150, -1]
    got, got_l = run_chunk(q, paged, new, lens=lens, expect=da.DA_DEVERR_SEQLENS)
    for lo, hi in ((0, 30), (70, 120)):
        assert torch.equal(got[lo:hi], out[lo:hi]) and torch.equal(got_l[lo:hi], lse[lo:hi])
    for lo, hi in ((30, 70), (120, 127)):
        assert (got[lo:hi] == 0).all() and torch.isneginf(got_l[lo:hi]).all()
    # rows that cannot be: the sequences around them count, theirs are left alone
    cache, ws = on_device(paged), da.alloc_paged_chunk_workspace(4, 2, 64)
    qd, o, l = q.cuda(), torch.full((127, 4, 64), 7.0, dtype=q.dtype, device="cuda"), torch.full((127, 4), 7.0, device="cuda")
    da.decode_attn_paged_chunk(qd, cache, ints([0, 30, 70, 120, 128]), ints(paged.lens), paged.table.cuda(), o, ws, lse=l)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_SEQLENS
    assert torch.equal(o[:120], out[:120]) and (o[120:] == 7.0).all() and (l[120:] == 7.0).all()
    # entries outside the cache: zeros
    table = paged.table.clone()
    at = int(table[1, 3])
    table[1, 3] = cache.num_pages
    table[2, 1] = -1
    zero = Paged([100, 200, 150, 7], 2, 64, kv, 16, VARLEN, seed=18)
    for x in (zero.k, zero.v):
        x.view(torch.uint8)[at] = 0
        x.view(torch.uint8)[int(paged.table[2, 1])] = 0
    want = chunk64(q, zero, new)
    da.decode_attn_paged_chunk(qd, cache, ints(starts(new)), ints(paged.lens), table.cuda(), o, ws, lse=l)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_PAGE
    assert check(o, l, want, DTYPES[dtype]) is None


def test_same_bits_again_and_on_another_stream_and_in_a_graph():
    paged, q, out, lse = compare([3000, 700, 1], [500, 700, 1], 8, 2, 128, "bf16", "bf16", 64, BHSD, seed=20)
    cache, ws = on_device(paged), da.alloc_paged_chunk_workspace(8, 2, 128)
    args = (q.cuda(), cache, ints(starts([500, 700, 1])), ints(paged.lens), paged.table.cuda())
    o, l = torch.empty_like(args[0]), torch.empty(1201, 8, device="cuda")
    for _ in range(5):
        da.decode_attn_paged_chunk(*args, o, ws, lse=l)
        assert torch.equal(o, out) and torch.equal(l, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    da.decode_attn_paged_chunk(*args, o, ws, lse=l, stream=side)
    side.synchronize()
    assert torch.equal(o, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_paged_chunk(*args, o, ws, lse=l)
        da.decode_attn_paged_chunk(*args, o, ws, lse=l)
    for _ in range(3):
        o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    # other lengths in the same buffers: the graph reads them anew
    args[3].copy_(ints([2500, 700, 0]))
    graph.replay()
    torch.cuda.synchronize()
    paged.lens = [2500, 700, 0]
    want = chunk64(q, paged, [500, 700, 1])
    assert check(o, l, want, torch.bfloat16) is None


def test_one_workspace_serves_every_call():
    """Chunk, decode and append share a workspace in stream order."""
    paged = Paged([900, 300], 2, 128, "f16", 16, VARLEN, seed=21)
    cache = on_device(paged)
    ws = da.alloc_paged_chunk_workspace(8, 2, 128)
    if ws.numel() < da.paged_workspace_size(4, 8, 2, 128):
        ws = da.alloc_paged_workspace(4, 8, 2, 128)
        if ws.numel() < da.paged_chunk_workspace_size(8, 2, 128):
            pytest.fail("one of the two is the larger")
    q = queries(8, 8, 128, "f16", 22)
    want = chunk64(q, paged, [4, 4])
    table, lens = paged.table.cuda(), ints(paged.lens)
    for _ in range(3):
        out, lse = run_chunk(q, paged, [4, 4], cache=cache, workspace=ws)
        assert check(out, lse, want, torch.float16) is None
        o, l = torch.empty(2, 4, 8, 128, dtype=torch.float16, device="cuda"), torch.empty(2, 4, 8, device="cuda")
        da.decode_attn_paged(q.view(2, 4, 8, 128).cuda(), cache, lens, table, o, ws, lse=l)
        assert check(o.view(8, 8, 128), l.view(8, 8), want, torch.float16) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
def test_many_sequences(kv, dtype):
    g = torch.Generator().manual_seed(23)
    lens = torch.randint(0, 90, (1024,), generator=g).tolist()
    new = [min(n, m) for n, m in zip(lens, torch.randint(0, 6, (1024,), generator=g).tolist())]
    new[500], lens[500] = 80, 80
    compare(lens, new, 2, 1, 64, kv, dtype, 16, VARLEN, seed=24)


def test_no_rows():
    paged = Paged([100], 1, 64, "f16", 16, VARLEN, seed=25)
    cache, ws = on_device(paged), da.alloc_paged_chunk_workspace(2, 1, 64)
    empty = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    da.decode_attn_paged_chunk(empty, cache, ints([0, 0]), ints([100]), paged.table.cuda(), empty.clone(), ws)
    run_chunk(queries(0, 2, 64, "f16"), paged, [0], cache=cache)


def test_prompt_in_parts_equals_the_prompt_at_once():
    """Append and attend part by part, as a server does it; against the whole prompt in one call."""
    Hq, Hkv, D, P, T = 8, 2, 128, 16, 700
    g = torch.Generator().manual_seed(26)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    angle = torch.arange(T, dtype=torch.float64)[:, None] * torch.pow(10000.0, -torch.arange(64, dtype=torch.float64) / 64)[None]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    cache = da.PagedCache.empty(50, P, Hkv, D, torch.bfloat16)
    table = torch.randperm(50, generator=g)[:44].to(torch.int32).view(1, 44).cuda()
    ws = da.alloc_paged_chunk_workspace(Hq, Hkv, D)
    out, rotated = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    done = 0
    for part in (1, 255, 300, 144):
        rows = slice(done, done + part)
        done += part
        da.decode_attn_paged_append(q[rows], k[rows], v[rows], cache, ints([0, part]), ints([done]), table, ws, cos_sin=cos_sin,
                                    q_out=rotated[rows])
        da.decode_attn_paged_chunk(rotated[rows], cache, ints([0, part]), ints([done]), table, out[rows], ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    paged = Paged([T], Hkv, D, "bf16", P, VARLEN, seed=0)
    paged.table, paged.k, paged.v = table.cpu(), cache.k.cpu(), cache.v.cpu()
    want = chunk64(rotated.cpu(), paged, [T])
    lse = torch.empty(T, Hq, device="cuda")
    once = torch.empty_like(out)
    da.decode_attn_paged_chunk(rotated, cache, ints([0, T]), ints([T]), table, once, ws, lse=lse)
    assert check(once, lse, want, torch.bfloat16) is None and check(out, lse, want, torch.bfloat16) is None


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (6000, 300)])
def test_long_histories_are_cut_and_joined(window, sinks, D, kv, dtype):
    """Few rows over many keys: parts of an item on many blocks, with values that are not finite in the first and the last."""
    paged = Paged([20000, 700, 9000], 1, D, kv, 64, BHSD, seed=30, scale_spread=4)
    new = [3, 1, 130]
    q = queries(134, 4, D, dtype, 31)
    want = chunk64(q, paged, new, None, window, sinks)
    out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
    assert check(out, lse, want, DTYPES[dtype]) is None
    for b, p in ((0, 19999), (2, 8900), (2, 8999)):
        token_view(paged.v, BHSD)[int(paged.table[b, p // 64]), p % 64, 0, 7] = math.nan
    want = chunk64(q, paged, new, None, window, sinks)
    out, lse = run_chunk(q, paged, new, window=window, sinks=sinks)
    assert torch.isnan(want[0]).any() and check(out, lse, want, DTYPES[dtype]) is None


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    import random
    rng = random.Random(seed)
    kv, dtype = TYPES[seed % 4]
    D, page, layout = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128, 272]), rng.choice([VARLEN, BHSD])
    Hkv, G, B = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.randint(1, 40)
    lens = [rng.choice([0, 1, rng.randint(1, 200), rng.randint(1, 1500)]) for _ in range(B)]
    new = [rng.choice([0, 1, min(n, rng.randint(0, 60)), min(n, rng.randint(0, 400))]) for n in lens]
    window, sinks = rng.choice([(0, 0), (0, 5), (rng.randint(1, 800), rng.choice([0, 4, rng.randint(1, 400)]))])
    compare(lens, new, Hkv * G, Hkv, D, kv, dtype, page, layout, window, sinks, seed=seed, spread=seed % 5, mean=(seed % 3) * 0.3)


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D,window", [(128, 0), (64, 0), (128, 3000)])
def test_long_calls_have_the_same_bits_every_time(D, window, kv, dtype):
    """Every block busy for hundreds of key tiles, again and again: a hand-over that comes too early shows in some run."""
    g = torch.Generator(device="cuda").manual_seed(50)
    lens, new, pages = [16384, 5000], [2048, 700], 400
    shape = (pages, 8, 64, D)
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).to(DTYPES[kv]) for _ in range(2))
    scales = [torch.exp2(torch.randint(-3, 3, (pages, 8), generator=g, device="cuda").float()) for _ in range(2)] if kv == "e4m3" else [None, None]
    cache = da.PagedCache(k, v, *scales, layout=BHSD)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:358]
    table = torch.stack([table[:256], torch.cat([table[256:], table.new_zeros(154)])])
    q = torch.randn(2748, 32, D, generator=g, device="cuda", dtype=DTYPES[dtype])
    ws = da.alloc_paged_chunk_workspace(32, 8, D)
    out, lse = torch.empty_like(q), torch.empty(2748, 32, device="cuda")
    first = None
    for _ in range(40):
        out.fill_(7.0)
        da.decode_attn_paged_chunk(q, cache, ints(starts(new)), ints(lens), table, out, ws, window=window, sinks=5, lse=lse)
        if first is None:
            first = (out.clone(), lse.clone())
            assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert da.decode_attn_splitkv_get_error(ws) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_two_calls_at_once(D):
    """Calls that overlap, on streams and with workspaces of their own, beside decode steps on a third."""
    cases = []
    for i, (kv, dtype) in enumerate([("bf16", "bf16"), ("e4m3", "f16")]):
        paged = Paged([900 + 300 * i, 64, 0, 2000], 2, D, kv, 16, VARLEN, seed=60 + i)
        new = [300, 64, 0, 1 + 200 * i]
        q = queries(sum(new), 8, D, dtype, 62 + i)
        qd = q.cuda()
        cases.append(dict(want=chunk64(q, paged, new), dtype=DTYPES[dtype], stream=torch.cuda.Stream(), out=torch.empty_like(qd),
                          lse=torch.empty(len(q), 8, device="cuda"),
                          args=(qd, on_device(paged), ints(starts(new)), ints(paged.lens), paged.table.cuda()),
                          ws=da.alloc_paged_chunk_workspace(8, 2, D)))
    last = cases[0]
    dec = da.alloc_paged_workspace(1, 8, 2, D)
    dq = queries(4, 8, D, "bf16", 70).cuda()
    dout, third = torch.empty_like(dq), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        for c in cases:
            da.decode_attn_paged_chunk(*c["args"], c["out"], c["ws"], lse=c["lse"], stream=c["stream"])
        da.decode_attn_paged_window(dq, last["args"][1], last["args"][3], last["args"][4], dout, dec, window=100, sinks=4, stream=third)
    torch.cuda.synchronize()
    for c in cases:
        assert da.decode_attn_splitkv_get_error(c["ws"]) == 0
        assert check(c["out"], c["lse"], c["want"], c["dtype"]) is None
    assert da.decode_attn_splitkv_get_error(dec) == 0


@pytest.mark.parametrize("kv,dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_on_16_byte_borders_only(D, kv, dtype):
    """Strides that are odd multiples of 16 bytes, and bases between 32-byte borders; parts and whole items alike."""
    paged = Paged([3000, 90], 1, D, kv, 16, VARLEN, seed=80)
    new = [40, 90]
    q = queries(130, 3, D, dtype, 81)
    want = chunk64(q, paged, new)
    flat_q = torch.full((130 * (3 * D + 8) + 8,), float("nan"), dtype=q.dtype, device="cuda")
    flat_o = torch.full_like(flat_q, 3.0)
    view = lambda x: x[8:].view(130, 3 * D + 8)[:, :3 * D].unflatten(1, (3, D))
    view(flat_q).copy_(q)
    out, lse = view(flat_o), torch.empty(130, 3, device="cuda")
    assert out.data_ptr() % 32 == 16 and out.stride(0) % 16 == 8
    ws = da.alloc_paged_chunk_workspace(3, 1, D)
    da.decode_attn_paged_chunk(view(flat_q), on_device(paged), ints(starts(new)), ints(paged.lens), paged.table.cuda(), out, ws, lse=lse)
    assert check(out, lse, want, DTYPES[dtype]) is None
    assert (flat_o[:8] == 3.0).all() and (flat_o[8:].view(130, 3 * D + 8)[:, 3 * D:] == 3.0).all()
