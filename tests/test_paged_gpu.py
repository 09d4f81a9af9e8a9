"""Decode attention over a paged cache and the append that fills it, against plain references in 64 bits."""
import itertools
import math
import zlib

import numpy as np
import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_ref import (BHSD, DTYPES, VARLEN, Paged, append32, attend64, half_step, needed, table_of, token_view, turned)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.load()


def on_gpu(p):
    """PagedCache, kv_lens and block table of a CPU-side Paged."""
    dev = lambda x: None if x is None else x.cuda()   # noqa: E731
    return (da.PagedCache(p.k.cuda(), p.v.cuda(), dev(p.k_scale), dev(p.v_scale), layout=p.layout),
            torch.tensor(p.lens, dtype=torch.int32, device="cuda"), p.table.cuda())


def queries(p, B, T, Hq, dtype, seed=1, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(B, T, Hq, p.D, generator=gen) * size).to(DTYPES[dtype])


def attend(p, q, scale=None, ws=None, lse=True, stream=None, tensors=None):
    cache, lens, table = on_gpu(p) if tensors is None else tensors
    qd = q.cuda()
    out = torch.full_like(qd, math.nan)
    l = torch.full(q.shape[:-1], math.nan, device="cuda") if lse else None
    ws = da.alloc_paged_workspace(q.shape[1], q.shape[2], p.Hkv, p.D) if ws is None else ws
    torch.cuda.synchronize()
    da.decode_attn_paged(qd, cache, lens, table, out, ws, scale=scale, lse=l, stream=stream)
    err = da.decode_attn_splitkv_get_error(ws, stream=stream)
    return out.double().cpu().numpy(), None if l is None else l.double().cpu().numpy(), err


def check(out, lse, ref, dtype, where=""):
    ro, rl, to, tl = ref
    off = np.abs(out - ro) - half_step(ro, DTYPES[dtype]) - to
    assert np.all(off <= 0), f"{where}: out is {np.nanmax(off)} over its tolerance"      # NaN fails too
    if lse is not None:
        assert np.array_equal(np.isneginf(lse), np.isneginf(rl)), where
        fine = np.isfinite(rl)
        off = np.abs(lse[fine] - rl[fine]) - tl[fine]
        assert np.all(off <= 0), f"{where}: lse is {np.nanmax(off, initial=-1)} over its tolerance"


ATTEND = [
    # kv, q type, T_q, Hq, Hkv, D, page, layout, lengths
    ("f16", "f16", 1, 4, 1, 64, 16, VARLEN, [37, 200]),
    ("f16", "f16", 1, 28, 4, 128, 64, VARLEN, [700, 64, 1, 0, 65]),
    ("bf16", "bf16", 1, 32, 8, 128, 64, BHSD, [513, 130]),
    ("bf16", "bf16", 1, 32, 8, 128, 16, VARLEN, [1024]),
    ("f16", "f16", 1, 8, 8, 128, 32, BHSD, [63, 64, 65, 127, 128, 129]),
    ("f16", "f16", 1, 3, 3, 64, 48, VARLEN, [47, 48, 49, 250]),          # pages that end inside a 64-key tile
    ("bf16", "bf16", 1, 5, 5, 64, 80, BHSD, [79, 80, 81, 400]),
    ("bf16", "bf16", 1, 16, 1, 128, 128, VARLEN, [300, 15, 16, 17]),     # 16 columns
    ("f16", "f16", 1, 40, 2, 64, 64, BHSD, [200, 5]),                    # 20 columns: two chunks
    ("f16", "f16", 4, 28, 4, 128, 64, VARLEN, [700, 64, 4, 3, 1, 0]),    # tokens that see nothing
    ("bf16", "bf16", 2, 32, 8, 128, 64, BHSD, [1000, 66, 130]),
    ("bf16", "bf16", 16, 16, 2, 128, 256, VARLEN, [900, 16]),            # 128 columns
    ("f16", "f16", 3, 4, 1, 64, 1024, BHSD, [2, 1500]),
    ("e4m3", "f16", 1, 4, 1, 64, 16, VARLEN, [37, 200]),
    ("e4m3", "f16", 1, 28, 4, 128, 64, BHSD, [700, 64, 1, 0, 65]),
    ("e4m3", "bf16", 1, 32, 8, 128, 64, VARLEN, [513, 130]),
    ("e4m3", "bf16", 1, 32, 8, 128, 16, BHSD, [1024]),
    ("e4m3", "f16", 1, 8, 8, 128, 32, VARLEN, [63, 64, 65, 127, 128, 129, 255, 256, 257]),
    ("e4m3", "bf16", 1, 3, 3, 64, 48, BHSD, [47, 48, 49, 250]),
    ("e4m3", "f16", 1, 5, 5, 64, 80, VARLEN, [79, 80, 81, 400]),
    ("e4m3", "bf16", 1, 16, 1, 128, 128, BHSD, [300, 15, 16, 17]),
    ("e4m3", "f16", 1, 40, 2, 64, 64, VARLEN, [200, 5]),
    ("e4m3", "bf16", 4, 28, 4, 128, 64, BHSD, [700, 64, 4, 3, 1, 0]),
    ("e4m3", "f16", 5, 16, 4, 64, 128, VARLEN, [1000, 66, 130]),
    ("e4m3", "bf16", 16, 16, 2, 128, 256, BHSD, [900, 16]),
    ("e4m3", "bf16", 3, 4, 1, 64, 1024, VARLEN, [2, 1500]),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_attention(case):
    kv, dt, T, Hq, Hkv, D, page, layout, lens = case
    seed = zlib.crc32(str(case).encode()) % 9973
    p = Paged(lens, Hkv, D, kv, page, layout, seed=seed, scale_spread=2 if kv == "e4m3" else 0)
    q = queries(p, len(lens), T, Hq, dt, seed)
    out, lse, err = attend(p, q)
    assert err == 0
    check(out, lse, attend64(q, p), dt)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[5000], [4097, 3, 1200], [300] * 40, list(range(0, 130, 3))], ids=["one", "skewed", "even", "all"])
def test_attention_over_many_pieces(kv, lens):
    """Lengths that are cut into several pieces, and batches whose pieces hold several sequences."""
    p = Paged(lens, 2, 128, kv, 64, BHSD, seed=3)
    q = queries(p, len(lens), 1, 8, "bf16")
    out, lse, err = attend(p, q)
    assert err == 0
    check(out, lse, attend64(q, p), "bf16")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 96, 128, 256, 1008])
@pytest.mark.parametrize("T,Hq,Hkv,layout", [(1, 8, 2, VARLEN), (3, 6, 1, BHSD), (1, 1, 1, BHSD), (2, 20, 1, VARLEN)])
def test_long_tables_of_16_bit_pages(page, T, Hq, Hkv, layout):
    """Head size 128 with tables of more than a thousand keys (CTAs of eight consumer warps): every page size, one
    and two n-tiles, pieces that begin and end anywhere, and a sequence without keys."""
    lens = [1100, 0, 2, 129, 1023, 640, 4000]
    p = Paged(lens, Hkv, 128, "bf16" if page % 32 else "f16", page, layout, seed=page + T)
    q = queries(p, len(lens), T, Hq, p.kv, page)
    out, lse, err = attend(p, q)
    assert err == 0
    check(out, lse, attend64(q, p), p.kv)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_short_sequences_under_a_very_wide_table_and_none_at_all(kv, D):
    p = Paged([5, 0, 17], 2, D, kv, 16, VARLEN, seed=15, width=9000)
    q = queries(p, 3, 1, 4, "f16")
    out, lse, err = attend(p, q)
    assert err == 0
    check(out, lse, attend64(q, p), "f16")
    cache, lens, table = on_gpu(p)
    lens.zero_()
    out, lse, err = attend(p, q, tensors=(cache, lens, table))
    assert err == 0 and np.all(out == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales_that_are_not_positive(scale):
    for kv in ("bf16", "e4m3"):
        p = Paged([70, 333], 1, 64, kv, 32, BHSD, seed=16)
        q = queries(p, 2, 2, 4, "bf16")
        out, lse, err = attend(p, q, scale=scale)
        assert err == 0
        check(out, lse, attend64(q, p, scale), "bf16")


@pytest.mark.parametrize("kv,q_size,k_size,scale", [
    ("bf16", -2.0 ** 60, 2.0 ** 60, 0.125),      # scores of -2^123 and below: still above a column without keys
    ("f16", 2.0 ** 12, 2.0 ** 12, 1.0), ("e4m3", -2.0 ** 100, 2.0 ** 8, 0.125), ("e4m3", 2.0 ** 10, 2.0, 1.0)])
@pytest.mark.parametrize("T,lens", [(1, [1, 50, 300, 0]), (3, [2, 700])])
def test_equal_scores_of_any_size_give_the_mean(kv, q_size, k_size, scale, T, lens):
    """Every key alike: the output is the mean of the values that a token sees, whatever the score. The products are
    powers of two, so every score is the same float; a weight is 1 or, of an e4m3 value, its page's scale relative to
    the largest in sight, rounded to fp16 (2^-11); sums of n float32 terms are off by n 2^-24, log2, exp2 and their
    arguments by less than 2^-17 for these scales."""
    q_type = "f16" if kv == "f16" else "bf16"
    p = Paged(lens, 1, 64, kv, 16, VARLEN, seed=17)
    p.k = torch.full_like(p.k.float(), k_size).to(p.k.dtype)
    if kv == "e4m3":
        p.k_scale = torch.ones_like(p.k_scale)
        p.v_scale = torch.rand(p.v_scale.shape, generator=torch.Generator().manual_seed(18)) * 3 + 0.3
    q = torch.full((len(lens), T, 2, 64), q_size).to(DTYPES[q_type])
    out, lse, err = attend(p, q, scale=scale)
    assert err == 0
    x = q_size * k_size * 64 * scale
    for b, L in enumerate(lens):
        v = p.sequence(b)[1].numpy()[:, 0] if L else None
        for t in range(T):
            n = L - T + 1 + t
            if n <= 0:
                assert np.all(out[b, t] == 0) and np.all(np.isneginf(lse[b, t]))
                continue
            mean, size = v[:n].mean(0), np.abs(v[:n]).mean(0)
            tol = half_step(mean, DTYPES[q_type]) + size * (2.0 ** -11 * (kv == "e4m3") + n * 2.0 ** -24 + 2.0 ** -17)
            assert np.all(np.abs(out[b, t] - mean) <= tol), (b, t)
            assert np.all(np.abs(lse[b, t] - (x + math.log(n))) <= 2.0 ** -21 * abs(x) + 1e-5)


def test_a_batch_of_the_largest_size():
    lens = [(7 * i) % 40 for i in range(da.DA_MAX_PAGED_BATCH)]
    for kv in ("f16", "e4m3"):
        p = Paged(lens, 1, 64, kv, 16, VARLEN, seed=4)
        q = queries(p, len(lens), 1, 2, "f16")
        out, lse, err = attend(p, q)
        assert err == 0
        check(out, lse, attend64(q, p), "f16")


def test_scales_of_very_unequal_size():
    """Pages whose scales differ by 2^40: the heavy pages' weights vanish, the light pages decide the answer,
    and the other way round."""
    for seed, small_first in ((5, True), (6, False)):
        p = Paged([256, 300], 2, 128, "e4m3", 64, BHSD, seed=seed)
        for b in range(2):
            at = p.table[b, :4].long()
            size = torch.tensor([2.0 ** -30, 2.0 ** -20, 1.0, 2.0 ** 10])
            p.v_scale[at] = (size if small_first else size.flip(0))[:, None].expand(4, 2)
            # keys of the pages with heavy values score far below the others
            p.k_scale[at] = 2.0 ** -6
        q = queries(p, 2, 1, 8, "bf16")
        for b in range(2):
            heavy = p.table[b, 3 if small_first else 0].long()
            k = p.k[heavy].float()
            k[:] = (-q[b, 0].float().view(2, 4, 128).mean(1) * 60).clamp(-448, 448)[:, None, :]
            p.k[heavy] = k.to(torch.float8_e4m3fn)
        out, lse, err = attend(p, q, scale=1.0)
        assert err == 0
        ro, rl, to, tl = attend64(q, p, scale=1.0)
        # the tolerance of the heaviest value, but weighed: sum of w |v| u bounds what the weights' rounding moves
        for b, h in itertools.product(range(2), range(8)):
            k, v = (x.numpy()[:, h // 4] for x in p.sequence(b))
            x = k @ q[b, 0, h].double().numpy()
            w = np.exp(x - rl[b, 0, h])
            dot = 132 * 2.0 ** -24 * (np.linalg.norm(q[b, 0, h].double().numpy()) * np.linalg.norm(k, axis=1)).max()
            rel = 2.0 ** -11 + 2 * (dot + 2.0 ** -22 * (1 + 2 * np.abs(x).max())) + 2 * len(x) * 2.0 ** -24
            # a weight below 2^-14 of the heaviest is a subnormal fp16, off by up to 2^-25 of that one; the
            # elements it meets are codes of at most 448, at most 8 times the heaviest key's largest
            bound = rel * (w[:, None] * np.abs(v)).sum(0) + 2.0 ** -25 * (w[:, None] * np.abs(v).max(1, keepdims=True)).max() * len(x) * 8
            off = np.abs(out[b, 0, h] - ro[b, 0, h]) - half_step(ro[b, 0, h], torch.bfloat16) - bound
            assert np.all(off <= 0), (b, h, off.max())


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_queries_of_any_bfloat16_size(size):
    """8-bit keys meet bf16 queries outside the fp16 range."""
    p = Paged([200, 90], 2, 128, "e4m3", 64, BHSD, seed=7)
    q = queries(p, 2, 1, 8, "bf16", size=size)
    scale = 1 / (size * math.sqrt(128))
    out, lse, err = attend(p, q, scale=scale)
    assert err == 0
    check(out, lse, attend64(q, p, scale), "bf16")


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_zero_and_extreme_queries(kv):
    p = Paged([130, 7], 1, 64, kv, 16, VARLEN, seed=8)
    q = queries(p, 2, 1, 8, "f16")
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 100          # one key takes all the weight
    q[1, 0, 2, 3] = 6e-8       # a subnormal fp16
    out, lse, err = attend(p, q)
    assert err == 0
    check(out, lse, attend64(q, p), "f16")
    assert abs(lse[0, 0, 0] - math.log(130)) < 1e-5


def test_nan_of_a_visible_key_reaches_only_its_sequence_and_head():
    for kv, code in (("bf16", 0x7FC0), ("e4m3", 0x7F)):
        p = Paged([90, 90], 2, 64, kv, 16, VARLEN, seed=9)
        q = queries(p, 2, 1, 4, "bf16")
        ref = attend64(q, p)
        raw = p.v.view(torch.uint8 if kv == "e4m3" else torch.int16)
        token_view(raw, VARLEN)[p.table[1, 2].long(), 5, 1, 7] = code
        out, lse, _ = attend(p, q)
        assert np.isnan(out[1, 0, 2:, 7]).all()
        out[1, 0, 2:, 7] = 0
        ref[0][1, 0, 2:, 7] = 0
        check(out, lse, ref, "bf16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_nan_scores_are_not_taken_for_masked_ones(kv):
    """A query of NaN, a key of NaN that is all a sequence has, and one among others in a later piece."""
    p = Paged([700, 1, 90], 2, 64, kv, 16, BHSD, seed=14)
    q = queries(p, 3, 1, 4, "bf16")
    ref = attend64(q, p)
    q[0, 0, 1, 5] = math.nan
    raw = p.k.view(torch.uint8 if kv == "e4m3" else torch.int16)
    code = 0x7F if kv == "e4m3" else 0x7FC0
    token_view(raw, BHSD)[p.table[1, 0].long(), 0, 0, 3] = code      # sequence 1's only key, KV head 0
    token_view(raw, BHSD)[p.table[2, 5].long(), 9, 1, 0] = code      # sequence 2's last one, KV head 1
    out, lse, err = attend(p, q)
    assert err == 0
    bad = np.zeros((3, 1, 4), dtype=bool)
    bad[0, 0, 1] = bad[1, 0, :2] = bad[2, 0, 2:] = True
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    out[bad], lse[bad] = ref[0][bad], ref[1][bad]
    check(out, lse, ref, "bf16")


def test_a_capture_as_the_very_first_call():
    """A process whose first calls are captured: what a call looks up once per device is no obstacle."""
    import subprocess
    import sys
    code = """
import torch
import split_kv_decode_decoding_gb300 as da
da.load()
dev = "cuda"
for dtype in (torch.float16, torch.float8_e4m3fn):
    cache = da.PagedCache.empty(4, 16, 1, 64, dtype)
    kv_lens = torch.tensor([20, 1], dtype=torch.int32, device=dev)
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 20, 21], dtype=torch.int32, device=dev)
    x = torch.randn(21, 4, 64, device=dev).half()
    out = torch.empty(2, 2, 64, dtype=torch.float16, device=dev)
    ws = da.alloc_paged_workspace(1, 2, 1, 64)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        da.decode_attn_paged_append(None, x[:, 2:3], x[:, 3:], cache, cu, kv_lens, table, ws)
        da.decode_attn_paged(x[:2, :2].contiguous(), cache, kv_lens, table, out, ws)
    g.replay()
    torch.cuda.synchronize()
    assert da.decode_attn_splitkv_get_error(ws) == 0
    assert torch.isfinite(out).all()
    first = out[1].float()                       # one key: its value, in fp16 or rounded to e4m3
    assert torch.allclose(first[0], x[20, 3].float(), rtol=2 ** -4, atol=2 ** -8), (first[0], x[20, 3])
print("captured")
"""
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured" in got.stdout, got.stderr[-2000:]


def test_shared_pages_and_a_wide_strided_table():
    p = Paged([100, 164], 2, 64, "f16", 32, VARLEN, seed=10, extra_pages=3)
    p.table[1, :2] = p.table[0, :2]      # a common prefix of 64 tokens
    q = queries(p, 2, 1, 4, "f16")
    cache, lens, table = on_gpu(p)
    wide = torch.full((2, 50), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    out, lse, err = attend(p, q, tensors=(cache, lens, wide[:, : table.shape[1]]))
    assert err == 0
    check(out, lse, attend64(q, p), "f16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", [VARLEN, BHSD])
def test_bad_pages_read_as_zeros(kv, layout):
    p = Paged([200, 100], 2, 64, kv, 32, layout, seed=11)
    q = queries(p, 2, 1, 4, "bf16")
    good = on_gpu(p)
    for entry in (-1, p.k.shape[0], 1 << 30, -(1 << 31)):
        table = p.table.clone()
        table[0, 3] = entry
        out, lse, err = attend(p, q, tensors=(good[0], good[1], table.cuda()))
        assert err == da.DA_DEVERR_PAGE
        # the same with a page of zeros in its place
        z = Paged([200, 100], 2, 64, kv, 32, layout, seed=11)
        for x in (z.k, z.v):
            x.view(torch.uint8 if kv == "e4m3" else torch.int16)[z.table[0, 3].long()] = 0
        check(out, lse, attend64(q, z), "bf16", str(entry))


def test_bad_lengths_count_as_empty():
    p = Paged([40, 50, 60], 1, 64, "f16", 16, VARLEN, seed=12)
    q = queries(p, 3, 2, 2, "f16")
    ref = attend64(q, p)
    cache, lens, table = on_gpu(p)
    for bad in (-1, 65, 1 << 30, -(1 << 31)):
        lens[1] = bad
        out, lse, err = attend(p, q, tensors=(cache, lens, table))
        assert err == da.DA_DEVERR_SEQLENS
        assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
        check(out[[0, 2]], lse[[0, 2]], [x[[0, 2]] for x in ref], "f16")


def test_three_dimensional_queries_and_no_lse():
    p = Paged([77, 140], 2, 128, "bf16", 64, VARLEN, seed=13)
    q = queries(p, 2, 1, 8, "bf16")
    cache, lens, table = on_gpu(p)
    ws = da.alloc_paged_workspace(1, 8, 2, 128)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    da.decode_attn_paged(q[:, 0].contiguous().cuda(), cache, lens, table, out, ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    check(out.double().cpu().numpy()[:, None], None, attend64(q, p), "bf16")


def test_one_workspace_for_calls_of_every_kind_and_the_same_bits_again():
    """Calls in a row share a workspace, none sees another's leftovers, and a repeated call gives the same bits."""
    ws = da.alloc_paged_workspace(4, 32, 4, 128)
    kinds = []
    for i, (kv, dt, T, Hq, Hkv, D, lens) in enumerate([
            ("f16", "f16", 1, 28, 4, 128, [3000, 5, 700]), ("e4m3", "bf16", 4, 32, 4, 128, [900, 2000]),
            ("bf16", "bf16", 1, 8, 8, 64, [64] * 20), ("e4m3", "f16", 1, 8, 1, 64, [6000])]):
        p = Paged(lens, Hkv, D, kv, 64, i % 2, seed=20 + i)
        q = queries(p, len(lens), T, Hq, dt)
        kinds.append((p, q, dt, attend64(q, p), on_gpu(p)))
    first = [attend(p, q, ws=ws, tensors=t) for p, q, dt, ref, t in kinds]
    for (out, lse, err), (p, q, dt, ref, t) in zip(first, kinds):
        assert err == 0
        check(out, lse, ref, dt)
    for _ in range(3):
        for (out, lse, _), (p, q, dt, ref, t) in zip(first, kinds):
            again, lse2, err = attend(p, q, ws=ws, tensors=t)
            assert err == 0 and np.array_equal(again, out) and np.array_equal(lse2, lse)


def test_a_side_stream_and_a_replayed_graph_with_growing_lengths():
    lens = [100, 1000, 64]
    p = Paged([n + 40 for n in lens], 2, 128, "e4m3", 64, BHSD, seed=30)
    q = queries(p, 3, 1, 8, "bf16")
    cache, _, table = on_gpu(p)
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = da.alloc_paged_workspace(1, 8, 2, 128)
    out = torch.empty_like(q.cuda())
    lse = torch.empty(3, 1, 8, device="cuda")
    qd = q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        da.decode_attn_paged(qd, cache, kv_lens, table, out, ws, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.decode_attn_paged(qd, cache, kv_lens, table, out, ws, lse=lse)
    for step in range(3):
        now = [n + 13 * step for n in lens]
        kv_lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(math.nan)
        graph.replay()
        assert da.decode_attn_splitkv_get_error(ws) == 0
        p.lens = now
        check(out.double().cpu().numpy(), lse.double().cpu().numpy(), attend64(q, p), "bf16", f"step {step}")


def test_two_graphs_replayed_at_once_with_a_workspace_each():
    p = Paged([2000, 1500], 4, 128, "f16", 64, VARLEN, seed=31)
    tensors = on_gpu(p)
    runs = []
    for i in range(2):
        q = queries(p, 2, 1, 16, "f16", seed=40 + i)
        qd, ws = q.cuda(), da.alloc_paged_workspace(1, 16, 4, 128)
        out = torch.empty_like(qd)
        da.decode_attn_paged(qd, *tensors[:1], tensors[1], tensors[2], out, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            da.decode_attn_paged(qd, tensors[0], tensors[1], tensors[2], out, ws)
        runs.append((q, out, ws, g, torch.cuda.Stream(), qd))
    for _ in range(20):
        for q, out, ws, g, s, qd in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for q, out, ws, g, s, qd in runs:
        assert da.decode_attn_splitkv_get_error(ws) == 0
        check(out.double().cpu().numpy(), None, attend64(q, p), "f16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_past_32_bits(kv):
    """A cache whose last pages lie past 2^32 elements."""
    D, Hkv, page = 128, 8, 64
    pages = (1 << 32) // (D * Hkv * page) + 8
    p = Paged([150, 260], Hkv, D, kv, page, BHSD, seed=50)
    far = torch.empty((pages, Hkv, page, D), dtype=p.k.dtype, device="cuda")
    far_v = torch.empty_like(far)
    n = p.k.shape[0]
    for big, small in ((far, p.k), (far_v, p.v)):
        raw = torch.uint8 if kv == "e4m3" else torch.int16
        big.view(raw)[pages - n:] = small.view(raw).cuda()
    scales = [None, None]
    if kv == "e4m3":
        scales = [torch.zeros(pages, Hkv, device="cuda") for _ in range(2)]
        scales[0][pages - n:], scales[1][pages - n:] = p.k_scale.cuda(), p.v_scale.cuda()
    cache = da.PagedCache(far, far_v, *scales, layout=BHSD)
    table = torch.where(p.table >= 0, p.table + (pages - n), p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    q = queries(p, 2, 1, 16, "bf16")
    out, lse, err = attend(p, q, tensors=(cache, lens, table))
    assert err == 0
    check(out, lse, attend64(q, p), "bf16")
    # and an append there
    T = 2
    x = torch.randn(T, Hkv, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ws = da.alloc_paged_workspace(1, 16, Hkv, D)
    da.decode_attn_paged_append(None, x.cuda(), x.cuda(), cache, cu, lens, table, ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    append32(p, None, x, x, p.lens, [1, 1], None, 0)
    raw = torch.uint8 if kv == "e4m3" else torch.int16
    assert torch.equal(far.view(raw)[pages - n:].cpu(), p.k.view(raw)) and torch.equal(far_v.view(raw)[pages - n:].cpu(), p.v.view(raw))


# ------------------------------------------------------------------ append
APPEND = [
    # kv, type, Hq, Hkv, D, page, layout, rope, rot, lengths after the append, new tokens
    ("f16", "f16", 28, 4, 128, 64, VARLEN, 1, 128, [1, 65, 64, 700, 128], [1, 1, 1, 1, 1]),
    ("bf16", "bf16", 32, 8, 128, 64, BHSD, 1, 128, [300, 77], [300, 70]),
    ("bf16", "bf16", 4, 1, 64, 16, VARLEN, 2, 64, [33, 16, 17, 100], [33, 3, 0, 50]),
    ("f16", "f16", 5, 5, 64, 48, BHSD, 2, 32, [49, 200], [2, 101]),
    ("f16", "f16", 8, 2, 128, 32, VARLEN, 1, 64, [31, 32, 33], [31, 1, 1]),
    ("f16", "f16", 3, 3, 64, 16, VARLEN, 0, 0, [20, 5], [7, 5]),
    ("bf16", "bf16", 7, 1, 128, 1024, BHSD, 1, 16, [1030, 5], [9, 4]),
    ("e4m3", "f16", 28, 4, 128, 64, VARLEN, 1, 128, [1, 65, 64, 700, 128], [1, 1, 1, 1, 1]),
    ("e4m3", "bf16", 32, 8, 128, 64, BHSD, 1, 128, [300, 77], [300, 70]),
    ("e4m3", "bf16", 4, 1, 64, 16, VARLEN, 2, 64, [33, 16, 17, 100], [33, 3, 0, 50]),
    ("e4m3", "f16", 5, 5, 64, 48, BHSD, 2, 32, [49, 200], [2, 101]),
    ("e4m3", "f16", 8, 2, 128, 32, VARLEN, 1, 64, [31, 32, 33], [31, 1, 1]),
    ("e4m3", "bf16", 3, 3, 64, 16, BHSD, 0, 0, [20, 5], [7, 5]),
    ("e4m3", "bf16", 7, 1, 128, 1024, VARLEN, 1, 16, [1030, 5], [9, 4]),
]


def fused_rows(T, Hq, Hkv, D, dtype, seed, pad=0):
    """q, k and v as slices of one projection's output."""
    x = torch.randn(T + pad, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype])
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def run_append(p, q, k, v, lens, new, cos_sin, rope, pad=0, q_out=None, ws=None, max_pos=None):
    """The append on the GPU; returns (q_out, cache on the GPU, error bits)."""
    cache, _, table = on_gpu(p)
    base = torch.cat([x for x in (q, k, v)], 1).cuda()      # one strided buffer again
    Hq, Hkv = q.shape[1], k.shape[1]
    qd, kd, vd = base[:, :Hq], base[:, Hq:Hq + Hkv], base[:, Hq + Hkv:]
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, -3.0, dtype=q.dtype, device="cuda") if q_out is None else qd
    ws = da.alloc_paged_workspace(1, max(Hq, 1), Hkv, p.D) if ws is None else ws
    da.decode_attn_paged_append(qd, kd, vd, cache, cu, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, ws,
                                cos_sin=None if rope == 0 else cos_sin.cuda(), rope=rope, q_out=out)
    return out, cache, da.decode_attn_splitkv_get_error(ws)


def same_bits(a, b):
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().contiguous().view(raw), b.cpu().contiguous().view(raw))


def check_append(p, got_q, cache, q_ref, T):
    assert same_bits(got_q[:T], q_ref), "queries"
    for name in ("k", "v"):
        assert same_bits(getattr(cache, name), getattr(p, name)), name
        if p.kv == "e4m3":
            assert same_bits(getattr(cache, name + "_scale"), getattr(p, name + "_scale")), name + "_scale"


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_append(case):
    """Bit for bit the step-by-step float32 evaluation, everything else in the cache untouched, and the
    rows behind the last sequence left as they were."""
    kv, dt, Hq, Hkv, D, page, layout, rope, rot, lens, new = case
    p = Paged(lens, Hkv, D, kv, page, layout, seed=60, scale_spread=3 if kv == "e4m3" else 0)
    T, pad = sum(new), 3
    q, k, v = fused_rows(T, Hq, Hkv, D, dt, 61, pad)
    cos_sin = table_of(max(lens), rot) if rope else None
    got, cache, err = run_append(p, q, k, v, lens, new, cos_sin, rope)
    assert err == 0
    q_ref = append32(p, q, k, v, lens, new, cos_sin, rope)
    check_append(p, got, cache, q_ref, T)
    assert torch.all(got[T:] == -3.0), "rows behind the last sequence"
    # and within what the types allow of the definition in 64 bits
    position = torch.tensor([x for n, m in zip(lens, new) for x in range(n - m, n)], dtype=torch.long)
    for ref, y in ((turned(q[:T], cos_sin, position, rope), got[:T].cpu().double()),):
        tol = half_step(ref.numpy(), q.dtype) + 4 * 2.0 ** -24 * np.abs(q[:T].double().numpy()).max() * 2
        assert np.all(np.abs(y.numpy() - ref.numpy()) <= tol)
    where = [(b, x) for b, (n, m) in enumerate(zip(lens, new)) for x in range(n - m, n)]
    for name, ref in (("k", turned(k[:T], cos_sin, position, rope)), ("v", v[:T].double())):
        pages = token_view(getattr(cache, name).cpu(), layout)
        for i, (b, x) in enumerate(where):
            pg, slot = int(p.table[b, x // page]), x % page
            y, r = pages.view(torch.uint8)[pg, slot].view(pages.dtype).double() if kv == "e4m3" else pages[pg, slot].double(), ref[i].numpy()
            f32 = 4 * 2.0 ** -24 * 2 * np.abs(r).max()
            if kv == "e4m3":
                s = getattr(cache, name + "_scale").cpu()[pg].double()[:, None].numpy()
                assert np.all(np.abs(r) <= 448 * s * (1 + 2.0 ** -22))
                tol = np.maximum(np.abs(r) * 2.0 ** -4, s * 2.0 ** -10) + f32     # half a step: 2^-4, or half of 2^-9
                assert np.all(np.abs(y.numpy() * s - r) <= tol)
            else:
                assert np.all(np.abs(y.numpy() - r) <= half_step(r, pages.dtype) + f32)


def test_a_page_scale_grows_and_earlier_elements_follow():
    """Tokens of growing, then shrinking size, one by one: the scale only grows, and every element stays
    within its rounding (one more for each time its page's scale grew)."""
    sizes = [2.0 ** -6, 1.0, 2.0 ** 7, 2.0 ** 3, 2.0 ** 9, 2.0 ** -8]
    p = Paged([len(sizes)], 2, 64, "e4m3", 16, BHSD, seed=70)
    cache, _, table = on_gpu(p)
    ws = da.alloc_paged_workspace(1, 2, 2, 64)
    rows = [torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) * s for i, s in enumerate(sizes)]
    for i, x in enumerate(rows):
        lens = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        da.decode_attn_paged_append(None, x.cuda(), (-x).cuda(), cache, cu, lens, table, ws)
        append32(p, None, x, -x, [i + 1], [1], None, 0)
        assert da.decode_attn_splitkv_get_error(ws) == 0
        for name in ("k", "v"):
            assert same_bits(getattr(cache, name), getattr(p, name)) and same_bits(getattr(cache, name + "_scale"), getattr(p, name + "_scale"))
    pg = int(p.table[0, 0])
    s = float(cache.k_scale[pg, 0])
    assert s == needed(max(float(x[:, 0].abs().max()) for x in rows))
    got = cache.k[pg, 0].double().cpu() * s
    for i, x in enumerate(rows):
        r = x[0, 0].double()
        assert torch.all((got[i] - r).abs() <= torch.maximum(r.abs() * 2 * 2.0 ** -4, torch.tensor(s * 2.0 ** -9))), i


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,layout", [(16, VARLEN), (32, BHSD), (48, VARLEN), (64, BHSD), (96, VARLEN), (256, BHSD)])
@pytest.mark.parametrize("rope,rot", [(0, 0), (1, 64), (2, 32)])
def test_prompts_with_infinities_and_nan_in_8_bit_pages(D, page, layout, rope, rot):
    """Units of every number of threads, each page several times what a block holds at once or less than that; some
    pages of some heads have an infinity (their threads look for the largest finite element again), some a NaN."""
    lens, new = [333, 70, 5, 600], [333, 33, 5, 401]
    p = Paged(lens, 3, D, "e4m3", page, layout, seed=80 + page)
    q, k, v = fused_rows(sum(new), 6, 3, D, "bf16", 81)
    k, v = k.clone(), v.clone()
    gen = torch.Generator().manual_seed(82)
    for x in (k, v):
        for value in (math.inf, -math.inf, math.nan):
            for row in torch.randint(0, sum(new), (4,), generator=gen).tolist():
                x[row, row % 3, -1 if rot < D else 5] = value        # dims past a part rotation, or values, stay as they are
    if rope and rot == D:
        k = torch.where(torch.isfinite(k), k, torch.ones_like(k))    # a rotated infinity may meet another: keys stay finite
    cs = None if rope == 0 else table_of(700, rot)
    got, cache, err = run_append(p, q, k, v, lens, new, cs, rope)
    assert err == 0
    check_append(p, got, cache, append32(p, q, k, v, lens, new, cs, rope), sum(new))


@pytest.mark.parametrize("D,page", [(64, 16), (64, 32), (64, 64), (64, 256), (128, 32), (128, 64), (128, 1024)])
def test_many_tokens_of_growing_size_into_a_begun_page(D, page):
    """Chunks of a prompt, each larger in value than the one before, several rows per thread and pages of
    more rows than a block holds at once: the begun page is rounded again each time."""
    chunks = [7, 150, 33, 900]
    total = sum(chunks)
    p = Paged([total], 2, D, "e4m3", page, VARLEN, seed=74)
    cache, _, table = on_gpu(p)
    ws, cs = da.alloc_paged_workspace(1, 2, 2, D), table_of(total, D)
    at = 0
    for i, m in enumerate(chunks):
        at += m
        q, k, v = fused_rows(m, 2, 2, D, "bf16", 75 + i)
        k, v = k * 4.0 ** i, v * 4.0 ** i
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        out = torch.empty(m, 2, D, dtype=torch.bfloat16, device="cuda")
        da.decode_attn_paged_append(q.cuda(), k.cuda(), v.cuda(), cache, cu, torch.tensor([at], dtype=torch.int32, device="cuda"),
                                    table, ws, cos_sin=cs.cuda(), q_out=out)
        assert da.decode_attn_splitkv_get_error(ws) == 0
        check_append(p, out, cache, append32(p, q, k, v, [at], [m], cs, 1), m)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_append_to_the_largest_batch(kv):
    B = da.DA_MAX_PAGED_BATCH
    new = [(i * 5) % 4 for i in range(B)]
    lens = [n + (i * 11) % 40 for i, n in enumerate(new)]
    p = Paged(lens, 1, 64, kv, 16, BHSD, seed=76)
    q, k, v = fused_rows(sum(new), 2, 1, 64, "f16", 77)
    cs = table_of(64, 64)
    got, cache, err = run_append(p, q, k, v, lens, new, cs, 2)
    assert err == 0
    check_append(p, got, cache, append32(p, q, k, v, lens, new, cs, 2), sum(new))


def test_a_batch_without_new_tokens_changes_nothing():
    for kv in ("bf16", "e4m3"):
        p = Paged([20, 0], 1, 64, kv, 16, VARLEN, seed=78)
        q, k, v = fused_rows(3, 2, 1, 64, "bf16", 79)
        got, cache, err = run_append(p, q, k, v, [20, 0], [0, 0], table_of(32, 64), 1)
        assert err == 0 and torch.all(got == -3.0)
        assert same_bits(cache.k, p.k) and same_bits(cache.v, p.v)


def test_scales_that_are_no_powers_of_two_and_stale_scales_of_fresh_pages():
    lens, new = [40, 33], [3, 1]            # a page begun before, and one that begins with this token
    p = Paged(lens, 2, 128, "e4m3", 32, VARLEN, seed=71)
    p.k_scale[p.table[0, 1].long()] = 0.0123      # a calibrated scale that the new tokens exceed
    p.v_scale[p.table[0, 1].long()] = 3.7         # and one that holds them
    p.k_scale[p.table[1, 1].long()] = 1e30        # stale
    p.v_scale[p.table[1, 1].long()] = math.nan
    q, k, v = fused_rows(4, 4, 2, 128, "bf16", 72)
    k = k * 4
    cs = table_of(64, 128)
    got, cache, err = run_append(p, q, k, v, lens, new, cs, 1)
    assert err == 0
    check_append(p, got, cache, append32(p, q, k, v, lens, new, cs, 1), 4)
    assert float(cache.v_scale[p.table[0, 1].long(), 0]) == pytest.approx(3.7)


def test_borders_zeros_infinities_and_nan_in_8_bit_pages():
    rows = torch.zeros(6, 1, 64)
    rows[0, 0, :4] = torch.tensor([3.5, -1.0, 17 / 16, 19 / 16])          # 3.5 = 448 * 2^-7 fits exactly; ties
    rows[2, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0])
    rows[3, 0, :2] = torch.tensor([math.nan, math.nan])
    rows[4, 0, 0] = 2.0 ** 120
    rows[5, 0, :2] = torch.tensor([2.0 ** -133, 2.0 ** -126])
    x = rows.to(torch.bfloat16)
    lens, new = [1] * 6, [1] * 6
    p = Paged(lens, 1, 64, "e4m3", 16, BHSD, seed=73)
    got, cache, err = run_append(p, x[:, :0], x, x, lens, new, None, 0, ws=da.alloc_paged_workspace(1, 1, 1, 64))
    assert err == 0
    for name in ("k", "v"):
        s = getattr(cache, name + "_scale").cpu()
        by = [float(s[p.table[b, 0].long(), 0]) for b in range(6)]
        assert by[0] == 2.0 ** -7 and by[1] == 2.0 ** -126 and by[2] == 2.0 ** -7 and by[3] == 2.0 ** -126
        assert by[4] == 2.0 ** 112 and by[5] == 2.0 ** -126
        y = [getattr(cache, name).cpu().view(torch.uint8)[p.table[b, 0].long(), 0, 0].view(torch.float8_e4m3fn).float() for b in range(6)]
        assert y[0][:4].tolist() == [448.0, -128.0, 128.0, 160.0]          # 136 and 152 are ties: to even
        assert torch.all(y[1] == 0)
        assert y[2][:2].tolist() == [448.0, -448.0] and math.isnan(y[2][2]) and y[2][3] == 256.0
        assert math.isnan(y[3][0]) and math.isnan(y[3][1]) and torch.all(y[3][2:] == 0)


def test_sequences_and_tokens_that_are_left_out():
    """Lengths, rows, pages and positions that cannot be: flagged, nothing written for them, the rest done."""
    for kv in ("bf16", "e4m3"):
        lens, new = [20, 30, 9, 40, 50], [2, 1, 1, 4, 1]
        p = Paged(lens, 2, 64, kv, 16, VARLEN, seed=80)
        q, k, v = fused_rows(sum(new), 4, 2, 64, "bf16", 81)
        cs = table_of(38, 64)                   # sequence 3's last two tokens and sequence 4's lie past it
        cache, _, table = on_gpu(p)
        table[2, 0] = p.k.shape[0]              # sequence 2: a page outside the cache
        kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kv_lens[1] = 16 * table.shape[1] + 1    # sequence 1: longer than its table
        cu = torch.tensor([0, 2, 3, 4, 8, 9], dtype=torch.int32, device="cuda")
        out = torch.full((9, 4, 64), -3.0, dtype=torch.bfloat16, device="cuda")
        ws = da.alloc_paged_workspace(1, 4, 2, 64)
        da.decode_attn_paged_append(q.cuda(), k.cuda(), v.cuda(), cache, cu, kv_lens, table, ws, cos_sin=cs.cuda(), q_out=out)
        assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_SEQLENS | da.DA_DEVERR_PAGE | da.DA_DEVERR_POSITION
        rows = torch.tensor([0, 1, 3, 4, 5])
        at = torch.tensor([18, 19, 8, 36, 37])
        assert same_bits(out.cpu()[rows], turned(q[rows], cs, at, 1, torch.float32).to(torch.bfloat16))
        assert torch.all(out.cpu()[[2, 6, 7, 8]] == -3.0)
        # what was written: sequences 0 and 3, the latter without its last two tokens
        append32(p, None, k[torch.tensor([0, 1])], v[torch.tensor([0, 1])], [20], [2], cs, 1)
        p.table = p.table[3:4]
        append32(p, None, k[4:6], v[4:6], [38], [2], cs, 1)
        for name in ("k", "v"):
            assert same_bits(getattr(cache, name), getattr(p, name))


@pytest.mark.parametrize("bad", [[0, 3, 2, 5], [0, 2, 3, 9], [-1, 2, 3, 5], [1 << 30, -(1 << 31), 4, 5]])
def test_row_bounds_that_cannot_be(bad):
    """cu_new that decreases, or leaves the rows: those sequences are left out, no access leaves a tensor."""
    for kv in ("f16", "e4m3"):
        p = Paged([10, 10, 10], 1, 64, kv, 16, VARLEN, seed=82)
        q, k, v = fused_rows(5, 2, 1, 64, "f16", 83)
        cache, lens, table = on_gpu(p)
        ws = da.alloc_paged_workspace(1, 2, 1, 64)
        out = torch.zeros(5, 2, 64, dtype=torch.float16, device="cuda")
        da.decode_attn_paged_append(q.cuda(), k.cuda(), v.cuda(), cache, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                                    lens, table, ws, q_out=out)
        assert da.decode_attn_splitkv_get_error(ws) & da.DA_DEVERR_SEQLENS


def test_queries_rotated_in_place():
    lens, new = [70, 5], [6, 5]
    for kv in ("f16", "e4m3"):
        p = Paged(lens, 2, 128, kv, 64, BHSD, seed=84)
        q, k, v = fused_rows(11, 8, 2, 128, "f16", 85)
        cs = table_of(128, 128)
        got, cache, err = run_append(p, q, k, v, lens, new, cs, 1, q_out="in place")
        assert err == 0
        check_append(p, got, cache, append32(p, q, k, v, lens, new, cs, 1), 11)


@pytest.mark.parametrize("kv,layout", [("bf16", VARLEN), ("e4m3", BHSD), ("e4m3", VARLEN)])
def test_prompt_then_decode_steps_in_a_graph(kv, layout):
    """The operators as a server uses them: prompts appended, then a captured step (append one token per
    sequence, attend) replayed, against attention in 64 bits over what the cache holds."""
    Hq, Hkv, D, page, steps = 8, 2, 128, 32, 40
    prompt = [45, 1, 130]
    full = Paged([n + steps for n in prompt], Hkv, D, kv, page, layout, seed=90)
    cache = da.PagedCache.empty(full.k.shape[0], page, Hkv, D, DTYPES[kv], layout=layout)
    cache.k.view(torch.uint8).fill_(0x7F)
    cache.v.view(torch.uint8).fill_(0x7F)
    table, cs = full.table.cuda(), table_of(256, D)
    csd = cs.cuda()
    q, k, v = (x.cuda() for x in fused_rows(sum(prompt), Hq, Hkv, D, "bf16", 91))
    kv_lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 45, 46, 176], dtype=torch.int32, device="cuda")
    ws = da.alloc_paged_workspace(1, Hq, Hkv, D)
    da.decode_attn_paged_append(q, k, v, cache, cu, kv_lens, table, ws, cos_sin=csd, q_out=torch.empty_like(q))
    one = torch.arange(4, dtype=torch.int32, device="cuda")
    step_rows = torch.zeros(3, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    sq, sk, sv = step_rows[:, :Hq], step_rows[:, Hq:Hq + Hkv], step_rows[:, Hq + Hkv:]
    turned_q = torch.empty(3, Hq, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(turned_q), torch.empty(3, Hq, device="cuda")

    def step():
        kv_lens.add_(1)
        da.decode_attn_paged_append(sq, sk, sv, cache, one, kv_lens, table, ws, cos_sin=csd, q_out=turned_q)
        da.decode_attn_paged(turned_q, cache, kv_lens, table, out, ws, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = None
    for i in range(steps):
        x = torch.randn(3, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(100 + i)) * (1 + i % 7)
        step_rows.copy_(x.to(torch.bfloat16))
        if i == 0:
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        assert da.decode_attn_splitkv_get_error(ws) == 0
        if i % 13 == 0 or i == steps - 1:
            held = Paged([n + i + 1 for n in prompt], Hkv, D, kv, page, layout, seed=90)
            held.table, held.k, held.v = full.table, cache.k.cpu(), cache.v.cpu()
            if kv == "e4m3":
                held.k_scale, held.v_scale = cache.k_scale.cpu(), cache.v_scale.cpu()
            qc = turned_q.cpu()[:, None]
            at = torch.tensor([n + i for n in prompt])
            assert same_bits(turned_q, turned(x.to(torch.bfloat16)[:, :Hq], cs, at, 1, torch.float32).to(torch.bfloat16))
            check(out.double().cpu().numpy()[:, None], lse.double().cpu().numpy()[:, None], attend64(qc, held), "bf16", f"step {i}")


def test_refusals_of_the_binding():
    p = Paged([20, 9], 2, 64, "f16", 16, VARLEN, seed=95)
    cache, lens, table = on_gpu(p)
    ws = da.alloc_paged_workspace(1, 4, 2, 64)
    q = queries(p, 2, 1, 4, "f16").cuda()
    out = torch.empty_like(q)
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for call in [
        lambda: da.decode_attn_paged(q.cpu(), cache, lens, table, out, ws),
        lambda: da.decode_attn_paged(q, cache, lens.cpu(), table, out, ws),
        lambda: da.decode_attn_paged(q, cache, lens.long(), table, out, ws),
        lambda: da.decode_attn_paged(q, cache, lens[:1], table, out, ws),
        lambda: da.decode_attn_paged(q, cache, lens, table.t(), out, ws),
        lambda: da.decode_attn_paged(q.bfloat16(), cache, lens, table, out.bfloat16(), ws),
        lambda: da.decode_attn_paged(q.float(), cache, lens, table, out.float(), ws),
        lambda: da.decode_attn_paged(q, cache, lens, table, out[:1], ws),
        lambda: da.decode_attn_paged(q[..., :32], cache, lens, table, out, ws),
        lambda: da.decode_attn_paged(q, cache, lens, table, out, ws, lse=torch.empty(2, 4, device="cuda")),
        lambda: da.decode_attn_paged(q, cache, lens, table, out, ws[:1024]),
        lambda: da.decode_attn_paged(q, cache, lens, table, out, ws.cpu()),
        lambda: da.decode_attn_paged_append(None, k, k[:1], cache, cu, lens, table, ws),
        lambda: da.decode_attn_paged_append(None, k.float(), k.float(), cache, cu, lens, table, ws),
        lambda: da.decode_attn_paged_append(k, k, k, cache, cu, lens, table, ws),
        lambda: da.decode_attn_paged_append(None, k, k, cache, cu.long(), lens, table, ws),
        lambda: da.decode_attn_paged_append(None, k, k, cache, cu[:2], lens, table, ws),
        lambda: da.decode_attn_paged_append(None, k.transpose(0, 1), k, cache, cu, lens, table, ws),
        lambda: da.decode_attn_paged_append(None, k, k, cache, cu, lens, table, ws, cos_sin=torch.zeros(30, 24, device="cuda")),
        lambda: da.PagedCache(cache.k.view(torch.float8_e4m3fn), cache.v.view(torch.float8_e4m3fn)),
    ]:
        with pytest.raises((ValueError, TypeError, da.DecodeAttnError)):
            call()
    assert da.decode_attn_splitkv_get_error(ws) == 0
