"""The paged cache's calls where a neighbour must not be touched: units and sequences that are left out between others,
values that a token does not see, weights and scales far below the largest."""
import itertools
import math

import numpy as np
import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_ref import BHSD, DTYPES, VARLEN, Paged, append32, attend64, half_step, table_of, token_view, turned
from test_paged_gpu import _lib, attend, check, fused_rows, on_gpu, queries, same_bits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,layout", [(128, 64, BHSD), (64, 64, VARLEN), (128, 16, VARLEN), (64, 32, BHSD)])
def test_prompts_with_pages_that_are_left_out_between_others(D, page, layout):
    """Every block has several units of several warps, a third of them through table entries outside the cache or past
    cos_sin: the pages and scales of the others come out bit for bit, again and again."""
    Hkv, Hq = 8, 8
    per_block = 256 // (D if page <= 32 else 2 * D)
    n = 3 * 152 * 3 * per_block // (2 * Hkv) * page             # with the others four units and more for each unit's threads
    new = [n, 37, n // 2]
    lens = [n + 5, 37, n // 2]
    p = Paged(lens, Hkv, D, "e4m3", page, layout, seed=100 + page)
    before = {name: getattr(p, name).clone() for name in ("k", "v", "k_scale", "v_scale")}
    q, k, v = fused_rows(sum(new), Hq, Hkv, D, "bf16", 101)
    k, v = (x * torch.exp2(torch.randint(-6, 7, (x.shape[0], 1, 1), generator=torch.Generator().manual_seed(s)).float()).to(x.dtype)
            for s, x in ((102, k), (103, v)))                   # pages of unequal size
    k[::97, 3, 40] = math.inf                                   # (a dim that does not turn) units that look for the largest finite element again
    max_pos = n - 3 * page // 2                                 # sequence 0: a page in part, and whole ones, past cos_sin
    cs = table_of(max_pos, 32)
    lens_written, new_written = [max_pos, 37, n // 2], [max_pos - 5, 37, n // 2]
    keep = torch.cat([torch.arange(max_pos - 5), torch.arange(n, sum(new))])
    append32(p, None, k[keep], v[keep], lens_written, new_written, cs, 2)
    cache_in = Paged(lens, Hkv, D, "e4m3", page, layout, seed=100 + page)
    table = p.table.clone()
    rng = np.random.default_rng(104)
    for b in range(3):
        for i in range(-(-lens[b] // page)):
            if rng.random() < 1 / 3:
                here = int(p.table[b, i])
                for name, x in before.items():
                    getattr(p, name).view(torch.uint8 if x.element_size() == 1 else torch.int32)[here] = \
                        x.view(torch.uint8 if x.element_size() == 1 else torch.int32)[here]
                table[b, i] = [-1, p.k.shape[0], 1 << 30][i % 3]
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device="cuda")
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table, csd, ws = table.cuda(), cs.cuda(), da.alloc_paged_workspace(1, Hq, Hkv, D)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    want = {name: getattr(p, name).cuda() for name in before}
    for _ in range(10):
        cache, _, _ = on_gpu(cache_in)
        da.decode_attn_paged_append(qd, kd, vd, cache, cu, kv_lens, table, ws, cos_sin=csd, rope=2, q_out=torch.empty_like(qd))
        for name, x in want.items():
            raw = torch.uint8 if x.element_size() == 1 else torch.int32
            assert torch.equal(getattr(cache, name).view(raw), x.view(raw)), name
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_PAGE | da.DA_DEVERR_POSITION


@pytest.mark.parametrize("kv,value", [("bf16", math.nan), ("bf16", -math.inf), ("f16", math.nan), ("f16", math.inf), ("e4m3", math.nan)])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,layout,longest", [
    (4, 4, 2, 128, 64, BHSD, 700), (4, 8, 2, 64, 16, VARLEN, 1100), (16, 2, 2, 64, 48, BHSD, 700), (5, 6, 2, 128, 32, VARLEN, 700),
    (4, 4, 2, 128, 64, VARLEN, 1100), (3, 16, 2, 128, 128, BHSD, 1100), (16, 4, 2, 128, 256, VARLEN, 1100)])
def test_values_of_later_tokens_that_are_not_finite(kv, value, T, Hq, Hkv, D, page, layout, longest):
    """A NaN or an infinity among the values of a key reaches the query tokens that see the key and no other, wherever
    the last keys lie in their box, stage and page: sequences that end everywhere in a stage, one shorter than its query
    tokens, one in several pieces. (16-bit pages of head size 128 have four consumer warps up to 1023 keys, then eight.)"""
    lens = [130, 128, 129, 127, 66, 65, 18, 17, 16, 2, longest, T]
    spoilt = {(b, n - 1 - (b * 5) % min(T, n)) for b, n in enumerate(lens)} | {(0, 129), (10, longest - T), (4, 65), (4, 64)}
    p = Paged(lens, Hkv, D, kv, page, layout, seed=110)
    rng = np.random.default_rng(111)
    where = [(b, j, int(rng.integers(Hkv)), int(rng.integers(D))) for b, j in sorted(spoilt)]
    code = 0x7F if kv == "e4m3" else int(torch.tensor(value).to(p.v.dtype).view(torch.int16))
    raw = token_view(p.v.view(torch.uint8 if kv == "e4m3" else torch.int16), layout)
    sound = p.v.clone()
    for b, j, h, d in where:
        raw[p.table[b, j // page].long(), j % page, h, d] = code
    q = queries(p, len(lens), T, Hq, "f16" if kv == "f16" else "bf16", 112)
    out, lse, err = attend(p, q)
    assert err == 0
    p.v = sound
    ref = attend64(q, p)
    hit = np.zeros(out.shape, dtype=bool)
    for b, j, h, d in where:
        for t in range(T):
            if j <= lens[b] - T + t:
                hit[b, t, h * Hq // Hkv:(h + 1) * Hq // Hkv, d] = True
    assert hit.any() and not np.isfinite(out[hit]).any()
    assert np.isnan(out[hit]).all() or math.isinf(value) and (out[hit] == value).all()
    out[hit] = ref[0][hit]
    check(out, lse, ref, "f16" if kv == "f16" else "bf16")


@pytest.mark.parametrize("lens", [[200, 7, 64], [1, 3000]])
@pytest.mark.parametrize("power", [-149, -140, -130, -126, 100])
def test_value_scales_from_the_least_float_on(power, lens):
    """Outputs follow the value scales, powers of two, down to subnormal ones (bf16 outputs reach as far). Relative to
    the same values at scale 1, whose tolerance is scaled alike; float32 itself ends at 2^-149."""
    p = Paged(lens, 2, 128, "e4m3", 64, BHSD, seed=120)
    p.v_scale.masked_fill_(~p.v_scale.isnan(), 1.0)
    q = queries(p, len(lens), 2, 8, "bf16", 121)
    ro, rl, to, tl = attend64(q, p)
    p.v_scale.masked_fill_(~p.v_scale.isnan(), 2.0 ** power)
    out, lse, err = attend(p, q)
    assert err == 0
    s = 2.0 ** power
    off = np.abs(out - ro * s) - half_step(ro * s, torch.bfloat16) - to * s - 4 * 2.0 ** -149
    assert np.all(off <= 0), off.max()
    assert np.abs(out).max() > 0 or 448 * s < 2.0 ** -134       # below half of the least bfloat16 everything is 0
    check(ro, lse, (ro, rl, to, tl), "bf16")


@pytest.mark.parametrize("kv,Hq,T,D,n", [("f16", 4, 1, 128, 40000), ("f16", 16, 1, 128, 9000), ("f16", 2, 1, 64, 20000), ("f16", 8, 2, 64, 900),
                                         ("f16", 2, 1, 128, 1000), ("e4m3", 4, 1, 128, 40000), ("e4m3", 4, 4, 128, 9000),
                                         ("e4m3", 2, 1, 64, 20000)])
@pytest.mark.parametrize("below", [13.3, 20.3, 24.5, 27.0, 31.7, 34.0])
def test_many_keys_far_below_a_few_with_small_values(kv, Hq, T, D, n, below):
    """Attention sinks: every sixteenth key outweighs the others by 2^`below` and has values of zero, so that the output
    is what the others leave. Relative to that, a weight is off by a rounding to fp16, 2^-11, or, below 2^-25 of the
    largest, by half of 2^-35 of that one (fp16 ends at 2^-24, the weights enter as 2^11 times theirs; with more than
    eight columns over 8-bit pages as 2^7 times theirs, hence 2^-31); its score by 2^-21 a unit; sums of n terms by
    n 2^-24."""
    p = Paged([n], 1, D, kv, 64, BHSD, seed=130)
    sink = torch.zeros(p.k.shape[0], p.page, dtype=torch.bool)
    for j in range(3, n, 16):
        sink[p.table[0, j // p.page].long(), j % p.page] = True
    values = (torch.rand(p.v.shape, generator=torch.Generator().manual_seed(131)) + 0.5) * (20000 if kv == "f16" else 200)
    values[(sink[:, None, :, None]).expand_as(values)] = 0
    p.v = values.to(p.v.dtype)
    p.k = sink[:, None, :, None].expand(p.k.shape).float().to(p.k.dtype).contiguous()
    if kv == "e4m3":
        p.k_scale.fill_(1.0)
        p.v_scale.fill_(2.0)
    q_type = "f16" if kv == "f16" else "bf16"
    q = torch.ones(1, T, Hq, D, dtype=DTYPES[q_type])
    scale = float(np.float32(below * math.log(2) / D))
    out, lse, err = attend(p, q, scale=scale)
    assert err == 0
    v = p.sequence(0)[1][:, 0].numpy()
    for t in range(T):
        m = n - T + 1 + t
        heavy = len(range(3, m, 16))
        w = math.exp(-scale * D)
        ref = w * v[:m].sum(0) / (heavy + (m - heavy) * w)
        rel = max(2.0 ** -11, 2.0 ** (-32 if kv == "e4m3" and Hq * T > 8 else -36) / w) + 2.0 ** -21 * (1 + 2 * below) + 2 * m * 2.0 ** -24
        off = np.abs(out[0, t] - ref) - half_step(ref, DTYPES[q_type]) - rel * ref
        assert np.all(off <= 0), (t, (np.abs(out[0, t] - ref) / ref).max(), rel)
        assert np.all(np.abs(lse[0, t] - (scale * D + math.log(heavy + (m - heavy) * w))) <= 2.0 ** -20 * (1 + below) + m * 2.0 ** -24)


@pytest.mark.parametrize("kv", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,width", [(1, 8, 2, 128, None), (1, 8, 2, 128, 20), (4, 6, 2, 128, None), (4, 6, 2, 128, 20),
                                              (1, 8, 2, 64, None), (5, 8, 4, 64, None)])
def test_weights_of_16_bit_pages_keep_more_bits_than_the_pages(kv, T, Hq, Hkv, D, width):
    """The output is off by its own rounding and little else: a weight enters as the sum of two 16-bit values, the first
    rounded down: off by 2^-15 of itself in bf16 (2^-8 of what that leaves, 2^-7) and by 2^-20 for the second's sign, by 2^-21
    (2^-11 of 2^-10) and 2^-34 of the largest in fp16. Small queries, so that the bound of the scores' error is no larger."""
    lens = [5, 6, 7, 9, 12, 17, 40, 3, 100]
    p = Paged(lens, Hkv, D, kv, 64, BHSD, seed=140, width=width)
    q = queries(p, len(lens), T, Hq, kv, 141, size=0.02)
    out, lse, err = attend(p, q)
    assert err == 0
    ro, rl, to, tl = attend64(q, p)
    # attend64's bound without its term for the weights' one rounding, 2^-8 or 2^-11 of the largest value
    once, twice = (2.0 ** -8, 2.0 ** -15 + 2.0 ** -20) if kv == "bf16" else (2.0 ** -11, 2.0 ** -21 + 2.0 ** -34)
    for b in range(len(lens)):
        v = p.sequence(b)[1].abs().numpy()
        for t, h in itertools.product(range(T), range(Hq)):
            n = lens[b] - T + t + 1
            if n > 0:
                to[b, t, h] -= (once - twice) * v[:n, h * Hkv // Hq].max()
    check(out, lse, (ro, rl, to, tl), kv)


def test_numbers_that_are_none_of_their_c_types():
    """Refused as other arguments are: a scale past float32, or none at all, and a rotation that is no integer."""
    p = Paged([20, 9], 2, 64, "f16", 16, VARLEN, seed=150)
    cache, lens, table = on_gpu(p)
    ws = da.alloc_paged_workspace(1, 4, 2, 64)
    q = queries(p, 2, 1, 4, "f16").cuda()
    out = torch.full_like(q, 7.0)
    for scale in (1e39, -1e300, "0.1", 1 + 2j, math.inf, math.nan):
        with pytest.raises((ValueError, TypeError, da.DecodeAttnError)):
            da.decode_attn_paged(q, cache, lens, table, out, ws, scale=scale)
    k = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    before = cache.k.clone()
    for rope in ("half", 1 << 40, None):
        with pytest.raises((ValueError, TypeError)):
            da.decode_attn_paged_append(None, k, k, cache, cu, lens, table, ws, cos_sin=table_of(32, 64).cuda(), rope=rope)
    assert torch.all(out == 7.0) and torch.equal(cache.k.view(torch.int16), before.view(torch.int16))
    assert da.decode_attn_splitkv_get_error(ws) == 0


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("bounds,done,claimed_twice", [
    ([0, 3, 2, 5], {0: range(0, 3), 2: range(2, 5)}, 2), ([0, 2, 3, 9], {0: range(0, 2), 1: range(2, 3)}, None),
    ([-1, 2, 3, 5], {1: range(2, 3), 2: range(3, 5)}, None), ([1 << 30, -(1 << 31), 4, 5], {2: range(4, 5)}, None),
    ([0, 2, 5, 5], {0: range(0, 2), 1: range(2, 5)}, None), ([0, 5, 6, 5], {0: range(0, 5)}, None)])
def test_rows_of_sequences_that_cannot_be(kv, bounds, done, claimed_twice):
    """cu_new that decreases or leaves the rows: what the other sequences append is right, and nothing else changes, in the
    pages, the scales, the rotated queries, and memory around them. (A row that two sequences claim, and the page that
    one of them has for it, are left aside.)"""
    dt = "bf16" if kv == "bf16" else "f16"
    lens = [10, 10, 10]
    p = Paged(lens, 2, 64, kv, 16, VARLEN, seed=160)
    q, k, v = fused_rows(5, 4, 2, 64, dt, 161)
    cs = table_of(16, 64)
    cache, kv_lens, table = on_gpu(p)
    n = p.k.shape[0]
    raw = torch.uint8 if kv == "e4m3" else torch.int16
    guarded = []
    for x in (cache.k, cache.v):                                # pages with as many guard pages on either side
        big = torch.full((3 * n, *x.shape[1:]), 0x55, dtype=raw, device="cuda").view(x.dtype)
        big.view(raw)[n:2 * n] = x.view(raw)
        guarded.append(big)
    cache = da.PagedCache(*(x[n:2 * n] for x in guarded), cache.k_scale, cache.v_scale, layout=VARLEN)
    out = torch.full((15, 4, 64), -3.0, dtype=DTYPES[dt], device="cuda")
    ws = da.alloc_paged_workspace(1, 4, 2, 64)
    da.decode_attn_paged_append(q.cuda(), k.cuda(), v.cuda(), cache, torch.tensor(bounds, dtype=torch.int32, device="cuda"), kv_lens,
                                table, ws, cos_sin=cs.cuda(), q_out=out[5:10])
    err = da.decode_attn_splitkv_get_error(ws)
    assert err == (0 if bounds[-2:] == [5, 5] else da.DA_DEVERR_SEQLENS)
    out = out.cpu()
    tables = p.table
    left_alone = set(range(15))
    for b, rows in done.items():
        r = torch.tensor(list(rows))
        at = torch.arange(10 - len(rows), 10)
        p.table = tables[b:b + 1]
        append32(p, None, k[r], v[r], [10], [len(rows)], cs, 1)
        want = turned(q[r], cs, at, 1, torch.float32).to(q.dtype)
        for i, row in enumerate(rows):
            left_alone.discard(5 + row)
            if row != claimed_twice:
                assert same_bits(out[5 + row], want[i]), row
    assert torch.all(out[sorted(left_alone)] == -3.0)
    same = torch.ones(n, dtype=torch.bool)
    if claimed_twice is not None:
        same[tables[2, 0].long()] = False
    for name, big in zip(("k", "v"), guarded):
        assert torch.all(big.view(raw)[:n] == 0x55) and torch.all(big.view(raw)[2 * n:] == 0x55)
        assert torch.equal(big.view(raw)[n:2 * n].cpu()[same], getattr(p, name).view(raw)[same]), name
        if kv == "e4m3":
            assert same_bits(getattr(cache, name + "_scale").cpu()[same], getattr(p, name + "_scale")[same])
