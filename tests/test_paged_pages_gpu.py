"""Forking, freeing and compacting pages against plain Python."""
import random

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, queries
from paged_ref import BHSD, VARLEN, Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.load()


KV = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def pool(lens, num_pages, page, Hkv, D, kv, layout, seed=0, shared=0.0, width=None):
    """A cache of random bits, and a table over scattered pages; `shared`: chance that a row begins with another's pages."""
    rng = random.Random(seed)
    order = list(range(num_pages))
    rng.shuffle(order)
    need = [-(-n // page) for n in lens]
    rows = []
    for n in need:
        row = list(rng.choice(rows))[:rng.randint(0, n)] if rows and rng.random() < shared else []
        while len(row) < n:
            row.append(order.pop())
        rows.append(row)
    width = max([1] + need) if width is None else width
    table = torch.tensor([r + [-5] * (width - len(r)) for r in rows], dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    inner = (page, Hkv) if layout == VARLEN else (Hkv, page)
    size = 1 if kv == "e4m3" else 2

    def pages():
        raw = torch.randint(0, 256, (num_pages, *inner, D * size), generator=g, dtype=torch.uint8).cuda()
        return raw.view(KV[kv])

    scales = [torch.rand(num_pages, Hkv, generator=g).cuda() for _ in range(2)] if kv == "e4m3" else [None, None]
    return da.PagedCache(pages(), pages(), *scales, layout=layout), table, rows, order


def raw(x):
    return x.view(torch.uint8).cpu()


def tokens(x, layout):
    return x if layout == VARLEN else x.transpose(1, 2)


CASES = [([100, 1, 0, 64, 63, 65], 40, 16), ([1000, 0, 700], 90, 32), ([1], 1, 16), ([0], 3, 64), ([5, 2000], 9, 256), ([300] * 300, 7000, 16),
         ([17] * 2000, 9000, 16)]


@pytest.mark.parametrize("lens,num_pages,page", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("shared", [0.0, 0.7])
def test_free_pages(lens, num_pages, page, shared):
    cache, table, rows, _ = pool(lens, num_pages, page, 1, 64, "f16", VARLEN, seed=num_pages, shared=shared)
    ws = da.alloc_paged_pages_workspace(num_pages)
    free = torch.full((num_pages,), -9, dtype=torch.int32, device="cuda")
    count = ints([-1])
    for _ in range(2):
        da.decode_attn_paged_free_pages(ints(lens), table.cuda(), free, count, ws, page_size=page)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    used = {p for r in rows for p in r}
    want = [p for p in range(num_pages) if p not in used]
    assert count.item() == len(want)
    assert free.tolist() == want + [-9] * (num_pages - len(want))


@pytest.mark.parametrize("num_pages,B,width", [(1 << 20, 1000, 40), (300001, 1, 200000), (262144, 3, 20), (262145, 3, 20), (31, 1, 32768), (33, 1, 32769)])
def test_free_pages_of_large_pools(num_pages, B, width):
    """Around the sizes from which several blocks do the work."""
    g = torch.Generator().manual_seed(num_pages)
    lens = torch.randint(0, min(width, num_pages // B) * 16 + 1, (B,), generator=g, dtype=torch.int32)
    order = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // 16)
        table[b, :n] = order[at:at + n]
        at += n
    ws = da.alloc_paged_pages_workspace(num_pages)
    free, count = torch.full((num_pages,), -9, dtype=torch.int32, device="cuda"), ints([-1])
    da.decode_attn_paged_free_pages(lens.cuda(), table.cuda(), free, count, ws, page_size=16)
    want = torch.sort(order[at:]).values
    assert count.item() == num_pages - at
    assert torch.equal(free[:num_pages - at].cpu(), want) and (free[num_pages - at:] == -9).all()
    assert da.decode_attn_splitkv_get_error(ws) == 0


@pytest.mark.parametrize("lens,num_pages,page", CASES[:6], ids=[str(i) for i in range(6)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", [VARLEN, BHSD])
@pytest.mark.parametrize("shared", [0.0, 0.7])
def test_compact(lens, num_pages, page, kv, layout, shared):
    cache, table, rows, _ = pool(lens, num_pages, page, 2, 64, kv, layout, seed=num_pages + 1, shared=shared)
    before = [raw(cache.k), raw(cache.v)] + ([cache.k_scale.cpu(), cache.v_scale.cpu()] if kv == "e4m3" else [])
    used = sorted({p for r in rows for p in r})
    n, taken = len(used), set(used)
    moves = dict(zip([p for p in used if p >= n], [p for p in range(n) if p not in taken]))
    ws = da.alloc_paged_pages_workspace(num_pages)
    out = torch.full((len(lens), table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
    count = ints([-1])
    for _ in range(2):   # repeated on the old table it moves the same pages to the same places
        da.decode_attn_paged_compact(cache, ints(lens), table.cuda(), out, count, ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    assert count.item() == n
    for b, r in enumerate(rows):
        assert out[b].tolist() == [moves.get(p, p) for p in r] + [-9] * (out.shape[1] - len(r))
    after = [raw(cache.k), raw(cache.v)] + ([cache.k_scale.cpu(), cache.v_scale.cpu()] if kv == "e4m3" else [])
    for x, y in zip(before, after):
        x = x.clone()
        for a, b in moves.items():
            x[b] = x[a]
        assert torch.equal(x, y)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
@pytest.mark.parametrize("layout", [VARLEN, BHSD])
@pytest.mark.parametrize("page,Hkv,D", [(16, 1, 64), (48, 3, 128), (1024, 2, 64)])
def test_fork(page, Hkv, D, kv, layout):
    lens = [5 * page // 2, page, 0, 1, 3 * page - 1, 2 * page + 16]
    cache, table, rows, order = pool(lens, 40, page, Hkv, D, kv, layout, seed=page)
    parents = [0, 0, 4, 2, 3, 1, 0, 5, 5, 4]
    fresh = [order[0], -1, order[1], order[2], order[3], order[4], -7, order[5], -1, order[6]]
    before = [raw(cache.k), raw(cache.v)]
    scales = [cache.k_scale.cpu(), cache.v_scale.cpu()] if kv == "e4m3" else []
    ws = da.alloc_paged_pages_workspace(40)
    out = torch.full((10, table.shape[1] + 2), -9, dtype=torch.int32, device="cuda")[:, :table.shape[1] + 1]
    got = ints([-1] * 10)
    for _ in range(2):
        da.decode_attn_paged_fork(cache, ints(lens), table.cuda(), ints(parents), ints(fresh), got, out, ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    assert got.tolist() == [lens[p] for p in parents]
    for i, (p, f) in enumerate(zip(parents, fresh)):
        row, part = list(rows[p]), lens[p] % page
        if part and f >= 0:
            for j, x in enumerate(before):
                tokens(x, layout)[f, :part] = tokens(x, layout)[row[-1], :part]
            for x in scales:
                x[f] = x[row[-1]]
            row[-1] = f
        assert out[i].tolist() == row + [-9] * (out.shape[1] - len(row))
    assert torch.equal(before[0], raw(cache.k)) and torch.equal(before[1], raw(cache.v))
    if scales:
        assert torch.equal(scales[0], cache.k_scale.cpu()) and torch.equal(scales[1], cache.v_scale.cpu())


def test_what_cannot_be_is_flagged():
    cache, table, rows, order = pool([100, 40], 20, 16, 1, 64, "f16", VARLEN, seed=3)
    ws = da.alloc_paged_pages_workspace(20)
    out, got = torch.full((3, 7), -9, dtype=torch.int32, device="cuda"), ints([-1] * 3)
    k = raw(cache.k)
    # parents that are none
    da.decode_attn_paged_fork(cache, ints([100, 40]), table.cuda(), ints([-1, 2, 1]), ints([order[0], order[1], -1]), got, out, ws)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_SEQLENS
    assert got.tolist() == [0, 0, 40] and (out[:2] == -9).all() and out[2].tolist() == rows[1] + [-9] * 4
    # a new page outside the cache is not written
    da.decode_attn_paged_fork(cache, ints([100, 40]), table.cuda(), ints([0]), ints([20]), got[:1], out[:1], ws)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_PAGE
    assert out[0].tolist() == rows[0][:-1] + [20] and torch.equal(raw(cache.k), k)
    # a length that does not fit
    free, count = torch.full((20,), -9, dtype=torch.int32, device="cuda"), ints([0])
    da.decode_attn_paged_free_pages(ints([100, 113]), table.cuda(), free, count, ws, page_size=16)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_SEQLENS
    assert count.item() == 13 and sorted(free.tolist()[:13] + rows[0]) == list(range(20))
    # entries outside the cache: no page of it is in use by them, and they stay what they are
    bad = table.clone()
    bad[0, 2], bad[1, 0] = 20, -3
    out2 = torch.full((2, 7), -9, dtype=torch.int32, device="cuda")
    da.decode_attn_paged_compact(cache, ints([100, 40]), bad.cuda(), out2, count, ws)
    assert da.decode_attn_splitkv_get_error(ws) == da.DA_DEVERR_PAGE
    assert count.item() == 8 and out2[0, 2] == 20 and out2[1, 0] == -3
    keep = [p for p in out2.flatten().tolist() if 0 <= p < 20]
    assert sorted(keep) == list(range(8))


def test_a_large_pool_moves_half_its_pages():
    lens = [1600] * 50
    cache, table, rows, _ = pool(lens, 10000, 16, 1, 64, "e4m3", BHSD, seed=4)
    k, v, ks = raw(cache.k), raw(cache.v), cache.k_scale.cpu()
    ws = da.alloc_paged_pages_workspace(10000)
    out, count = torch.zeros(50, 100, dtype=torch.int32, device="cuda"), ints([0])
    da.decode_attn_paged_compact(cache, ints(lens), table.cuda(), out, count, ws)
    assert count.item() == 5000 and sorted(out.flatten().tolist()) == list(range(5000))
    new = out.flatten().long().cpu()
    old = table.flatten().long()
    assert torch.equal(raw(cache.k)[new], k[old]) and torch.equal(raw(cache.v)[new], v[old])
    assert torch.equal(cache.k_scale.cpu()[new], ks[old])


def test_as_a_server_uses_them_together():
    """A prompt, three answers that continue it, an answer that ends, compaction; attention sees the same keys all along."""
    Hq, Hkv, D, P = 4, 2, 64, 16
    paged = Paged([77, 130], Hkv, D, "bf16", P, VARLEN, seed=5, extra_pages=30)
    cache = da.PagedCache(paged.k.cuda(), paged.v.cuda(), layout=VARLEN)
    n = cache.num_pages
    ws, aws = da.alloc_paged_pages_workspace(n), da.alloc_paged_chunk_workspace(Hq, Hkv, D)
    lens = ints(paged.lens)
    table = torch.zeros(2, 12, dtype=torch.int32, device="cuda")
    table[:, :paged.table.shape[1]] = paged.table.cuda()
    free, count = torch.empty(n, dtype=torch.int32, device="cuda"), ints([0])
    da.decode_attn_paged_free_pages(lens, table, free, count, ws, page_size=P)
    # three answers to the first prompt, the second goes on alone; the new pages come from the list on the device
    fresh = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    fresh[:2] = free[:2]
    lens2, table2 = ints([0] * 4), torch.zeros(4, 12, dtype=torch.int32, device="cuda")
    da.decode_attn_paged_fork(cache, lens, table, ints([0, 0, 0, 1]), fresh, lens2, table2, ws)
    # each gets a token of its own
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(4, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    lens2 += 1
    da.decode_attn_paged_append(None, k.cuda(), v.cuda(), cache, ints(list(range(5))), lens2, table2, aws)
    q = queries(4, Hq, D, "bf16", 7)

    def attend(lens, table, q):
        out, lse = torch.empty(len(lens), Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(len(lens), Hq, device="cuda")
        da.decode_attn_paged_chunk(q.cuda(), cache, ints(list(range(len(lens) + 1))), lens, table, out, aws, lse=lse)
        assert da.decode_attn_splitkv_get_error(aws) == 0
        return out, lse

    out, lse = attend(lens2, table2, q)
    for i, parent in enumerate([0, 0, 0, 1]):
        one = Paged([paged.lens[parent] + 1], Hkv, D, "bf16", P, VARLEN, seed=8)
        pk, pv = paged.sequence(parent)
        for p in range(paged.lens[parent] + 1):
            at = (int(one.table[0, p // P]), p % P)
            one.k[at] = pk[p].to(torch.bfloat16) if p < len(pk) else k[i]
            one.v[at] = pv[p].to(torch.bfloat16) if p < len(pv) else v[i]
        assert check(out[i:i + 1], lse[i:i + 1], chunk64(q[i:i + 1], one, [1]), torch.bfloat16) is None
    # the second answer ends; the rest moves to the front
    lens2[1] = 0
    table3 = torch.zeros_like(table2)
    da.decode_attn_paged_compact(cache, lens2, table2, table3, count, ws)
    assert da.decode_attn_splitkv_get_error(ws) == 0
    used = count.item()
    live = [table3[b, :-(-int(lens2[b]) // P)].tolist() for b in range(4)]
    assert sorted({p for r in live for p in r}) == list(range(used))
    again, _ = attend(lens2, table3, q)
    assert torch.equal(again[[0, 2, 3]], out[[0, 2, 3]]) and (again[1] == 0).all()
