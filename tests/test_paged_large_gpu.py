"""Caches whose elements lie past 32 bits: chunk and windowed attention, forking and compacting."""
import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import check, chunk64
from paged_more_util import ints, queries, starts
from paged_ref import BHSD, VARLEN, Paged, token_view

pytestmark = pytest.mark.gpu
PAGES, P, Hkv, D = 150000, 64, 4, 128          # 2^32.2 elements, 9.8 GB a tensor in 16 bits


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    da.build()
    da.load()


@pytest.mark.parametrize("layout", [VARLEN, BHSD])
def test_pages_past_32_bits(layout):
    paged = Paged([700, 333], Hkv, D, "bf16", P, layout, seed=1)
    inner = (P, Hkv) if layout == VARLEN else (Hkv, P)
    k, v = (torch.empty(PAGES, *inner, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 32
    n = paged.k.shape[0]
    high = PAGES - n                       # the small cache's pages, at the end of the large one
    k[high:], v[high:] = paged.k.cuda(), paged.v.cuda()
    cache = da.PagedCache(k, v, layout=layout)
    need = [-(-m // P) for m in paged.lens]
    table = torch.zeros(2, max(need), dtype=torch.int32)
    for b, m in enumerate(need):
        table[b, :m] = paged.table[b, :m] + high
    new = [65, 1]
    q = queries(66, 8, D, "bf16", 2)

    def attend(table, window=0, sinks=0):
        ws = da.alloc_paged_chunk_workspace(8, Hkv, D)
        out, lse = torch.empty(66, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(66, 8, device="cuda")
        da.decode_attn_paged_chunk(q.cuda(), cache, ints(starts(new)), ints(paged.lens), table, out, ws, window=window, sinks=sinks, lse=lse)
        assert da.decode_attn_splitkv_get_error(ws) == 0
        return out, lse

    for window, sinks in ((0, 0), (100, 5)):
        assert check(*attend(table.cuda(), window, sinks), chunk64(q, paged, new, None, window, sinks), torch.bfloat16) is None
    ws = da.alloc_paged_workspace(1, 8, Hkv, D)
    one = queries(2, 8, D, "bf16", 3)
    out, lse = torch.empty(2, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")
    da.decode_attn_paged_window(one.cuda(), cache, ints(paged.lens), table.cuda(), out, ws, window=200, sinks=3, lse=lse)
    assert check(out, lse, chunk64(one, paged, [1, 1], None, 200, 3), torch.bfloat16) is None
    # a row of its own for a copy of the first sequence, from and to pages past 32 bits
    pws = da.alloc_paged_pages_workspace(PAGES)
    spare = high - 7
    lens2, table2 = ints([0, 0]), torch.zeros(2, max(need), dtype=torch.int32, device="cuda")
    da.decode_attn_paged_fork(cache, ints(paged.lens), table.cuda(), ints([0, 1]), ints([spare, -1]), lens2, table2, pws)
    part = 700 % P
    old = int(table[0, need[0] - 1])
    for x in (k, v):
        assert torch.equal(token_view(x, layout)[spare, :part].view(torch.int16), token_view(x, layout)[old, :part].view(torch.int16))
    want = chunk64(q, paged, new)
    assert table2[0, need[0] - 1] == spare and check(*attend(table2), want, torch.bfloat16) is None
    # and everything to the front
    table3, count = torch.zeros_like(table2), ints([0])
    da.decode_attn_paged_compact(cache, lens2, table2, table3, count, pws)
    assert da.decode_attn_splitkv_get_error(pws) == 0
    assert count.item() == sum(need) and sorted(table3[0, :need[0]].tolist() + table3[1, :need[1]].tolist()) == list(range(sum(need)))
    assert check(*attend(table3), want, torch.bfloat16) is None
