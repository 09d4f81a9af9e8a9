"""The paged cache's calls where a neighbour must not be touched: units and sequences that are left out between others,
values that a token does not see, weights and scales far below the largest."""
import itertools
import math

import numpy as np
import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_ref import BHSD, VARLEN, Paged, append32, table_of
from test_paged_gpu import _lib, fused_rows, on_gpu  # noqa: F401

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
