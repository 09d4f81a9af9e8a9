"""Helpers of the GPU tests of chunk and windowed attention: pages on the device, calls, guards."""
import itertools

import torch

import split_kv_decode_decoding_gb300 as da
from paged_ref import DTYPES


def on_device(paged):
    scales = (None, None) if paged.k_scale is None else (paged.k_scale.cuda(), paged.v_scale.cuda())
    return da.PagedCache(paged.k.cuda(), paged.v.cuda(), *scales, layout=paged.layout)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(new):
    return [0, *itertools.accumulate(new)]


def queries(rows, Hq, D, dtype, seed=0, mean=0.0):
    return (torch.randn(rows, Hq, D, generator=torch.Generator().manual_seed(seed)) + mean).to(DTYPES[dtype])


def run_chunk(q, paged, new, cache=None, scale=None, window=0, sinks=0, workspace=None, stream=None, lens=None, expect=0, extra=3):
    """One call with `extra` rows behind the last sequence, which have to stay as they were; (out, lse)."""
    cache = on_device(paged) if cache is None else cache
    T, Hq, D = q.shape
    ws = da.alloc_paged_chunk_workspace(Hq, cache.Hkv, D) if workspace is None else workspace
    qd = torch.cat([q, q.new_full((extra, Hq, D), float("nan"))]).cuda()
    out = torch.full_like(qd, 7.0)
    lse = torch.full((T + extra, Hq), 7.0, device="cuda")
    table = paged.table.cuda() if paged.table.shape[1] else ints([[0]] * len(new))
    da.decode_attn_paged_chunk(qd, cache, ints(starts(new)), ints(paged.lens if lens is None else lens), table, out, ws, scale=scale,
                               window=window, sinks=sinks, lse=lse, stream=stream)
    assert da.decode_attn_splitkv_get_error(ws) == expect
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()
    return out[:T], lse[:T]


def unseen_entries(paged, new, window, sinks):
    """Take away the pages that no token sees: their block-table entries become invalid, their contents NaN."""
    P = paged.page
    kept = set()
    for b, (n, m) in enumerate(zip(paged.lens, new)):
        low = max(0, max(0, n - m) - window + 1)
        for i in range(-(-n // P)):
            if (i + 1) * P > low or i * P < sinks:
                kept.add((b, i))
    gone = [int(paged.table[b, i]) for b, n in enumerate(paged.lens) for i in range(-(-n // P)) if (b, i) not in kept]
    for b, n in enumerate(paged.lens):
        for i in range(-(-n // P)):
            if (b, i) not in kept:
                paged.table[b, i] = -7 if i % 2 else 1 << 30
    for x in (paged.k, paged.v):
        raw = x.view(torch.uint8 if paged.kv == "e4m3" else torch.int16)
        raw[gone] = 0x7F if paged.kv == "e4m3" else 0x7FFF
    return gone
