"""Chunk and windowed attention and the page operators on the host: sizes and refusals. Every case is answered by the
host-side checks, before any CUDA call."""
import ctypes
import math
import os
import re
import struct
import subprocess

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_more_ref import chunk64, sees
from paged_ref import VARLEN, Paged, attend64
from test_paged_host import ATTEND, BAD_CACHE, HEADER, cache_struct

ARG, UNSUP, ALIGN, SMALL = da.DA_ERR_INVALID_ARG, da.DA_ERR_UNSUPPORTED, da.DA_ERR_ALIGNMENT, da.DA_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    da.build()
    return da.load()


# addresses that are never followed: the calls below are refused before any device work
CHUNK = dict(q=5 << 20, q_stride=1024, cu=13 << 20, lens=6 << 20, table=7 << 20, max_pages=4, table_stride=4, B=2, T=2, Hq=8, dtype=0,
             scale=0.1, window=0, sinks=0, out=8 << 20, out_stride=1024, lse=0, ws=9 << 20, ws_bytes=1 << 30)
ROWS = dict(lens=6 << 20, table=7 << 20, max_pages=4, table_stride=4, B=2, page_size=64, num_pages=10, ws=9 << 20, ws_bytes=1 << 30)


def chunk(lib, cache={}, **change):
    from split_kv_decode_decoding_gb300.paged import _pack_chunk
    a = {**CHUNK, **change}
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged_chunk(
        _pack_chunk(a["q"], a["q_stride"], 0 if c is None else ctypes.addressof(c), a["cu"], a["lens"], a["table"], a["max_pages"],
                    a["table_stride"], a["B"], a["T"], a["Hq"], a["dtype"], a["scale"], a["window"], a["sinks"], a["out"],
                    a["out_stride"], a["lse"], a["ws"], a["ws_bytes"]), None)


def window(lib, window=10, sinks=0, cache={}, **change):
    from split_kv_decode_decoding_gb300.paged import _pack_attn
    a = {**ATTEND, **change}
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged_window(
        _pack_attn(a["q"], 0 if c is None else ctypes.addressof(c), a["lens"], a["table"], a["max_pages"], a["table_stride"], a["B"],
                   a["T_q"], a["Hq"], a["dtype"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"]), window, sinks, None)


def rows(**change):
    from split_kv_decode_decoding_gb300.paged import _pack_rows
    a = {**ROWS, **change}
    return _pack_rows(a["lens"], a["table"], a["max_pages"], a["table_stride"], a["B"], a["page_size"], a["num_pages"], a["ws"], a["ws_bytes"])


def free(lib, out=20 << 20, count=21 << 20, **change):
    return lib.decode_attn_paged_free_pages(rows(**change), out, count, None)


def fork(lib, cache={}, parents=22 << 20, fresh=23 << 20, n=3, lens_out=24 << 20, table_out=25 << 20, out_stride=4, **change):
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged_fork(rows(**change), None if c is None else ctypes.addressof(c), parents, fresh, n, lens_out, table_out,
                                      out_stride, None)


def compact(lib, cache={}, table_out=25 << 20, out_stride=4, count=21 << 20, **change):
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged_compact(rows(**change), None if c is None else ctypes.addressof(c), table_out, out_stride, count, None)


def test_packed_structs_lie_as_the_header_declares(tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    from split_kv_decode_decoding_gb300 import paged
    for name, fmt in (("da_paged_chunk", "@PqPPPPiiiiiifiiPqPPN"), ("da_paged_rows", "@PPiiiiiPN")):
        assert getattr(paged, "_pack_" + name.rsplit("_", 1)[1]).__self__.format == fmt
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        fields = [w.strip(" *") for d in body.split(";") if d.strip() for w in re.sub(r"^\s*(const\s+)?\w+", "", d.strip()).split(",")]
        assert len(fields) == len(fmt) - 1
        src = tmp_path / (name + ".c")
        src.write_text('#include <stdio.h>\n#include "decode_attn_paged.h"\nint main(void) {\n' + "".join(
            f'printf("%zu ", offsetof({name}, {f}));\n' for f in fields) + f'printf("%zu", sizeof({name}));\nreturn 0; }}\n')
        exe = tmp_path / name
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), "-o", str(exe), str(src)], check=True)
        got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        want = [struct.calcsize(fmt[:i + 1] + "0" + fmt[i + 1]) for i in range(len(fields))]
        assert got[:-1] == want and got[-1] == struct.calcsize(fmt + "0P")
    assert int(re.search(r"#define DA_MAX_PAGED_ROWS (\d+)", text).group(1)) == da.DA_MAX_PAGED_ROWS


def test_workspace_sizes(lib):
    small, large = da.paged_chunk_workspace_size(8, 8, 64), da.paged_chunk_workspace_size(128, 8, 128)
    assert 0 < small < large <= 64 << 20
    assert da.paged_chunk_workspace_size(8, 2, 128) == large                 # any heads
    for bad in ((30, 8, 128), (32, 0, 128), (0, 1, 128), (32, 8, 96), (-8, 8, 128)):
        assert da.paged_chunk_workspace_size(*bad) == 0, bad
        with pytest.raises(ValueError):
            da.alloc_paged_chunk_workspace(*bad, device="cpu")
    assert 0 < da.paged_pages_workspace_size(1) < da.paged_pages_workspace_size(1 << 20) < 16 << 20
    for bad in (0, -1, 1 << 30):
        assert da.paged_pages_workspace_size(bad) == 0, bad
        with pytest.raises(ValueError):
            da.alloc_paged_pages_workspace(bad, device="cpu")
    # every workspace holds what workspace_init clears
    v = ctypes.c_void_p
    for size in (small, da.paged_pages_workspace_size(1)):
        assert lib.decode_attn_paged_workspace_init(v(4096 + 16), size, None) == ALIGN
        assert lib.decode_attn_paged_workspace_init(None, size, None) == ARG


def test_null_arguments(lib):
    assert lib.decode_attn_paged_chunk(None, None) == ARG
    assert lib.decode_attn_paged_window(None, 1, 0, None) == ARG
    assert lib.decode_attn_paged_free_pages(None, 20 << 20, 21 << 20, None) == ARG
    assert lib.decode_attn_paged_fork(None, None, 1 << 20, 2 << 20, 1, 3 << 20, 4 << 20, 4, None) == ARG
    assert lib.decode_attn_paged_compact(None, None, 1 << 20, 4, 2 << 20, None) == ARG


@pytest.mark.parametrize("change,status", BAD_CACHE, ids=[str(c) for c, _ in BAD_CACHE])
def test_cache_refusals(lib, change, status):
    assert chunk(lib, cache=change) == status
    assert window(lib, cache=change) == status


@pytest.mark.parametrize("change,status", [c for c in BAD_CACHE if c[0] is None or not set(c[0]) & {"Hkv"}][:12] + [
    (dict(page_size=32), ARG), (dict(num_pages=11), ARG), (dict(kv_dtype=3), ARG), (dict(kv_dtype=2, k_scale=0), ARG), (dict(Hkv=0), ARG)], ids=str)
def test_cache_refusals_of_the_page_operators(lib, change, status):
    assert fork(lib, cache=change) == status
    assert compact(lib, cache=change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=0), ARG), (dict(out=0), ARG), (dict(cu=0), ARG), (dict(lens=0), ARG), (dict(table=0), ARG), (dict(ws=0), ARG),
    (dict(q=8), ALIGN), (dict(out=(8 << 20) + 8), ALIGN), (dict(lse=2), ALIGN), (dict(lens=2), ALIGN), (dict(table=6), ALIGN), (dict(cu=2), ALIGN),
    (dict(ws=(9 << 20) + 128), ALIGN), (dict(ws_bytes=1000), SMALL), (dict(B=0), ARG), (dict(B=-3), ARG), (dict(B=1025), UNSUP),
    (dict(T=-1), ARG), (dict(T=1 << 30), ARG), (dict(Hq=0), ARG), (dict(Hq=6), ARG), (dict(max_pages=0), ARG), (dict(table_stride=3), ARG),
    (dict(max_pages=1 << 26, table_stride=1 << 26), ARG), (dict(dtype=2), ARG), (dict(dtype=1), ARG), (dict(scale=math.inf), ARG),
    (dict(scale=math.nan), ARG), (dict(window=-1), ARG), (dict(window=4, sinks=-1), ARG), (dict(q_stride=1016), ARG), (dict(out_stride=1016), ARG),
    (dict(q_stride=1028), ALIGN), (dict(out_stride=1028), ALIGN), (dict(q_stride=-1024), ARG),
], ids=str)
def test_chunk_refusals(lib, change, status):
    assert chunk(lib, **change) == status


def test_nothing_new_is_no_launch(lib):
    assert chunk(lib, T=0) == da.DA_OK
    assert chunk(lib, T=0, q=0, out=0) == da.DA_OK


@pytest.mark.parametrize("change,status", [
    (dict(window=0), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(q=0), ARG), (dict(out=0), ARG), (dict(ws=0), ARG), (dict(q=8), ALIGN),
    (dict(ws_bytes=1000), SMALL), (dict(T_q=17), ARG), (dict(B=1025), UNSUP), (dict(scale=math.nan), ARG), (dict(dtype=1), ARG),
], ids=str)
def test_window_refusals(lib, change, status):
    assert window(lib, **change) == status


ROW_REFUSALS = [
    (dict(lens=0), ARG), (dict(table=0), ARG), (dict(ws=0), ARG), (dict(lens=2), ALIGN), (dict(table=2), ALIGN), (dict(ws=64), ALIGN),
    (dict(ws_bytes=4096), SMALL), (dict(B=0), ARG), (dict(B=65537), UNSUP), (dict(max_pages=0), ARG), (dict(table_stride=3), ARG),
    (dict(page_size=0), ARG), (dict(page_size=24), ARG), (dict(page_size=1040), ARG), (dict(num_pages=0), ARG),
    (dict(num_pages=1 << 26), ARG), (dict(B=65536, max_pages=1 << 16, table_stride=1 << 16, page_size=16), ARG),
]


@pytest.mark.parametrize("change,status", ROW_REFUSALS, ids=str)
def test_rows_refusals(lib, change, status):
    assert free(lib, **change) == status
    assert fork(lib, **change) == status
    assert compact(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(out=0), ARG), (dict(count=0), ARG), (dict(out=2), ALIGN), (dict(count=6), ALIGN),
    (dict(out=7 << 20), ARG), (dict(out=(7 << 20) - 36), ARG), (dict(out=6 << 20), ARG), (dict(count=(20 << 20) + 36), ARG), (dict(count=(7 << 20) + 28), ARG), (dict(count=(6 << 20) + 4), ARG),
], ids=str)
def test_free_refusals(lib, change, status):
    assert free(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(parents=0), ARG), (dict(fresh=0), ARG), (dict(lens_out=0), ARG), (dict(table_out=0), ARG), (dict(n=0), ARG), (dict(n=65537), UNSUP),
    (dict(out_stride=3), ARG), (dict(parents=2), ALIGN), (dict(fresh=2), ALIGN), (dict(lens_out=2), ALIGN), (dict(table_out=2), ALIGN),
    (dict(table_out=7 << 20), ARG), (dict(table_out=(7 << 20) - 44), ARG), (dict(lens_out=6 << 20), ARG), (dict(lens_out=(7 << 20) + 16), ARG),
    (dict(lens_out=22 << 20), ARG), (dict(table_out=23 << 20), ARG), (dict(lens_out=(25 << 20) + 4), ARG),
], ids=str)
def test_fork_refusals(lib, change, status):
    assert fork(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(table_out=0), ARG), (dict(count=0), ARG), (dict(out_stride=3), ARG), (dict(table_out=2), ALIGN), (dict(count=2), ALIGN),
    (dict(table_out=7 << 20), ARG), (dict(table_out=6 << 20), ARG), (dict(count=6 << 20), ARG), (dict(count=(7 << 20) + 4), ARG), (dict(count=(25 << 20) + 4), ARG),
], ids=str)
def test_compact_refusals(lib, change, status):
    assert compact(lib, **change) == status


def test_binding_refuses_what_is_no_number_of_its_type(lib):
    from split_kv_decode_decoding_gb300.paged import _int32_of
    for bad in (1.5, "4", None, True, 1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError):
            _int32_of(bad, "window")
    assert _int32_of(7, "window") == 7


def test_the_reference_itself():
    """chunk64 against the decode reference of the same cache, and its window against counting."""
    paged = Paged([37, 5, 0], 2, 64, "f16", 16, VARLEN, seed=1)
    q = torch.randn(3, 4, 4, 64, generator=torch.Generator().manual_seed(2)).half()
    out, lse, _, _ = attend64(q, paged)
    got, got_l, tol_o, tol_l = chunk64(q.view(12, 4, 64), paged, [4, 4, 4])
    assert torch.allclose(got, torch.from_numpy(out).view(12, 4, 64), rtol=1e-12, atol=1e-15)
    assert torch.equal(torch.isinf(got_l), torch.isinf(torch.from_numpy(lse).view(12, 4)))
    assert (tol_o[:4] > 0).all() and (tol_o < 0.01).all() and (tol_l >= 0).all()   # (rows without keys: exact)
    seen = sees(torch.arange(20), torch.arange(20), 5, 3)
    for p in range(20):
        assert [j for j in range(20) if seen[p, j]] == [j for j in range(p + 1) if j > p - 5 or j < 3]
