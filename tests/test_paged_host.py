"""The paged-cache entry points on the host: symbols, sizes, refusals. Every case is answered by the
host-side checks, before any CUDA call."""
import ctypes
import math
import os
import re

import pytest
import torch

import split_kv_decode_decoding_gb300 as da
from paged_ref import needed, to_e4m3

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "decode_attn_paged.h")


@pytest.fixture(scope="module")
def lib():
    da.build()
    return da.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(decode_attn_paged\w*)\s*\(", text))
    assert names == set(da.EXPORTED_PAGED)
    for n in names:
        assert hasattr(lib, n), n


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name, value in (("DA_E4M3", da.DA_E4M3), ("DA_MAX_PAGED_BATCH", da.DA_MAX_PAGED_BATCH),
                        ("DA_MAX_PAGE_SIZE", da.DA_MAX_PAGE_SIZE)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value
    for name, value in (("DA_DEVERR_PAGE", da.DA_DEVERR_PAGE), ("DA_DEVERR_POSITION", da.DA_DEVERR_POSITION)):
        assert int(re.search(rf"#define {name} (0x\d+)u", text).group(1), 16) == value
    bits = [da.DA_DEVERR_SEQLENS, da.DA_DEVERR_TIMEOUT, da.DA_DEVERR_PAGE, da.DA_DEVERR_POSITION]
    assert sum(bits) == 0xF
    assert re.search(r"DA_ROPE_NONE = 0,.*DA_ROPE_HALF = 1,.*DA_ROPE_INTERLEAVED = 2", text, re.S)


def test_workspace_size(lib):
    one, four = da.paged_workspace_size(1, 32, 8, 128), da.paged_workspace_size(4, 32, 8, 128)
    assert 0 < one < four <= 64 << 20
    assert da.paged_workspace_size(2, 32, 8, 128) == one          # 8 columns either way
    for bad in ((0, 32, 8, 128), (17, 32, 8, 128), (1, 30, 8, 128), (1, 32, 0, 128), (1, 0, 1, 128), (1, 32, 8, 96)):
        assert da.paged_workspace_size(*bad) == 0, bad
        with pytest.raises(ValueError):
            da.alloc_paged_workspace(*bad, device="cpu")
    v = ctypes.c_void_p
    assert lib.decode_attn_paged_workspace_init(None, 1 << 20, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_paged_workspace_init(v(4096), 256, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_paged_workspace_init(v(4096 + 16), 1 << 20, None) == da.DA_ERR_ALIGNMENT


# addresses that are never followed: the calls below are refused before any device work
CACHE = dict(k=1 << 20, v=2 << 20, k_scale=3 << 20, v_scale=4 << 20, num_pages=10, page_size=64, Hkv=4, D=128, kv_dtype=0,
             layout=0)
ATTEND = dict(q=5 << 20, lens=6 << 20, table=7 << 20, max_pages=4, table_stride=4, B=2, T_q=1, Hq=8, dtype=0, scale=0.1,
              out=8 << 20, lse=0, ws=9 << 20, ws_bytes=1 << 30)
APPEND = dict(q=5 << 20, q_stride=1024, k=10 << 20, k_stride=512, v=11 << 20, v_stride=512, cos_sin=12 << 20, max_pos=256,
              rot=128, rope=1, cu=13 << 20, lens=6 << 20, table=7 << 20, max_pages=4, table_stride=4, B=2, T=2, Hq=8,
              dtype=0, q_out=14 << 20, q_out_stride=1024, ws=9 << 20)


def cache_struct(**change):
    from split_kv_decode_decoding_gb300.paged import _CacheStruct
    return _CacheStruct(**{**CACHE, **change})


def attend(lib, cache={}, **change):
    from split_kv_decode_decoding_gb300.paged import _pack_attn
    a = {**ATTEND, **change}
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged(
        _pack_attn(a["q"], 0 if c is None else ctypes.addressof(c), a["lens"], a["table"], a["max_pages"], a["table_stride"], a["B"],
                   a["T_q"], a["Hq"], a["dtype"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"]), None)


def append(lib, cache={}, **change):
    from split_kv_decode_decoding_gb300.paged import _pack_append
    a = {**APPEND, **change}
    c = cache_struct(**cache) if cache is not None else None
    return lib.decode_attn_paged_append(
        _pack_append(a["q"], a["k"], a["v"], a["q_stride"], a["k_stride"], a["v_stride"], a["cos_sin"], a["max_pos"], a["rot"],
                     a["rope"], a["cu"], a["lens"], a["table"], a["max_pages"], a["table_stride"], a["B"], a["T"], a["Hq"],
                     a["dtype"], 0 if c is None else ctypes.addressof(c), a["q_out"], a["q_out_stride"], a["ws"]), None)


def test_packed_structs_lie_as_the_header_declares(tmp_path):
    """Offsets of every field of the two argument structs, from the C compiler, against the binding's formats."""
    import struct as st
    import subprocess
    from split_kv_decode_decoding_gb300 import paged
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, fmt in (("da_paged_attn", "@PPPPiiiiiifPPPN"), ("da_paged_append", "@PPPqqqPiiiPPPiiiiiiPPqP")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        fields = [w.strip(" *") for d in body.split(";") if d.strip() for w in re.sub(r"^\s*(const\s+)?\w+", "", d.strip()).split(",")]
        assert len(fields) == len(fmt) - 1
        src = tmp_path / (name + ".c")
        src.write_text('#include <stdio.h>\n#include "decode_attn_paged.h"\nint main(void) {\n' + "".join(
            f'printf("%zu ", offsetof({name}, {f}));\n' for f in fields) + f'printf("%zu", sizeof({name}));\nreturn 0; }}\n')
        exe = tmp_path / name
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), "-o", str(exe), str(src)], check=True)
        got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        want = [st.calcsize(fmt[:i + 1] + "0" + fmt[i + 1]) for i in range(len(fields))]
        assert got[:-1] == want and got[-1] == st.calcsize(fmt + "0P")
    assert paged._pack_attn(*([0] * 10), 0.0, 0, 0, 0, 0)[:8] == bytes(8)


def test_null_arguments(lib):
    assert lib.decode_attn_paged(None, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_paged_append(None, None) == da.DA_ERR_INVALID_ARG


ARG, UNSUP, ALIGN, SMALL = da.DA_ERR_INVALID_ARG, da.DA_ERR_UNSUPPORTED, da.DA_ERR_ALIGNMENT, da.DA_ERR_WORKSPACE_TOO_SMALL
BAD_CACHE = [
    (None, ARG), (dict(k=0), ARG), (dict(v=0), ARG), (dict(k=(1 << 20) + 8), ALIGN), (dict(v=(1 << 20) + 2), ALIGN),
    (dict(num_pages=0), ARG), (dict(num_pages=-1), ARG), (dict(page_size=0), ARG), (dict(page_size=8), ARG),
    (dict(page_size=24), ARG), (dict(page_size=1040), ARG), (dict(Hkv=0), ARG), (dict(Hkv=3), ARG), (dict(D=96), UNSUP),
    (dict(D=256), UNSUP), (dict(kv_dtype=1), ARG), (dict(kv_dtype=3), ARG), (dict(layout=2), ARG),
    (dict(kv_dtype=2, k_scale=0), ARG), (dict(kv_dtype=2, v_scale=0), ARG), (dict(kv_dtype=2, v_scale=(1 << 20) + 2), ALIGN),
    (dict(num_pages=1 << 26), ARG),                      # rows past 32 bits
    (dict(num_pages=1 << 30, Hkv=8, page_size=16), ARG),
]


@pytest.mark.parametrize("change,status", BAD_CACHE, ids=[str(c) for c, _ in BAD_CACHE])
def test_cache_refusals(lib, change, status):
    assert attend(lib, cache=change) == status
    assert append(lib, cache=change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=0), ARG), (dict(out=0), ARG), (dict(lens=0), ARG), (dict(table=0), ARG), (dict(ws=0), ARG),
    (dict(q=8), ALIGN), (dict(out=(8 << 20) + 8), ALIGN), (dict(lse=2), ALIGN), (dict(lens=2), ALIGN), (dict(table=6), ALIGN),
    (dict(ws=(9 << 20) + 128), ALIGN), (dict(ws_bytes=1000), SMALL), (dict(B=0), ARG), (dict(B=-3), ARG), (dict(B=1025), UNSUP),
    (dict(T_q=0), ARG), (dict(T_q=17), ARG), (dict(Hq=0), ARG), (dict(Hq=6), ARG), (dict(max_pages=0), ARG),
    (dict(table_stride=3), ARG), (dict(max_pages=1 << 26, table_stride=1 << 26), ARG), (dict(dtype=2), ARG), (dict(dtype=1), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG),
], ids=str)
def test_attend_refusals(lib, change, status):
    assert attend(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(k=0), ARG), (dict(v=0), ARG), (dict(cu=0), ARG), (dict(lens=0), ARG), (dict(table=0), ARG), (dict(ws=0), ARG),
    (dict(q_out=0), ARG), (dict(T=-1), ARG), (dict(rope=3), ARG), (dict(cos_sin=0), ARG), (dict(max_pos=0), ARG),
    (dict(rot=0), ARG), (dict(rot=24), ARG), (dict(rot=144), ARG), (dict(k_stride=504), ARG), (dict(v_stride=0), ARG),
    (dict(q_stride=1016), ARG), (dict(q_out_stride=8), ARG), (dict(k_stride=516), ALIGN), (dict(v_stride=516), ALIGN),
    (dict(q_stride=1028), ALIGN), (dict(q_out_stride=1028), ALIGN), (dict(k=8), ALIGN), (dict(v=24), ALIGN), (dict(q=8), ALIGN),
    (dict(q_out=8), ALIGN), (dict(cos_sin=4), ALIGN), (dict(cu=2), ALIGN), (dict(ws=64), ALIGN), (dict(B=0), ARG),
    (dict(B=1025), UNSUP), (dict(Hq=6), ARG), (dict(table_stride=3), ARG), (dict(dtype=1), ARG),
], ids=str)
def test_append_refusals(lib, change, status):
    assert append(lib, **change) == status


def test_nothing_to_append_is_no_launch(lib):
    assert append(lib, T=0) == da.DA_OK
    assert append(lib, T=0, q=0, k=0, v=0, rope=0, cos_sin=0) == da.DA_OK


def test_binding_refuses_cpu_and_ill_shaped_tensors(lib):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        da.PagedCache(k, k.clone())                                   # not on a GPU
    with pytest.raises(TypeError):
        da.PagedCache(k.float(), k.float())
    with pytest.raises(ValueError):
        da.PagedCache(k, k[:3])
    with pytest.raises(ValueError):
        da.PagedCache(k.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(ValueError):
        da.PagedCache(k, k, layout=2)


def test_scale_rule_of_the_reference():
    """The tests' own scale rule at its borders: 448 * 2^e itself still fits 2^e."""
    assert needed(448.0) == 1.0 and needed(448.0000001) == 2.0 and needed(3.5) == 2.0 ** -7 and needed(0.0) == 2.0 ** -126
    assert float(to_e4m3(torch.tensor(17.0))) == 16.0 and float(to_e4m3(torch.tensor(19.0))) == 20.0
    assert float(to_e4m3(torch.tensor(math.inf))) == 448.0 and math.isnan(float(to_e4m3(torch.tensor(math.nan))))
