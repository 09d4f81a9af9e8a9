"""Python binding of the paged-cache part of the library (include/decode_attn_paged.h).

Argument marshalling only, like the rest of the binding, with the checks that need a
tensor's shape, type or device (ValueError or TypeError); the library makes the others
(DecodeAttnError). A PagedCache is made once per cache and describes it to every call.
"""
from __future__ import annotations

import ctypes
import math
import operator
import struct

DA_E4M3 = 2
DA_DEVERR_PAGE, DA_DEVERR_POSITION = 0x4, 0x8
DA_MAX_PAGED_BATCH, DA_MAX_PAGE_SIZE = 1024, 1024
DA_MAX_PAGED_ROWS = 65536
DA_ROPE_NONE, DA_ROPE_HALF, DA_ROPE_INTERLEAVED = 0, 1, 2

EXPORTED_PAGED = [
    "decode_attn_paged_workspace_size", "decode_attn_paged_workspace_init", "decode_attn_paged",
    "decode_attn_paged_append", "decode_attn_paged_window", "decode_attn_paged_chunk_workspace_size",
    "decode_attn_paged_chunk", "decode_attn_paged_pages_workspace_size", "decode_attn_paged_free_pages",
    "decode_attn_paged_fork", "decode_attn_paged_compact",
]


class _CacheStruct(ctypes.Structure):
    """da_paged_cache"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("kv_dtype", ctypes.c_int), ("layout", ctypes.c_int)]


_handle = None


def declare(lib) -> None:
    """Argument and result types of the paged entry points (called once, by load())."""
    global _handle
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.decode_attn_paged_workspace_size.argtypes = [I, I, I, I]
    lib.decode_attn_paged_workspace_size.restype = SZ
    lib.decode_attn_paged_workspace_init.argtypes = [P, SZ, P]
    lib.decode_attn_paged_workspace_init.restype = I
    lib.decode_attn_paged_chunk_workspace_size.argtypes = [I, I, I]
    lib.decode_attn_paged_chunk_workspace_size.restype = SZ
    lib.decode_attn_paged_pages_workspace_size.argtypes = [I]
    lib.decode_attn_paged_pages_workspace_size.restype = SZ
    S = ctypes.c_char_p
    for f, more in ((lib.decode_attn_paged, []), (lib.decode_attn_paged_append, []), (lib.decode_attn_paged_window, [I, I]),
                    (lib.decode_attn_paged_chunk, []), (lib.decode_attn_paged_free_pages, [P, P]),
                    (lib.decode_attn_paged_fork, [P, P, P, I, P, P, I]), (lib.decode_attn_paged_compact, [P, P, I, P])):
        f.argtypes = [S, *more, P]
        f.restype = I
    _handle = lib


# da_paged_attn, da_paged_append, da_paged_chunk and da_paged_rows, field by field: packing a struct costs a third of what ctypes
# takes to convert as many arguments
_pack_attn = struct.Struct("@PPPPiiiiiifPPPN").pack
_pack_append = struct.Struct("@PPPqqqPiiiPPPiiiiiiPPqP").pack
_pack_chunk = struct.Struct("@PqPPPPiiiiiifiiPqPPN").pack
_pack_rows = struct.Struct("@PPiiiiiPN").pack


def _lib():
    if _handle is None:
        from . import load
        load()
    return _handle


def _fail(status: int, where: str) -> None:
    from . import DecodeAttnError
    raise DecodeAttnError(status, where)


# torch's types and device queries, looked up on first use (importing the binding does not import torch)
_int32 = _float32 = _codes = _current_device = _current_stream = None


def _init() -> None:
    global _int32, _float32, _codes, _current_device, _current_stream
    import torch
    _int32, _float32 = torch.int32, torch.float32
    _current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _codes = {torch.float16: 0, torch.bfloat16: 1, torch.float8_e4m3fn: DA_E4M3}


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_device(device: int) -> None:
    if device < 0:
        raise ValueError("tensors must be CUDA tensors")
    if device != _current_device():
        raise ValueError(f"tensors are on cuda:{device}, which is not the current device")


class PagedCache:
    """A KV cache in pages.

    k, v: [num_pages, page_size, Hkv, D] (layout DA_LAYOUT_VARLEN) or [num_pages, Hkv, page_size, D]
    (DA_LAYOUT_BHSD), contiguous, float16, bfloat16 or float8_e4m3fn. float8 pages take k_scale and
    v_scale, float32 [num_pages, Hkv]. The tensors stay the caller's; the cache keeps them alive.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None, *, layout: int = 0):
        if _codes is None:
            _init()
        if layout not in (0, 1):
            raise ValueError(f"unknown layout {layout}")
        code = _codes.get(k.dtype)
        if code is None:
            raise TypeError(f"k must be float16, bfloat16 or float8_e4m3fn, not {k.dtype}")
        if v.dtype != k.dtype or v.shape != k.shape or k.dim() != 4:
            raise ValueError("k and v must be 4-dimensional, of one shape and type")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k and v must be contiguous")
        self.device = k.get_device()
        if self.device < 0 or v.get_device() != self.device:
            raise ValueError("k and v must be on one CUDA device")
        pages = k.shape[0]
        page_size, heads = (k.shape[1], k.shape[2]) if layout == 0 else (k.shape[2], k.shape[1])
        if code == DA_E4M3:
            for s in (k_scale, v_scale):
                if s is None or s.dtype is not _float32 or tuple(s.shape) != (pages, heads) or not s.is_contiguous() \
                        or s.get_device() != self.device:
                    raise ValueError("float8 pages need contiguous float32 scales [num_pages, Hkv] on the pages' device")
        else:
            k_scale = v_scale = None
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.Hkv, self.D = pages, page_size, heads, k.shape[3]
        self.kv_dtype, self.layout, self.dtype = code, layout, k.dtype
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
                                    0 if v_scale is None else v_scale.data_ptr(), pages, page_size, heads, self.D, code,
                                    layout)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hkv: int, D: int, dtype, *, layout: int = 0, device="cuda"):
        """A cache of uninitialised pages (an append gives a page its scale when it writes its first slot)."""
        import torch
        inner = (page_size, Hkv) if layout == 0 else (Hkv, page_size)
        k, v = (torch.empty(num_pages, *inner, D, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v, layout=layout)
        ks, vs = (torch.empty(num_pages, Hkv, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs, layout=layout)


def paged_workspace_size(T_q: int, Hq: int, Hkv: int, D: int) -> int:
    return _lib().decode_attn_paged_workspace_size(T_q, Hq, Hkv, D)


def _alloc(nbytes: int, device, stream):
    import torch
    if _codes is None:
        _init()
    if nbytes == 0:
        raise ValueError("the workspace size was rejected: a size is out of range")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check_device(ws.get_device())
    st = _lib().decode_attn_paged_workspace_init(ws.data_ptr(), nbytes, _raw_stream(stream, ws.get_device()))
    if st:
        _fail(st, "decode_attn_paged_workspace_init")
    return ws


def alloc_paged_workspace(T_q: int, Hq: int, Hkv: int, D: int, device="cuda", stream=None):
    """Allocate (through PyTorch) and initialise a workspace for calls with these heads, of up to T_q query tokens."""
    return _alloc(paged_workspace_size(T_q, Hq, Hkv, D), device, stream)


def paged_chunk_workspace_size(Hq: int, Hkv: int, D: int) -> int:
    return _lib().decode_attn_paged_chunk_workspace_size(Hq, Hkv, D)


def paged_pages_workspace_size(num_pages: int) -> int:
    return _lib().decode_attn_paged_pages_workspace_size(num_pages)


def alloc_paged_chunk_workspace(Hq: int, Hkv: int, D: int, device="cuda", stream=None):
    """Allocate and initialise a workspace for decode_attn_paged_chunk with these heads."""
    return _alloc(paged_chunk_workspace_size(Hq, Hkv, D), device, stream)


def alloc_paged_pages_workspace(num_pages: int, device="cuda", stream=None):
    """Allocate and initialise a workspace for free_pages, fork and compact over a cache of num_pages pages."""
    return _alloc(paged_pages_workspace_size(num_pages), device, stream)


def _check_sequences(kv_lens, block_table, dev):
    """(B, max_pages, table_stride) of kv_lens [B] and block_table [B, max_pages]."""
    if kv_lens.dtype is not _int32 or block_table.dtype is not _int32:
        raise TypeError("kv_lens and block_table must be int32")
    if block_table.dim() != 2 or kv_lens.shape != block_table.shape[:1]:
        raise ValueError("kv_lens must be [B] and block_table [B, max_pages]")
    (B, max_pages), (stride, one) = block_table.shape, block_table.stride()
    if not kv_lens.is_contiguous() or (one != 1 and max_pages > 1):   # (a row of one entry: any stride)
        raise ValueError("kv_lens and the rows of block_table must be contiguous")
    if kv_lens.get_device() != dev or block_table.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    return B, max_pages, stride if B > 1 else max_pages   # the stride of a single row is any number


def _decode_args(q, cache: PagedCache, kv_lens, block_table, out, workspace, scale, lse):
    """(packed da_paged_attn, device) of a decode call."""
    if _codes is None:
        _init()
    dev = q.get_device()
    _check_device(dev)
    if cache.device != dev:
        raise ValueError("the cache must be on the tensors' device")
    B, max_pages, table_stride = _check_sequences(kv_lens, block_table, dev)
    shape, dtype = q.shape, q.dtype
    code = _codes.get(dtype, -1)
    if code not in (0, 1):
        raise TypeError(f"q must be float16 or bfloat16, not {dtype}")
    if cache.kv_dtype != DA_E4M3 and cache.kv_dtype != code:
        raise TypeError(f"q is {dtype}, the cache {cache.dtype}")
    if len(shape) == 4:
        n, T_q, Hq, D = shape
    elif len(shape) == 3:
        (n, Hq, D), T_q = shape, 1
    else:
        raise ValueError(f"q must be [B, T_q, Hq, D] or [B, Hq, D], not {tuple(shape)}")
    if n != B or D != cache.D:
        raise ValueError(f"q {tuple(shape)} does not fit {B} sequences of head size {cache.D}")
    if out.shape != shape or out.dtype is not dtype or out.get_device() != dev:
        raise ValueError("out must have q's shape, type and device")
    if not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError("q and out must be contiguous")
    lse_ptr = 0
    if lse is not None:
        if lse.shape != shape[:-1] or lse.dtype is not _float32 or not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError("lse must be contiguous float32 of q's shape without its last dimension")
        lse_ptr = lse.data_ptr()
    if workspace.get_device() != dev:
        raise ValueError("the workspace must be on q's device")
    try:
        args = _pack_attn(q.data_ptr(), cache._ref, kv_lens.data_ptr(), block_table.data_ptr(), max_pages, table_stride, B, T_q,
                          Hq, code, 1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(), lse_ptr,
                          workspace.data_ptr(), workspace.nbytes)
    except struct.error as e:
        raise ValueError(f"scale, or a size, is no number of its C type: {e}") from None
    return args, dev


def decode_attn_paged(q, cache: PagedCache, kv_lens, block_table, out, workspace, *, scale: float | None = None, lse=None,
                      stream=None):
    """out = decode attention of q over a paged cache; see the C header.

    q, out: [B, T_q, Hq, D], or [B, Hq, D] for one query token; lse (optional): float32 of the same
    shape without D. kv_lens: int32 [B]; block_table: int32 [B, max_pages].
    """
    args, dev = _decode_args(q, cache, kv_lens, block_table, out, workspace, scale, lse)
    st = _lib().decode_attn_paged(args, _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged")
    return out


def _int32_of(x, name):
    """x, a whole number of Python's or of a type with __index__, as a C int."""
    try:
        n = operator.index(x)
    except TypeError:
        n = None
    if n is None or isinstance(x, bool) or not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} must be a whole number of 32 bits, not {x!r}")
    return n


def decode_attn_paged_window(q, cache: PagedCache, kv_lens, block_table, out, workspace, *, window: int, sinks: int = 0,
                             scale: float | None = None, lse=None, stream=None):
    """decode_attn_paged where a token sees itself, the window - 1 tokens before it and the first `sinks` tokens."""
    args, dev = _decode_args(q, cache, kv_lens, block_table, out, workspace, scale, lse)
    st = _lib().decode_attn_paged_window(args, _int32_of(window, "window"), _int32_of(sinks, "sinks"), _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_window")
    return out


def _length(x, name):
    """The first dimension of a tensor that has one."""
    if x.dim() == 0:
        raise ValueError(f"{name} must have a dimension")
    return x.shape[0]


def _rows(x, name, T, heads, D, dtype, dev):
    """Check [T, heads, D] rows with contiguous heads; their row stride."""
    if x.shape != (T, heads, D):
        raise ValueError(f"{name} must be {(T, heads, D)}, not {tuple(x.shape)}")
    row, head, one = x.stride()
    if one != 1 or (head != D and heads > 1):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if x.dtype is not dtype or x.get_device() != dev:
        raise ValueError(f"{name} must have k's type and device")
    return row if T > 1 else heads * D   # the stride of a single row is any number


def decode_attn_paged_append(q, k, v, cache: PagedCache, cu_new, kv_lens, block_table, workspace, *, cos_sin=None,
                             rope: int = DA_ROPE_HALF, q_out=None, stream=None):
    """Rotate new tokens by their positions and append them to a paged cache; see the C header.

    q: [T, Hq, D] or None; k, v: [T, Hkv, D]; rows may be strided (slices of one projection's
    output). cu_new: int32 [B + 1]; kv_lens: int32 [B], the new tokens counted. cos_sin: float32
    [max_pos, rot_dim], or None for no rotation. q_out: like q (q itself to rotate in place);
    returned.
    """
    if _codes is None:
        _init()
    dev = k.get_device()
    _check_device(dev)
    if cache.device != dev:
        raise ValueError("the cache must be on the tensors' device")
    B, max_pages, table_stride = _check_sequences(kv_lens, block_table, dev)
    dtype = k.dtype
    code = _codes.get(dtype, -1)
    if code not in (0, 1):
        raise TypeError(f"k must be float16 or bfloat16, not {dtype}")
    if cache.kv_dtype != DA_E4M3 and cache.kv_dtype != code:
        raise TypeError(f"k is {dtype}, the cache {cache.dtype}")
    T, D = _length(k, "k"), cache.D
    k_stride = _rows(k, "k", T, cache.Hkv, D, dtype, dev)
    v_stride = _rows(v, "v", T, cache.Hkv, D, dtype, dev)
    q_ptr = out_ptr = q_stride = out_stride = Hq = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        if q.dim() != 3:
            raise ValueError(f"q must be [T, Hq, D], not {tuple(q.shape)}")
        Hq = q.shape[1]
        q_stride = _rows(q, "q", T, Hq, D, dtype, dev)
        out_stride = q_stride if q_out is q else _rows(q_out, "q_out", T, Hq, D, dtype, dev)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    if cu_new.dtype is not _int32 or cu_new.shape != (B + 1,) or not cu_new.is_contiguous() or cu_new.get_device() != dev:
        raise ValueError("cu_new must be contiguous int32 [B + 1]")
    if cos_sin is None:
        rope, cs_ptr, max_pos, rot = DA_ROPE_NONE, 0, 0, 0
    else:
        if cos_sin.dtype is not _float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.get_device() != dev:
            raise ValueError("cos_sin must be contiguous float32 [max_pos, rot_dim]")
        cs_ptr, (max_pos, rot) = cos_sin.data_ptr(), cos_sin.shape
    if workspace.get_device() != dev or workspace.nbytes < 256:
        raise ValueError("the workspace must be on the tensors' device")
    try:
        args = _pack_append(q_ptr, k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, cs_ptr, max_pos, rot, rope,
                            cu_new.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), max_pages, table_stride, B, T, Hq,
                            code, cache._ref, out_ptr, out_stride, workspace.data_ptr())
    except struct.error as e:
        raise ValueError(f"rope, or a size, is no number of its C type: {e}") from None
    st = _lib().decode_attn_paged_append(args, _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_append")
    return q_out


def decode_attn_paged_chunk(q, cache: PagedCache, cu_new, kv_lens, block_table, out, workspace, *, scale: float | None = None,
                            window: int | None = None, sinks: int = 0, lse=None, stream=None):
    """out = attention of a chunk of new tokens of each sequence over the paged cache; see the C header.

    q, out: [T, Hq, D], rows may be strided; cu_new: int32 [B + 1]; kv_lens: int32 [B], the new
    tokens counted (their keys and values are in the pages); block_table: int32 [B, max_pages];
    lse (optional): float32 [T, Hq]. window None or 0: no limit.
    """
    if _codes is None:
        _init()
    dev = q.get_device()
    _check_device(dev)
    if cache.device != dev:
        raise ValueError("the cache must be on the tensors' device")
    B, max_pages, table_stride = _check_sequences(kv_lens, block_table, dev)
    dtype, D = q.dtype, cache.D
    code = _codes.get(dtype, -1)
    if code not in (0, 1):
        raise TypeError(f"q must be float16 or bfloat16, not {dtype}")
    if cache.kv_dtype != DA_E4M3 and cache.kv_dtype != code:
        raise TypeError(f"q is {dtype}, the cache {cache.dtype}")
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, D], not {tuple(q.shape)}")
    T, Hq = q.shape[0], q.shape[1]
    q_stride = _rows(q, "q", T, Hq, D, dtype, dev)
    out_stride = _rows(out, "out", T, Hq, D, dtype, dev)
    if cu_new.dtype is not _int32 or cu_new.shape != (B + 1,) or not cu_new.is_contiguous() or cu_new.get_device() != dev:
        raise ValueError("cu_new must be contiguous int32 [B + 1]")
    lse_ptr = 0
    if lse is not None:
        if lse.shape != (T, Hq) or lse.dtype is not _float32 or not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError("lse must be contiguous float32 [T, Hq]")
        lse_ptr = lse.data_ptr()
    if workspace.get_device() != dev:
        raise ValueError("the workspace must be on q's device")
    try:
        args = _pack_chunk(q.data_ptr(), q_stride, cache._ref, cu_new.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(),
                           max_pages, table_stride, B, T, Hq, code, 1.0 / math.sqrt(D) if scale is None else scale,
                           0 if window is None else _int32_of(window, "window"), _int32_of(sinks, "sinks"), out.data_ptr(),
                           out_stride, lse_ptr, workspace.data_ptr(), workspace.nbytes)
    except struct.error as e:
        raise ValueError(f"scale, or a size, is no number of its C type: {e}") from None
    st = _lib().decode_attn_paged_chunk(args, _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_chunk")
    return out


# ------------------------------------------------------------ managing the pages
def _rows_args(kv_lens, block_table, workspace, page_size, num_pages):
    """(packed da_paged_rows, B, max_pages, device)"""
    if _codes is None:
        _init()
    dev = kv_lens.get_device()
    _check_device(dev)
    B, max_pages, table_stride = _check_sequences(kv_lens, block_table, dev)
    if workspace.get_device() != dev:
        raise ValueError("the workspace must be on the tensors' device")
    try:
        args = _pack_rows(kv_lens.data_ptr(), block_table.data_ptr(), max_pages, table_stride, B, page_size, num_pages,
                          workspace.data_ptr(), workspace.nbytes)
    except struct.error as e:
        raise ValueError(f"page_size, or a size, is no number of its C type: {e}") from None
    return args, B, max_pages, dev


def _list(x, name, n, dev):
    """Check a contiguous int32 [n] tensor; its address."""
    if x.dtype is not _int32 or x.shape != (n,) or not x.is_contiguous() or x.get_device() != dev:
        raise ValueError(f"{name} must be contiguous int32 [{n}] on the tensors' device")
    return x.data_ptr()


def _table_out(x, B, max_pages, dev):
    """Check a block table to write; its row stride."""
    if x.dtype is not _int32 or x.dim() != 2 or x.shape[0] != B or x.shape[1] < max_pages or x.get_device() != dev:
        raise ValueError(f"block_table_out must be int32 [{B}, max_pages] on the tensors' device, with max_pages >= {max_pages}")
    stride, one = x.stride()
    if (one != 1 and x.shape[1] > 1) or (B > 1 and stride < x.shape[1]):
        raise ValueError("the rows of block_table_out must be contiguous and apart")
    return stride if B > 1 else x.shape[1]


def decode_attn_paged_free_pages(kv_lens, block_table, free_pages, num_free, workspace, *, page_size: int, stream=None):
    """free_pages[:n] = the pages that no sequence uses, ascending, num_free[0] = n; see the C header.

    kv_lens: int32 [B]; block_table: int32 [B, max_pages]; free_pages: int32 [num_pages] of the cache;
    num_free: int32 [1]. Returned.
    """
    n = _length(free_pages, "free_pages")
    args, _, _, dev = _rows_args(kv_lens, block_table, workspace, page_size, n)
    st = _lib().decode_attn_paged_free_pages(args, _list(free_pages, "free_pages", n, dev),
                                             _list(num_free, "num_free", 1, dev), _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_free_pages")
    return free_pages, num_free


def decode_attn_paged_fork(cache: PagedCache, kv_lens, block_table, parents, new_pages, kv_lens_out, block_table_out, workspace,
                           *, stream=None):
    """Rows that continue other rows of a block table and share their pages; see the C header.

    parents, new_pages, kv_lens_out: int32 [n]; block_table_out: int32 [n, max_pages]. Returned:
    kv_lens_out, block_table_out.
    """
    args, _, max_pages, dev = _rows_args(kv_lens, block_table, workspace, cache.page_size, cache.num_pages)
    if cache.device != dev:
        raise ValueError("the cache must be on the tensors' device")
    n = _length(parents, "parents")
    stride = _table_out(block_table_out, n, max_pages, dev)
    st = _lib().decode_attn_paged_fork(args, cache._ref, _list(parents, "parents", n, dev), _list(new_pages, "new_pages", n, dev), n,
                                       _list(kv_lens_out, "kv_lens_out", n, dev), block_table_out.data_ptr(), stride,
                                       _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_fork")
    return kv_lens_out, block_table_out


def decode_attn_paged_compact(cache: PagedCache, kv_lens, block_table, block_table_out, num_used, workspace, *, stream=None):
    """Move the n pages in use to the front of the cache; block_table_out names them there, num_used[0] = n.

    block_table_out: int32 [B, max_pages], another tensor than block_table; num_used: int32 [1]. Returned.
    """
    args, B, max_pages, dev = _rows_args(kv_lens, block_table, workspace, cache.page_size, cache.num_pages)
    if cache.device != dev:
        raise ValueError("the cache must be on the tensors' device")
    stride = _table_out(block_table_out, B, max_pages, dev)
    st = _lib().decode_attn_paged_compact(args, cache._ref, block_table_out.data_ptr(), stride, _list(num_used, "num_used", 1, dev),
                                          _raw_stream(stream, dev))
    if st:
        _fail(st, "decode_attn_paged_compact")
    return block_table_out, num_used
