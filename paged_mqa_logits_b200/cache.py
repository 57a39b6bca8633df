"""The cache around the logits: appends, attention over a 4-bit cache, pages.

Argument marshalling for include/mqa_cache.h, in the manner of the package's
other calls: tensors become pointers, shapes a params struct, every step runs in
the CUDA kernels, and there is no fallback. All tensors of a call are on one
device, which need not be the current one. Calls run on `stream` (a
torch.cuda.Stream or a raw handle), else on the device's current stream; what a
call allocates (results and workspaces that were not given) belongs to that
stream. The caller orders the inputs' producers before that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional, Sequence, Union

import torch

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_INT, _BYTE, _FLOAT = torch.int32, torch.uint8, torch.float32
MQA_PAGES_MAX_CACHES = 256


class AttentionParams(ctypes.Structure):
    """Mirror of struct mqa_attention_params."""
    _fields_ = [(n, _I32) for n in (
        "batch", "next_n", "num_heads", "num_kv_heads", "head_dim", "page_size", "num_pages",
        "max_pages_per_row", "topk", "num_ctas", "dtype")] + [
        ("flags", ctypes.c_uint32), ("softmax_scale", ctypes.c_float), ("reserved", _I32),
        ("q_stride_b", _I64), ("q_stride_n", _I64), ("q_stride_h", _I64),
        ("workspace_bytes", ctypes.c_uint64), ("status", _P)]


class AppendParams(ctypes.Structure):
    """Mirror of struct mqa_append_params."""
    _fields_ = [(n, _I32) for n in (
        "batch", "num_tokens", "num_kv_heads", "head_dim", "page_size", "num_pages",
        "max_pages_per_row", "dtype")] + [
        ("flags", ctypes.c_uint32), ("reserved", _I32), ("k_stride_t", _I64),
        ("k_stride_h", _I64), ("v_stride_t", _I64), ("v_stride_h", _I64), ("status", _P)]


class PagesParams(ctypes.Structure):
    """Mirror of struct mqa_pages_params."""
    _fields_ = [(n, _I32) for n in (
        "batch", "out_batch", "max_pages_per_row", "num_pages", "page_size")] + [
        ("flags", ctypes.c_uint32), ("status", _P)]


# The calls below pack the same structs into bytes: a fifth of the time that filling
# a ctypes.Structure takes, and small calls are bound by the host.
_ATTENTION, _APPEND, _PAGES = struct.Struct("@11iIfi3qQP"), struct.Struct("@8iIi4qP"), struct.Struct("@5iIP")
assert _ATTENTION.size == ctypes.sizeof(AttentionParams)
assert _APPEND.size == ctypes.sizeof(AppendParams)
assert _PAGES.size == ctypes.sizeof(PagesParams)


def declare(lib) -> None:
    """Argument types of the entry points of include/mqa_cache.h."""
    for name, types in {
        "paged_mqa_attention_fp4": [_P] * 12,
        "mqa_attention_workspace_size": [_P, _P],
        "mqa_cache_append_fp8": [_P] * 8,
        "mqa_cache_append_fp4": [_P] * 11,
        "mqa_pages_fork": [_P] * 8,
        "mqa_pages_resize": [_P] * 8,
        "mqa_pages_compact": [_P] * 9,
        "mqa_pages_copy": [_P, _P, _I32, _P, _P, _I32, _P, _P, _P],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int


_library = None


def _lib():
    global _library
    if _library is None:
        from . import library
        _library = library()
    return _library


def _check(rc: int) -> None:
    if rc != 0:
        from . import _check as check
        check(rc)


# of the current device, without torch.cuda's own check that CUDA is set up (a CUDA tensor is there)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """Whether a call on t's device and `stream` needs the current ones changed."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return stream is not None or dev != _current()


@contextlib.contextmanager
def _there(t: torch.Tensor, stream):
    """t's device and `stream` (None: the device's current one) as the current ones."""
    with torch.cuda.device(t.device):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            # handle 0 is the default stream; ExternalStream takes it for none given and makes a new one
            stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                      else torch.cuda.default_stream(t.device))
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.stream(stream):
            yield


_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _ptr(t: Optional[torch.Tensor], dev: int, dtype, name: str):
    """Device pointer of a contiguous tensor (None: NULL) after its checks."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected CUDA device {dev}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _shaped(t: Optional[torch.Tensor], shape, dev: int, dtype, name: str):
    """The same of a tensor with a given shape."""
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    return _ptr(t, dev, dtype, name)


def _sized(t: Optional[torch.Tensor], n: int, dev: int, dtype, name: str):
    """The same of a tensor with n entries."""
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} entries (got {t.numel()})")
    return _ptr(t, dev, dtype, name)


def _page_size(cache: torch.Tensor, row_bytes: int, page_size: Optional[int], name: str) -> int:
    """Tokens of a page of `cache` (uint8 [num_pages, ...]) with row_bytes bytes a token."""
    if cache.dim() < 2:
        raise ValueError(f"{name} must be [num_pages, ...]")
    num_pages = cache.shape[0]
    page_bytes = cache.numel() // num_pages if num_pages else 0
    if page_size is None:
        page_size = page_bytes // row_bytes
    if page_size * row_bytes != page_bytes:
        raise ValueError(f"{name} pages hold {page_bytes} bytes, expected page_size*{row_bytes}")
    return page_size


def _width(block_table: torch.Tensor, batch: int) -> int:
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, max_pages_per_row] (got {list(shape)})")
    return shape[1]


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16 or float16")
    return code


# ---------------------------------------------------------------- attention
def mqa_attention_workspace(q: torch.Tensor, *, kv_heads: int = 1, topk: int = 0,
                            num_ctas: Optional[int] = None) -> torch.Tensor:
    """Workspace (uint8) for paged_mqa_attention_fp4 with this q [B, next_n, H, D],
    a schedule of num_ctas CTAs (None: the device's SMs) or token lists of length
    topk. One serves every layer and step with no more rows and positions than q's, but
    not two calls at the same time."""
    if q.dim() != 4:
        raise ValueError("q must be [B, next_n, H, D]")
    if _elsewhere(q, None):
        with _there(q, None):
            return mqa_attention_workspace(q, kv_heads=kv_heads, topk=topk, num_ctas=num_ctas)
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(q.device).multi_processor_count
    B, next_n, H, D = q.shape
    p = _ATTENTION.pack(B, next_n, H, kv_heads, D, 64, 1, 1, topk, num_ctas, _dtype(q, "q"), 0,
                        1.0, 0, 0, 0, 0, 0, 0)
    return torch.empty(_workspace_bytes(p), dtype=_BYTE, device=q.device)


def _workspace_bytes(params: bytes) -> int:
    size = ctypes.c_uint64(0)
    _check(_lib().mqa_attention_workspace_size(params, ctypes.byref(size)))
    return size.value


def paged_mqa_attention_fp4(q, k_cache, v_cache, block_table, context_lens, schedule=None, *,
                            kv_heads: int = 1, scale: Optional[float] = None,
                            indices: Optional[torch.Tensor] = None,
                            page_size: Optional[int] = None,
                            out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, with_lse: bool = False,
                            workspace: Optional[torch.Tensor] = None, flags: int = 0,
                            status: Optional[torch.Tensor] = None, stream=None):
    """Softmax attention over a paged FP4 cache; see include/mqa_cache.h.

    q: bf16 or f16 [B, next_n, H, D], last dimension contiguous, other strides
    multiples of 8; k_cache, v_cache: uint8 [num_pages, kv_heads * page_size *
    (D/2 + D/16)]; block_table int32 [B, max_pages]; context_lens int32 [B].
    Either `schedule` (mqa_logits_schedule of these context_lens: every cached
    token) or `indices` (int32 [B, next_n, k], as mqa_logits_topk gives them).
    scale: of the scores, 1/sqrt(D) if None. workspace: see
    mqa_attention_workspace; allocated if None. Returns out [B, next_n, H, D] of
    q's type, or (out, lse) with lse fp32 [B, next_n, H]."""
    if q.dim() != 4:
        raise ValueError("q must be [B, next_n, H, D]")
    if (schedule is None) == (indices is None):
        raise ValueError("give either schedule or indices")
    B, next_n, H, D = shape = q.shape
    sb, sn, sh, sd = q.stride()
    if sd != 1:
        raise ValueError("the last dimension of q must be contiguous")
    dtype = _dtype(q, "q")
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"k_cache and v_cache differ in shape ({list(k_cache.shape)}, "
                         f"{list(v_cache.shape)})")
    page_size = _page_size(k_cache, kv_heads * (D // 2 + D // 16), page_size, "k_cache")
    width = _width(block_table, B)
    if indices is None:
        topk, num_ctas = 0, schedule.numel() // 2 - 1
    else:
        topk, num_ctas = indices.shape[-1], 0
        if indices.shape != (B, next_n, topk):
            raise ValueError(f"indices must be [{B}, {next_n}, k] (got {list(indices.shape)})")
        if topk < 1:
            raise ValueError("indices must list at least one entry a position")
    if _elsewhere(q, stream):
        with _there(q, stream):
            return paged_mqa_attention_fp4(
                q, k_cache, v_cache, block_table, context_lens, schedule, kv_heads=kv_heads,
                scale=scale, indices=indices, page_size=page_size, out=out, lse=lse,
                with_lse=with_lse, workspace=workspace, flags=flags, status=status)
    dev = q.get_device()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        out_ptr = out.data_ptr()
    else:
        out_ptr = _shaped(out, shape, dev, q.dtype, "out")
    if lse is not None:
        lse_ptr = _shaped(lse, shape[:3], dev, _FLOAT, "lse")
    elif with_lse:
        lse = q.new_empty((B, next_n, H), dtype=_FLOAT)
        lse_ptr = lse.data_ptr()
    else:
        lse_ptr = None
    st = _ptr(status, dev, _INT, "status") or 0
    if scale is None:
        scale = D ** -0.5

    def params(size):
        return _ATTENTION.pack(B, next_n, H, kv_heads, D, page_size, k_cache.shape[0], width, topk,
                               num_ctas, dtype, flags, scale, 0, sb, sn, sh, size, st)

    if workspace is None:
        workspace = torch.empty(_workspace_bytes(params(0)), dtype=_BYTE, device=q.device)
    _check(_lib().paged_mqa_attention_fp4(
        q.data_ptr(), _ptr(k_cache, dev, _BYTE, "k_cache"), _ptr(v_cache, dev, _BYTE, "v_cache"),
        _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"), _ptr(schedule, dev, _INT, "schedule"),
        _ptr(indices, dev, _INT, "indices"), out_ptr, lse_ptr,
        _ptr(workspace, dev, _BYTE, "workspace"), params(workspace.numel()), _stream(dev)))
    return out if lse is None else (out, lse)


# ---------------------------------------------------------------- appends
def _values(values, x, dev: int, name: str, wanted: bool):
    if values is None:
        if not wanted:
            return None, None
        values = torch.empty_like(x, memory_format=torch.contiguous_format)
    return values, _shaped(values, x.shape, dev, x.dtype, name)


def mqa_cache_append_fp8(x, kv_cache, block_table, context_lens, row_offsets=None, *,
                         page_size: Optional[int] = None, values: Optional[torch.Tensor] = None,
                         with_values: bool = False, flags: int = 0,
                         status: Optional[torch.Tensor] = None, stream=None):
    """Quantise new tokens x (bf16 or f16 [T, D]) into the FP8 cache that
    paged_mqa_logits_fp8 reads (uint8 [num_pages, page_size * (D + 4)]), at the last
    positions of their rows: row b's are x[row_offsets[b]:row_offsets[b + 1]] (int32
    [B + 1]; None: T / B a row), context_lens int32 [B] counts them already. With
    with_values (or `values` [T, D]) returns what the cache now holds for them, in
    x's type; see include/mqa_cache.h."""
    if x.dim() != 2:
        raise ValueError("x must be [T, D]")
    T, D = x.shape
    sx, sd = x.stride()
    if sd != 1:
        raise ValueError("the last dimension of x must be contiguous")
    dtype = _dtype(x, "x")
    B = block_table.shape[0]
    page_size = _page_size(kv_cache, D + 4, page_size, "kv_cache")
    width = _width(block_table, B)
    if _elsewhere(x, stream):
        with _there(x, stream):
            return mqa_cache_append_fp8(
                x, kv_cache, block_table, context_lens, row_offsets, page_size=page_size,
                values=values, with_values=with_values, flags=flags, status=status)
    dev = x.get_device()
    values, vp = _values(values, x, dev, "values", with_values)
    _check(_lib().mqa_cache_append_fp8(
        x.data_ptr(), _ptr(kv_cache, dev, _BYTE, "kv_cache"),
        _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"),
        _sized(row_offsets, B + 1, dev, _INT, "row_offsets"), vp,
        _APPEND.pack(B, T, 1, D, page_size, kv_cache.shape[0], width, dtype, flags, 0, sx, 0, 0, 0,
                     _ptr(status, dev, _INT, "status") or 0), _stream(dev)))
    return values


def mqa_cache_append_fp4(k, v, k_cache, v_cache, block_table, context_lens, row_offsets=None, *,
                         page_size: Optional[int] = None,
                         k_values: Optional[torch.Tensor] = None,
                         v_values: Optional[torch.Tensor] = None, with_values: bool = False,
                         flags: int = 0, status: Optional[torch.Tensor] = None, stream=None):
    """Quantise new tokens k and v (bf16 or f16 [T, kv_heads, D]) into FP4 caches
    (uint8 [num_pages, kv_heads * page_size * (D/2 + D/16)]); v and v_cache may be
    None (keys alone, as paged_mqa_logits_fp4 reads them). Rows and positions as
    for mqa_cache_append_fp8. With with_values (or k_values, v_values) returns
    (k_values, v_values), what the caches now hold for the tokens, in their type."""
    if k.dim() != 3:
        raise ValueError("k must be [T, kv_heads, D]")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    T, heads, D = k.shape
    kt, kh, sd = k.stride()
    vt = vh = 0
    dtype = _dtype(k, "k")
    if v is not None:
        if v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("v must have the shape and type of k")
        if v_cache.shape != k_cache.shape:
            raise ValueError("v_cache must have the shape of k_cache")
        vt, vh, vd = v.stride()
        if vd != 1:
            raise ValueError("the last dimension of v must be contiguous")
    elif v_values is not None:
        raise ValueError("v_values without v")
    if sd != 1:
        raise ValueError("the last dimension of k must be contiguous")
    B = block_table.shape[0]
    page_size = _page_size(k_cache, heads * (D // 2 + D // 16), page_size, "k_cache")
    width = _width(block_table, B)
    if _elsewhere(k, stream):
        with _there(k, stream):
            return mqa_cache_append_fp4(
                k, v, k_cache, v_cache, block_table, context_lens, row_offsets, page_size=page_size,
                k_values=k_values, v_values=v_values, with_values=with_values, flags=flags,
                status=status)
    dev = k.get_device()
    vp = vvp = None
    if v is not None:
        if v.get_device() != dev:
            raise ValueError(f"v is on {v.device}, expected CUDA device {dev}")
        vp = v.data_ptr()
        v_values, vvp = _values(v_values, v, dev, "v_values", with_values)
    k_values, kvp = _values(k_values, k, dev, "k_values", with_values)
    _check(_lib().mqa_cache_append_fp4(
        k.data_ptr(), vp, _ptr(k_cache, dev, _BYTE, "k_cache"),
        _ptr(v_cache, dev, _BYTE, "v_cache"), _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"),
        _sized(row_offsets, B + 1, dev, _INT, "row_offsets"), kvp, vvp,
        _APPEND.pack(B, T, heads, D, page_size, k_cache.shape[0], width, dtype, flags, 0, kt, kh,
                     vt, vh, _ptr(status, dev, _INT, "status") or 0), _stream(dev)))
    return None if k_values is None and v_values is None else (k_values, v_values)


# ---------------------------------------------------------------- pages
def mqa_pages_fork(block_table, context_lens, parents, page_refs, *, page_size: int,
                   out_table: Optional[torch.Tensor] = None,
                   out_lens: Optional[torch.Tensor] = None, flags: int = 0,
                   status: Optional[torch.Tensor] = None, stream=None):
    """New rows that go on from old ones, sharing their pages: row r from row
    parents[r] (int32 [R]; -1: an empty row). page_refs (int32 [num_pages], how many
    table entries point at each page) is recounted in place for the new table.
    Returns (out_table int32 [R, max_pages], out_lens int32 [R])."""
    B, R = block_table.shape[0], parents.numel()
    width = _width(block_table, B)
    if _elsewhere(page_refs, stream):
        with _there(page_refs, stream):
            return mqa_pages_fork(block_table, context_lens, parents, page_refs,
                                  page_size=page_size, out_table=out_table, out_lens=out_lens,
                                  flags=flags, status=status)
    dev = page_refs.get_device()
    if out_table is None:
        out_table = page_refs.new_empty((R, width), dtype=_INT)
    if out_lens is None:
        out_lens = page_refs.new_empty((R,), dtype=_INT)
    _check(_lib().mqa_pages_fork(
        _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"), _ptr(parents, dev, _INT, "parents"),
        _ptr(page_refs, dev, _INT, "page_refs"),
        _shaped(out_table, (R, width), dev, _INT, "out_table"),
        _sized(out_lens, R, dev, _INT, "out_lens"),
        _PAGES.pack(B, R, width, page_refs.numel(), page_size, flags,
                    _ptr(status, dev, _INT, "status") or 0), _stream(dev)))
    return out_table, out_lens


def mqa_pages_resize(block_table, context_lens, new_lens, page_refs, *, page_size: int,
                     copy_src: Optional[torch.Tensor] = None,
                     copy_dst: Optional[torch.Tensor] = None, flags: int = 0,
                     status: Optional[torch.Tensor] = None, stream=None):
    """Give every row the length new_lens[b] (int32 [B]), in place: pages behind a
    new end are freed, growing rows take free pages, and a shared page that a row
    is about to write to is replaced by one of its own. Returns (copy_src,
    copy_dst), int32 [B]: the page copies to make (mqa_pages_copy), -1 for none.
    Rows for which no pages were left keep their length (context_lens tells;
    MQA_STATUS_NO_PAGES)."""
    B = block_table.shape[0]
    width = _width(block_table, B)
    if _elsewhere(page_refs, stream):
        with _there(page_refs, stream):
            return mqa_pages_resize(block_table, context_lens, new_lens, page_refs,
                                    page_size=page_size, copy_src=copy_src, copy_dst=copy_dst,
                                    flags=flags, status=status)
    dev = page_refs.get_device()
    if copy_src is None and copy_dst is None:
        copy_src, copy_dst = page_refs.new_empty((2, B), dtype=_INT)
    elif copy_src is None:
        copy_src = torch.empty_like(copy_dst)
    elif copy_dst is None:
        copy_dst = torch.empty_like(copy_src)
    _check(_lib().mqa_pages_resize(
        _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"),
        _sized(new_lens, B, dev, _INT, "new_lens"), _ptr(page_refs, dev, _INT, "page_refs"),
        _sized(copy_src, B, dev, _INT, "copy_src"), _sized(copy_dst, B, dev, _INT, "copy_dst"),
        _PAGES.pack(B, 0, width, page_refs.numel(), page_size, flags,
                    _ptr(status, dev, _INT, "status") or 0), _stream(dev)))
    return copy_src, copy_dst


def mqa_pages_compact(block_table, context_lens, page_refs, *, page_size: int,
                      copy_src: Optional[torch.Tensor] = None,
                      copy_dst: Optional[torch.Tensor] = None,
                      count: Optional[torch.Tensor] = None,
                      page_map: Optional[torch.Tensor] = None, flags: int = 0,
                      status: Optional[torch.Tensor] = None, stream=None):
    """Pack the pages in use to the front of the pool: block_table and page_refs
    are renumbered in place. Returns (copy_src, copy_dst, count, page_map): the
    first count[0] pairs are the copies to make (mqa_pages_copy with `count`), and
    page_map[p] is page p's new number, -1 for a free page."""
    B, P = block_table.shape[0], page_refs.numel()
    width = _width(block_table, B)
    if _elsewhere(page_refs, stream):
        with _there(page_refs, stream):
            return mqa_pages_compact(block_table, context_lens, page_refs, page_size=page_size,
                                     copy_src=copy_src, copy_dst=copy_dst, count=count,
                                     page_map=page_map, flags=flags, status=status)
    dev = page_refs.get_device()
    copy_src, copy_dst, count, page_map = (
        page_refs.new_empty((n,), dtype=_INT) if t is None else t
        for t, n in ((copy_src, P // 2), (copy_dst, P // 2), (count, 1), (page_map, P)))
    _check(_lib().mqa_pages_compact(
        _ptr(block_table, dev, _INT, "block_table"),
        _sized(context_lens, B, dev, _INT, "context_lens"),
        _ptr(page_refs, dev, _INT, "page_refs"), _sized(copy_src, P // 2, dev, _INT, "copy_src"),
        _sized(copy_dst, P // 2, dev, _INT, "copy_dst"), _sized(count, 1, dev, _INT, "count"),
        _sized(page_map, P, dev, _INT, "page_map"),
        _PAGES.pack(B, 0, width, P, page_size, flags, _ptr(status, dev, _INT, "status") or 0),
        _stream(dev)))
    return copy_src, copy_dst, count, page_map


def mqa_pages_copy(caches: Union[torch.Tensor, Sequence[torch.Tensor]], src, dst, count=None, *,
                   flags: int = 0, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy pages src[i] to dst[i] (int32 [n], -1 for none) in one cache or in
    each of several (uint8 [num_pages, bytes], bytes a multiple of 16): every
    layer's caches in one launch. count: int32 [1] on the device, only the first
    count[0] pairs."""
    if isinstance(caches, torch.Tensor):
        caches = (caches,)
    if not caches:
        raise ValueError("give at least one cache")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have one shape")
    first = caches[0]
    num_pages, n = first.shape[0], len(caches)
    if _elsewhere(first, stream):
        with _there(first, stream):
            return mqa_pages_copy(caches, src, dst, count, flags=flags, status=status)
    dev = first.get_device()
    ptrs, sizes = [], []
    for c in caches:
        if c.dim() < 2 or c.shape[0] != num_pages:
            raise ValueError(f"caches must all be [{num_pages}, ...]")
        ptrs.append(_ptr(c, dev, _BYTE, "cache"))
        sizes.append(c.numel() // max(num_pages, 1))
    _check(_lib().mqa_pages_copy(
        struct.pack(f"@{n}P", *ptrs), struct.pack(f"@{n}q", *sizes), n,
        _ptr(src, dev, _INT, "src"), _ptr(dst, dev, _INT, "dst"), src.numel(),
        _sized(count, 1, dev, _INT, "count"),
        _PAGES.pack(0, 0, 0, num_pages, 0, flags, _ptr(status, dev, _INT, "status") or 0),
        _stream(dev)))
