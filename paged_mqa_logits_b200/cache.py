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
from typing import Optional, Sequence, Union

import torch

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
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


def declare(lib) -> None:
    """Argument types of the entry points of include/mqa_cache.h."""
    a, n, p = (ctypes.POINTER(t) for t in (AttentionParams, AppendParams, PagesParams))
    for name, types in {
        "paged_mqa_attention_fp4": [_P] * 10 + [a, _P],
        "mqa_attention_workspace_size": [a, ctypes.POINTER(ctypes.c_uint64)],
        "mqa_cache_append_fp8": [_P] * 6 + [n, _P],
        "mqa_cache_append_fp4": [_P] * 9 + [n, _P],
        "mqa_pages_fork": [_P] * 6 + [p, _P],
        "mqa_pages_resize": [_P] * 6 + [p, _P],
        "mqa_pages_compact": [_P] * 7 + [p, _P],
        "mqa_pages_copy": [_P, _P, _I32, _P, _P, _I32, _P, p, _P],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int


def _lib():
    from . import library
    return library()


def _check(rc: int) -> None:
    if rc != 0:
        from . import _check as check
        check(rc)


class _Call:
    """Device and stream of one call: entered around the allocations and the launch."""

    __slots__ = ("device", "stream", "_guards")

    def __init__(self, device: torch.device, stream):
        if device.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        self.device, self._guards = device, None
        guards = []
        if device.index != torch.cuda.current_device():
            guards.append(torch.cuda.device(device))
        if stream is None:
            self.stream = torch.cuda.current_stream(device).cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.stream = stream.cuda_stream
            guards.append(torch.cuda.stream(stream))
        if guards:
            self._guards = contextlib.ExitStack()
            for g in guards:
                self._guards.enter_context(g)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self._guards is not None:
            self._guards.close()

    def ptr(self, t: Optional[torch.Tensor], name: str, dtype, shape=None, numel=None):
        """Device pointer of a contiguous tensor (None: NULL) after its checks."""
        if t is None:
            return None
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, expected {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{name} must hold {numel} entries (got {t.numel()})")
        return t.data_ptr()

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)


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


def _table(call: _Call, block_table, context_lens, batch):
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, max_pages_per_row] "
                         f"(got {list(block_table.shape)})")
    return (call.ptr(block_table, "block_table", torch.int32),
            call.ptr(context_lens, "context_lens", torch.int32, numel=batch))


# ---------------------------------------------------------------- attention
def mqa_attention_workspace(q: torch.Tensor, *, kv_heads: int = 1, topk: int = 0,
                            num_ctas: Optional[int] = None) -> torch.Tensor:
    """Workspace (uint8) for paged_mqa_attention_fp4 with this q [B, next_n, H, D],
    a schedule of num_ctas CTAs (None: the device's SMs) or token lists of length
    topk. One serves every layer and step, but not two calls at the same time."""
    if q.dim() != 4:
        raise ValueError("q must be [B, next_n, H, D]")
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(q.device).multi_processor_count
    B, next_n, H, D = q.shape
    with _Call(q.device, None) as call:
        p = AttentionParams(B, next_n, H, kv_heads, D, 64, 1, 1, topk, num_ctas,
                            _dtype(q, "q"), 0, 1.0, 0)
        size = ctypes.c_uint64(0)
        _check(_lib().mqa_attention_workspace_size(ctypes.byref(p), ctypes.byref(size)))
        return call.empty(size.value, torch.uint8)


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16 or float16")
    return _DTYPES[t.dtype]


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
    B, next_n, H, D = q.shape
    if q.stride(3) != 1:
        raise ValueError("the last dimension of q must be contiguous")
    dtype = _dtype(q, "q")
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"k_cache and v_cache differ in shape ({list(k_cache.shape)}, "
                         f"{list(v_cache.shape)})")
    page_size = _page_size(k_cache, kv_heads * (D // 2 + D // 16), page_size, "k_cache")
    topk, num_ctas = 0, 0
    if indices is not None:
        if indices.dim() != 3 or indices.shape[0] != B or indices.shape[1] != next_n:
            raise ValueError(f"indices must be [{B}, {next_n}, k] (got {list(indices.shape)})")
        topk = indices.shape[2]
        if topk < 1:
            raise ValueError("indices must list at least one entry a position")
    else:
        num_ctas = schedule.numel() // 2 - 1
    with _Call(q.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        sched = call.ptr(schedule, "schedule", torch.int32)
        idx = call.ptr(indices, "indices", torch.int32)
        kp = call.ptr(k_cache, "k_cache", torch.uint8)
        vp = call.ptr(v_cache, "v_cache", torch.uint8)
        st = call.ptr(status, "status", torch.int32)
        if out is None:
            out = call.empty((B, next_n, H, D), q.dtype)
        op = call.ptr(out, "out", q.dtype, shape=q.shape)
        if lse is None and with_lse:
            lse = call.empty((B, next_n, H), torch.float32)
        lp = call.ptr(lse, "lse", torch.float32, shape=q.shape[:3])
        p = AttentionParams(B, next_n, H, kv_heads, D, page_size, k_cache.shape[0],
                            block_table.shape[1], topk, num_ctas, dtype, flags,
                            D ** -0.5 if scale is None else scale, 0, q.stride(0), q.stride(1),
                            q.stride(2), 0, st)
        lib = _lib()
        if workspace is None:
            size = ctypes.c_uint64(0)
            _check(lib.mqa_attention_workspace_size(ctypes.byref(p), ctypes.byref(size)))
            workspace = call.empty(size.value, torch.uint8)
        p.workspace_bytes = workspace.numel()
        wp = call.ptr(workspace, "workspace", torch.uint8)
        _check(lib.paged_mqa_attention_fp4(q.data_ptr(), kp, vp, table, lens, sched, idx, op, lp,
                                           wp, ctypes.byref(p), call.stream))
    return out if lse is None else (out, lse)


# ---------------------------------------------------------------- appends
def _tokens(call: _Call, x, name: str, heads: Optional[int]):
    """Pointer and strides of new tokens [T, D] (heads None) or [T, heads, D]."""
    if x.device != call.device:
        raise ValueError(f"{name} is on {x.device}, expected {call.device}")
    if x.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return x.data_ptr(), x.stride(0), 0 if heads is None else x.stride(1)


def _values(call: _Call, values, x, name: str, wanted: bool):
    if values is None and wanted:
        values = call.empty(x.shape, x.dtype)
    return values, call.ptr(values, name, x.dtype, shape=x.shape)


def _rows(call: _Call, row_offsets, batch: int):
    if row_offsets is None:
        return None
    return call.ptr(row_offsets, "row_offsets", torch.int32, numel=batch + 1)


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
    dtype = _dtype(x, "x")
    B = block_table.shape[0]
    page_size = _page_size(kv_cache, D + 4, page_size, "kv_cache")
    with _Call(x.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        xp, st, _ = _tokens(call, x, "x", None)
        values, vp = _values(call, values, x, "values", with_values)
        p = AppendParams(B, T, 1, D, page_size, kv_cache.shape[0], block_table.shape[1], dtype,
                         flags, 0, st, 0, 0, 0, call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_cache_append_fp8(
            xp, call.ptr(kv_cache, "kv_cache", torch.uint8), table, lens,
            _rows(call, row_offsets, B), vp, ctypes.byref(p), call.stream))
    return values


def mqa_cache_append_fp4(k, v, k_cache, v_cache, block_table, context_lens, row_offsets=None, *,
                         page_size: Optional[int] = None,
                         k_values: Optional[torch.Tensor] = None,
                         v_values: Optional[torch.Tensor] = None, with_values: bool = False,
                         flags: int = 0, status: Optional[torch.Tensor] = None, stream=None):
    """Quantise new tokens k and v (bf16 or f16 [T, kv_heads, D]) into FP4 caches
    (uint8 [num_pages, kv_heads * page_size * (D/2 + D/16)]); v and v_cache may be
    None (keys alone, as paged_mqa_logits_fp4 reads them). Rows and positions as
    for mqa_cache_append_fp8. With with_values returns (k_values, v_values), what
    the caches now hold for the tokens, in their type."""
    if k.dim() != 3:
        raise ValueError("k must be [T, kv_heads, D]")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    T, heads, D = k.shape
    dtype = _dtype(k, "k")
    if v is not None and (v.shape != k.shape or v.dtype != k.dtype):
        raise ValueError("v must have the shape and type of k")
    B = block_table.shape[0]
    page_size = _page_size(k_cache, heads * (D // 2 + D // 16), page_size, "k_cache")
    if v_cache is not None and v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have the shape of k_cache")
    if v is None and v_values is not None:
        raise ValueError("v_values without v")
    with _Call(k.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        kp, kt, kh = _tokens(call, k, "k", heads)
        vp, vt, vh = (None, 0, 0) if v is None else _tokens(call, v, "v", heads)
        k_values, kvp = _values(call, k_values, k, "k_values", with_values)
        vvp = None
        if v is not None:
            v_values, vvp = _values(call, v_values, v, "v_values", with_values)
        p = AppendParams(B, T, heads, D, page_size, k_cache.shape[0], block_table.shape[1], dtype,
                         flags, 0, kt, kh, vt, vh, call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_cache_append_fp4(
            kp, vp, call.ptr(k_cache, "k_cache", torch.uint8),
            call.ptr(v_cache, "v_cache", torch.uint8), table, lens, _rows(call, row_offsets, B),
            kvp, vvp, ctypes.byref(p), call.stream))
    return (k_values, v_values) if with_values or k_values is not None or v_values is not None else None


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
    with _Call(page_refs.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        if out_table is None:
            out_table = call.empty((R, block_table.shape[1]), torch.int32)
        if out_lens is None:
            out_lens = call.empty((R,), torch.int32)
        p = PagesParams(B, R, block_table.shape[1], page_refs.numel(), page_size, flags,
                        call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_pages_fork(
            table, lens, call.ptr(parents, "parents", torch.int32),
            call.ptr(page_refs, "page_refs", torch.int32),
            call.ptr(out_table, "out_table", torch.int32, shape=(R, block_table.shape[1])),
            call.ptr(out_lens, "out_lens", torch.int32, numel=R), ctypes.byref(p), call.stream))
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
    with _Call(page_refs.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        if copy_src is None:
            copy_src = call.empty((B,), torch.int32)
        if copy_dst is None:
            copy_dst = call.empty((B,), torch.int32)
        p = PagesParams(B, 0, block_table.shape[1], page_refs.numel(), page_size, flags,
                        call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_pages_resize(
            table, lens, call.ptr(new_lens, "new_lens", torch.int32, numel=B),
            call.ptr(page_refs, "page_refs", torch.int32),
            call.ptr(copy_src, "copy_src", torch.int32, numel=B),
            call.ptr(copy_dst, "copy_dst", torch.int32, numel=B), ctypes.byref(p), call.stream))
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
    with _Call(page_refs.device, stream) as call:
        table, lens = _table(call, block_table, context_lens, B)
        copy_src, copy_dst, count, page_map = (
            call.empty((n,), torch.int32) if t is None else t
            for t, n in ((copy_src, P // 2), (copy_dst, P // 2), (count, 1), (page_map, P)))
        p = PagesParams(B, 0, block_table.shape[1], P, page_size, flags,
                        call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_pages_compact(
            table, lens, call.ptr(page_refs, "page_refs", torch.int32),
            call.ptr(copy_src, "copy_src", torch.int32, numel=P // 2),
            call.ptr(copy_dst, "copy_dst", torch.int32, numel=P // 2),
            call.ptr(count, "count", torch.int32, numel=1),
            call.ptr(page_map, "page_map", torch.int32, numel=P), ctypes.byref(p), call.stream))
    return copy_src, copy_dst, count, page_map


def mqa_pages_copy(caches: Union[torch.Tensor, Sequence[torch.Tensor]], src, dst, count=None, *,
                   flags: int = 0, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy pages src[i] to dst[i] (int32 [n], -1 for none) in one cache or in
    each of several (uint8 [num_pages, bytes], bytes a multiple of 16): every
    layer's caches in one launch. count: int32 [1] on the device, only the first
    count[0] pairs."""
    if isinstance(caches, torch.Tensor):
        caches = (caches,)
    caches = list(caches)
    if not caches:
        raise ValueError("give at least one cache")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have one shape")
    num_pages = caches[0].shape[0]
    n = len(caches)
    with _Call(caches[0].device, stream) as call:
        ptrs, sizes = (_P * n)(), (_I64 * n)()
        for i, c in enumerate(caches):
            if c.dim() < 2 or c.shape[0] != num_pages:
                raise ValueError(f"caches must all be [{num_pages}, ...]")
            ptrs[i] = call.ptr(c, "cache", torch.uint8)
            sizes[i] = c.numel() // max(num_pages, 1)
        p = PagesParams(0, 0, 0, num_pages, 0, flags, call.ptr(status, "status", torch.int32))
        _check(_lib().mqa_pages_copy(
            ptrs, sizes, n, call.ptr(src, "src", torch.int32), call.ptr(dst, "dst", torch.int32),
            src.numel(), call.ptr(count, "count", torch.int32, numel=1), ctypes.byref(p),
            call.stream))
