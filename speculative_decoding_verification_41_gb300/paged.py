"""The paged key-value cache around a speculative step (include/dspark_paged.h),
argument checks and marshalling only, every step runs in the CUDA kernels of
libdspark.so. A call with its buffers goes through the _paged_binding module
(csrc/paged_binding.cpp), which makes the same checks in a fraction of the time;
what does not pass them there comes back to the ones here, and through ctypes.

  dspark_pages_reserve(...)    pages, slots, positions and row offsets of new tokens
  dspark_kv_append(...)        their keys and values into the cache
  dspark_paged_attention(...)  attention of the new tokens over the cache
  dspark_pages_release(...)    pages of rejected tokens and finished requests back

Caches are [num_pages, page_size, heads, D] tensors of any strides with
contiguous D: a cache stored [num_pages, heads, page_size, D] is passed as its
.transpose(1, 2).
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

from . import binding, build
from .binding import DSPARK_BF16, DsparkError, made_on

HEADER = os.path.join(binding.ROOT, "include", "dspark_paged.h")
EXPORTED = ("dspark_pages_reserve", "dspark_pages_release", "dspark_kv_append",
            "dspark_paged_attention")


def _header_const(name: str) -> int:
    return int(re.search(rf"#define {name} (\d+)", open(HEADER).read()).group(1))


DSPARK_F16 = _header_const("DSPARK_F16")
DSPARK_ERR_TOO_LARGE = 6
DSPARK_ERR_NO_PAGES = _header_const("DSPARK_ERR_NO_PAGES")
PAGED_MAX_ROWS = _header_const("DSPARK_PAGED_MAX_ROWS")
PAGED_MAX_CTAS = _header_const("DSPARK_PAGED_MAX_CTAS")
binding.STATUS_NAMES[DSPARK_ERR_NO_PAGES] = "DSPARK_ERR_NO_PAGES"
_DTYPES = {torch.bfloat16: DSPARK_BF16, torch.float16: DSPARK_F16}

_fns = None
_ext = None


def _native():
    """The _paged_binding module, with libdspark's functions bound. Raises if it has not been
    built: there is no fallback."""
    global _ext
    if _ext is None:
        fns = _load()
        if not build.binding_fits():  # its machine code knows one torch's tensors
            raise RuntimeError("the _paged_binding module is not built, or not for this Python and "
                               "torch; run `python -c 'import __graft_entry__ as g; g.build()'`")
        from . import _paged_binding
        _paged_binding.bind(*(ctypes.cast(fns[name], ctypes.c_void_p).value for name in EXPORTED))
        _ext = _paged_binding
    return _ext


def _load():
    global _fns
    if _fns is None:
        lib = binding.load()
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        lib.dspark_pages_reserve.argtypes = [vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp, i32,
                                             vp, vp, vp, vp, vp, vp, vp, vp]
        lib.dspark_pages_release.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp,
                                             vp, vp, vp, vp]
        lib.dspark_kv_append.argtypes = [vp, vp, i64, i64, vp, i32, i32, i32, i32, vp, vp, i64,
                                         i64, i64, i32, i32, vp, vp]
        lib.dspark_paged_attention.argtypes = [vp, i64, i64, vp, vp, i64, i64, i64, i32, i32, vp,
                                               i64, i32, vp, vp, i32, i32, i32, i32, i32, i32, f32,
                                               i32, i32, vp, vp, vp, vp, sz, vp]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        _fns = {name: getattr(lib, name) for name in EXPORTED}
    return _fns


def paged_attention_workspace_bytes(Hq: int, Hkv: int, max_new: int, D: int) -> int:
    """Python statement of DSPARK_PAGED_ATTENTION_WS_BYTES (include/dspark_paged.h)."""
    rows = min(16 * (-(-(Hq // Hkv) * max_new // 16)), PAGED_MAX_ROWS)
    return ((PAGED_MAX_CTAS * 64 + 255) & ~255) + 2 * PAGED_MAX_CTAS * rows * (4 * D + 8)


_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice
_I32, _I64 = torch.int32, torch.int64


def _index(name: str, t) -> int:
    """The device number of the call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libdspark has no CPU path)")
    return t.get_device()


def _want(name: str, t: torch.Tensor, dtype, index: int, shape=None):
    """A contiguous CUDA tensor of this type, place and shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous() and (shape is None or t.shape == shape)):
        return
    device = torch.device("cuda", index)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libdspark has no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _table(block_table: torch.Tensor, B: int, index: int):
    """Stride and width of a block table's rows."""
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise ValueError("block_table must be a CUDA tensor (libdspark has no CPU path)")
    if block_table.dtype is not _I32 or block_table.get_device() != index:
        raise ValueError(f"block_table must be torch.int32 on cuda:{index}")
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages]")
    width = shape[1]
    stride, inner = block_table.stride()
    if inner != 1 and width > 1 and B > 0:
        raise ValueError("rows of block_table must be contiguous")
    return (stride if B > 1 else width), width


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, index: int):
    """Shape, strides and type number of the two caches."""
    if not isinstance(v_cache, torch.Tensor) or v_cache.get_device() != index:
        raise ValueError(f"v_cache must be a CUDA tensor on cuda:{index}")
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError("caches must be [pages, page_size, heads, D] with contiguous D")
    if v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    dtype = _DTYPES.get(k_cache.dtype)
    if dtype is None or v_cache.dtype is not k_cache.dtype:
        raise ValueError(f"caches must be bfloat16 or float16 alike, got {k_cache.dtype} and "
                         f"{v_cache.dtype}")
    return shape, stride, dtype


def _on(stream, index: int) -> int:
    """The stream's handle; a stream of another device than the tensors' is refused."""
    if stream is None:
        return _raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _handle(stream, t):
    """A given stream's handle for the usual path; None: the current stream."""
    if stream is None:
        return None
    return _on(stream, t.get_device() if isinstance(t, torch.Tensor) else -1)


def _fn(name: str, index: int):
    """The library's function, called on the tensors' device."""
    fn = (_fns or _load())[name]
    if _get_device() == index:
        return fn

    def there(*args):
        with torch.cuda.device(index):
            return fn(*args)
    return there


def _checked(name: str, status: torch.Tensor, stream):
    """Wait for the call and raise on a status that is not OK."""
    (stream or torch.cuda.current_stream(status.device)).synchronize()
    st = int(status.item())
    if st != 0:
        raise DsparkError(f"{name} (device)", st)


class ReserveBuffers:
    """Outputs of dspark_pages_reserve for B requests and max_tokens rows, so that
    repeated calls (and CUDA-graph capture) allocate nothing."""

    def __init__(self, B: int, max_tokens: int, device):
        dev = torch.device(device)
        self.B, self.max_tokens = B, max_tokens
        self.context_len = torch.empty(B, dtype=torch.int32, device=dev)
        self.row_off = torch.empty(B + 1, dtype=torch.int64, device=dev)
        self.draft_off = torch.empty(B + 1, dtype=torch.int64, device=dev)
        self.slot_map = torch.empty(max_tokens, dtype=torch.int32, device=dev)
        self.positions = torch.empty(max_tokens, dtype=torch.int32, device=dev)
        self.free_count = torch.empty(1, dtype=torch.int32, device=dev)
        self.device_status = torch.zeros(1, dtype=torch.int32, device=dev)


def dspark_pages_reserve(context_len: torch.Tensor, new_len: torch.Tensor,
                         block_table: torch.Tensor, free_pages: torch.Tensor,
                         free_count: torch.Tensor, *, page_size: int, max_tokens: int,
                         extra: int = 0, buffers: Optional[ReserveBuffers] = None, stream=None,
                         check: bool = False) -> dict:
    """Pages, slots and row offsets for new_len[r] + extra new tokens of every
    request (include/dspark_paged.h). block_table is written in place; free_pages
    is an array of all the pool's ids, the first free_count[0] of them free.

    Returns context_len [B], row_off [B+1] int64 (dspark_verify's target_row_off
    with extra = 1), draft_off [B+1] int64 (its draft_row_off), slot_map and
    positions [max_tokens], free_count [1], device_status [1] (device tensors).
    With check=True the call synchronises and raises on a non-OK device status."""
    buf, rc = buffers, None
    if buf is not None:
        rc = (_ext or _native()).reserve(
            context_len, new_len, block_table, free_pages, free_count, page_size, max_tokens,
            extra, buf.context_len, buf.row_off, buf.draft_off, buf.slot_map, buf.positions,
            buf.free_count, buf.device_status, _handle(stream, context_len))
    if rc is None:
        dev = _index("context_len", context_len)
        B = context_len.numel()
        _want("context_len", context_len, _I32, dev, (B,))
        _want("new_len", new_len, _I32, dev, (B,))
        stride, width = _table(block_table, B, dev)
        _want("free_pages", free_pages, _I32, dev)
        _want("free_count", free_count, _I32, dev, (1,))
        s = _on(stream, dev)
        if buf is None:
            buf = made_on(stream, lambda: ReserveBuffers(B, max_tokens, context_len.device))
        for name, dtype, n in (("context_len", _I32, B), ("row_off", _I64, B + 1),
                               ("draft_off", _I64, B + 1), ("slot_map", _I32, max_tokens),
                               ("positions", _I32, max_tokens), ("free_count", _I32, 1),
                               ("device_status", _I32, 1)):
            _want(f"buffers.{name}", getattr(buf, name), dtype, dev, (n,))
        rc = _fn("dspark_pages_reserve", dev)(
            context_len.data_ptr(), new_len.data_ptr(), extra, B, page_size, free_pages.numel(),
            block_table.data_ptr(), stride, width, free_pages.data_ptr(), free_count.data_ptr(),
            max_tokens, buf.context_len.data_ptr(), buf.row_off.data_ptr(),
            buf.draft_off.data_ptr(), buf.slot_map.data_ptr(), buf.positions.data_ptr(),
            buf.free_count.data_ptr(), buf.device_status.data_ptr(), s)
    if rc != 0:
        raise DsparkError("dspark_pages_reserve", rc)
    if check:
        _checked("dspark_pages_reserve", buf.device_status, stream)
    return {"context_len": buf.context_len, "row_off": buf.row_off, "draft_off": buf.draft_off,
            "slot_map": buf.slot_map, "positions": buf.positions, "free_count": buf.free_count,
            "device_status": buf.device_status}


class ReleaseBuffers:
    """Outputs of dspark_pages_release for B requests."""

    def __init__(self, B: int, device):
        dev = torch.device(device)
        self.B = B
        self.context_len = torch.empty(B, dtype=torch.int32, device=dev)
        self.free_count = torch.empty(1, dtype=torch.int32, device=dev)
        self.device_status = torch.zeros(1, dtype=torch.int32, device=dev)


def dspark_pages_release(context_len: torch.Tensor, reserved_len: torch.Tensor,
                         kept_len: torch.Tensor, block_table: torch.Tensor,
                         free_pages: torch.Tensor, free_count: torch.Tensor, *, page_size: int,
                         extra: int = 0, buffers: Optional[ReleaseBuffers] = None, stream=None,
                         check: bool = False) -> dict:
    """After the verification: request r keeps context_len[r] + kept_len[r] + extra
    of its reserved_len[r] tokens (kept_len[r] = -1: none, it is finished); the
    pages past them go back on free_pages, in place (include/dspark_paged.h).

    Returns context_len [B], free_count [1], device_status [1] (device tensors)."""
    buf, rc = buffers, None
    if buf is not None:
        rc = (_ext or _native()).release(
            context_len, reserved_len, kept_len, block_table, free_pages, free_count, page_size,
            extra, buf.context_len, buf.free_count, buf.device_status,
            _handle(stream, context_len))
    if rc is None:
        dev = _index("context_len", context_len)
        B = context_len.numel()
        _want("context_len", context_len, _I32, dev, (B,))
        _want("reserved_len", reserved_len, _I32, dev, (B,))
        _want("kept_len", kept_len, _I32, dev, (B,))
        stride, width = _table(block_table, B, dev)
        _want("free_pages", free_pages, _I32, dev)
        _want("free_count", free_count, _I32, dev, (1,))
        s = _on(stream, dev)
        if buf is None:
            buf = made_on(stream, lambda: ReleaseBuffers(B, context_len.device))
        for name, n in (("context_len", B), ("free_count", 1), ("device_status", 1)):
            _want(f"buffers.{name}", getattr(buf, name), _I32, dev, (n,))
        rc = _fn("dspark_pages_release", dev)(
            context_len.data_ptr(), reserved_len.data_ptr(), kept_len.data_ptr(), extra, B,
            page_size, free_pages.numel(), block_table.data_ptr(), stride, width,
            free_pages.data_ptr(), free_count.data_ptr(), buf.context_len.data_ptr(),
            buf.free_count.data_ptr(), buf.device_status.data_ptr(), s)
    if rc != 0:
        raise DsparkError("dspark_pages_release", rc)
    if check:
        _checked("dspark_pages_release", buf.device_status, stream)
    return {"context_len": buf.context_len, "free_count": buf.free_count,
            "device_status": buf.device_status}


def dspark_kv_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                     k_cache: torch.Tensor, v_cache: torch.Tensor, *,
                     device_status: Optional[torch.Tensor] = None, stream=None,
                     check: bool = False) -> dict:
    """Row i of k and v ([n, heads, D], any strides alike, contiguous D) into slot
    slot_map[i] of the caches, in place; negative slots are skipped
    (include/dspark_paged.h). slot_map may be longer than n (a reservation's whole
    map): its first n entries count. Returns device_status [1]."""
    rc = None
    if device_status is not None:
        rc = (_ext or _native()).append(k, v, slot_map, k_cache, v_cache, device_status,
                                        _handle(stream, k_cache))
    if rc is None:
        dev = _index("k_cache", k_cache)
        (pages, page_size, Hkv, D), (sp, st, sh, _), dtype = _cache(k_cache, v_cache, dev)
        for name, x in (("k", k), ("v", v)):
            if not isinstance(x, torch.Tensor) or x.get_device() != dev:
                raise ValueError(f"{name} must be a CUDA tensor on cuda:{dev}")
        shape, strides = k.shape, k.stride()
        if len(shape) != 3 or strides[2] != 1 or shape[1] != Hkv or shape[2] != D:
            raise ValueError(f"k must be [n, {Hkv}, {D}] with contiguous rows")
        if k.dtype is not k_cache.dtype or v.dtype is not k.dtype:
            raise ValueError(f"k and v must be {k_cache.dtype}, got {k.dtype} and {v.dtype}")
        if v.shape != shape or v.stride() != strides:
            raise ValueError("k and v must have the same shape and strides")
        n = shape[0]
        _want("slot_map", slot_map, _I32, dev)
        if slot_map.numel() < n:
            raise ValueError(f"slot_map has {slot_map.numel()} entries for {n} rows")
        s = _on(stream, dev)
        if device_status is None:
            device_status = made_on(
                stream, lambda: torch.empty(1, dtype=_I32, device=k_cache.device))
        else:
            _want("device_status", device_status, _I32, dev, (1,))
        rc = _fn("dspark_kv_append", dev)(
            k.data_ptr(), v.data_ptr(), strides[0], strides[1], slot_map.data_ptr(), n, Hkv, D,
            dtype, k_cache.data_ptr(), v_cache.data_ptr(), sp, st, sh, page_size, pages,
            device_status.data_ptr(), s)
    if rc != 0:
        raise DsparkError("dspark_kv_append", rc)
    if check:
        _checked("dspark_kv_append", device_status, stream)
    return {"device_status": device_status}


class AttentionBuffers:
    """Outputs and workspace of dspark_paged_attention for n_tokens rows, so that
    repeated calls (and CUDA-graph capture) allocate nothing."""

    def __init__(self, n_tokens: int, Hq: int, Hkv: int, D: int, max_new: int, dtype, device,
                 with_lse: bool = False):
        dev = torch.device(device)
        self.out = torch.empty(n_tokens, Hq, D, dtype=dtype, device=dev)
        self.lse = torch.empty(n_tokens, Hq, dtype=torch.float32, device=dev) if with_lse else None
        self.device_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(paged_attention_workspace_bytes(Hq, Hkv, max_new, D),
                                     dtype=torch.uint8, device=dev)


def dspark_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_table: torch.Tensor, context_len: torch.Tensor,
                           row_off: torch.Tensor, *, scale: float, max_new: int, window: int = 0,
                           with_lse: bool = False, buffers: Optional[AttentionBuffers] = None,
                           stream=None, check: bool = False) -> dict:
    """Attention of each request's newest tokens over its pages
    (include/dspark_paged.h). q is [n_tokens, Hq, D] (contiguous D); rows
    row_off[r] .. row_off[r+1]-1, at most max_new, are the last ones of request
    r's context_len[r] cached tokens, and each sees those up to itself (with a
    window, the last `window` of them).

    Returns out [n_tokens, Hq, D], lse [n_tokens, Hq] float32 (or None) and
    device_status [1] (device tensors)."""
    buf, rc = buffers, None
    if buf is not None:
        if with_lse and buf.lse is None:
            raise ValueError("buffers were made without lse (AttentionBuffers(..., with_lse=True))")
        rc = (_ext or _native()).attention(
            q, k_cache, v_cache, block_table, context_len, row_off, scale, max_new, window,
            buf.out, buf.lse if with_lse else None, buf.device_status, buf.workspace,
            _handle(stream, k_cache))
    if rc is None:
        dev = _index("k_cache", k_cache)
        (pages, page_size, Hkv, D), (sp, st, sh, _), dtype = _cache(k_cache, v_cache, dev)
        if not isinstance(q, torch.Tensor) or q.get_device() != dev:
            raise ValueError(f"q must be a CUDA tensor on cuda:{dev}")
        if q.dtype is not k_cache.dtype:
            raise ValueError(f"q must be {k_cache.dtype}, got {q.dtype}")
        shape, strides = q.shape, q.stride()
        if len(shape) != 3 or strides[2] != 1 or shape[2] != D:
            raise ValueError(f"q must be [n_tokens, heads, {D}] with contiguous rows")
        n, Hq, _ = shape
        B = context_len.numel()
        _want("context_len", context_len, _I32, dev, (B,))
        _want("row_off", row_off, _I64, dev, (B + 1,))
        stride, width = _table(block_table, B, dev)
        if Hkv < 1 or Hq < 1 or Hq % Hkv != 0 or max_new < 1:
            raise ValueError(f"{Hq} query heads on {Hkv} key heads, max_new {max_new}")
        s = _on(stream, dev)
        if buf is None:
            buf = made_on(stream, lambda: AttentionBuffers(n, Hq, Hkv, D, max_new, q.dtype,
                                                           q.device, with_lse))
        _want("buffers.out", buf.out, q.dtype, dev, shape)
        if with_lse:
            _want("buffers.lse", buf.lse, torch.float32, dev, (n, Hq))
        _want("buffers.device_status", buf.device_status, _I32, dev, (1,))
        _want("buffers.workspace", buf.workspace, torch.uint8, dev)
        rc = _fn("dspark_paged_attention", dev)(
            q.data_ptr(), strides[0], strides[1], k_cache.data_ptr(), v_cache.data_ptr(), sp, st,
            sh, page_size, pages, block_table.data_ptr(), stride, width, context_len.data_ptr(),
            row_off.data_ptr(), B, n, Hq, Hkv, D, max_new, scale, window, dtype,
            buf.out.data_ptr(), buf.lse.data_ptr() if with_lse else None,
            buf.device_status.data_ptr(), buf.workspace.data_ptr(), buf.workspace.numel(), s)
    if rc != 0:
        raise DsparkError("dspark_paged_attention", rc)
    if check:
        _checked("dspark_paged_attention", buf.device_status, stream)
    return {"out": buf.out, "lse": buf.lse if with_lse else None,
            "device_status": buf.device_status}
