"""Torch-side calls of the paged key-value cache: appending new rows (bf16, or quantised to
e4m3 as they are written), reading rows back into contiguous bf16, and the attention of the
last tokens of every sequence over the cached rows.

The caller owns the page tables and the lengths (int32 device tensors) and decides which
pages a sequence holds; torch provides memory and the stream, every step is one call into
``libsparse_attn.so``. Calls may name another stream than the current one (``stream=``) and
tensors of another device than the current one: buffers that a call makes belong to the
stream and the device that it runs on. As for every call on a stream of its own, the caller
orders it behind what made the inputs and keeps them until it is done.

    cache = allocate_cache(num_pages, H, page=64, d=128, dtype=torch.float8_e4m3fn)
    cache_append(cache, k, v, page_table, start)          # k, v: [B,H,T,d] bf16 rows
    out = decode(q, cache, page_table, lens)              # q: [B,Hq,T,d], T new tokens
    cache_read(cache, page_table, lens, k_all, v_all)     # [B,H,N,d] bf16 for BlockSparseAttention
"""
from __future__ import annotations

import contextlib
import dataclasses
import functools
import math
from typing import Optional

import torch

from . import sparse_attn as C

PAGE_SIZES = (16, 32, 64, 128, 256)


@dataclasses.dataclass
class PagedCache:
    """A pool of pages (layouts as in include/sparse_attn.h)."""
    k: torch.Tensor                           # [num_pages,H,page,d] bf16 or float8_e4m3fn
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None    # [num_pages,H,page] float8_e8m0fnu (e4m3 only)
    v_scale: Optional[torch.Tensor] = None


def allocate_cache(num_pages: int, H: int, page: int = 64, d: int = 128, dtype=torch.bfloat16,
                   device="cuda") -> PagedCache:
    """An uninitialised pool. ``dtype`` bf16, or float8_e4m3fn with a scale per row."""
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError("a cache holds bfloat16 or float8_e4m3fn rows")
    if page not in PAGE_SIZES:
        raise ValueError(f"page must be one of {PAGE_SIZES}")
    rows = lambda: torch.empty(num_pages, H, page, d, dtype=dtype, device=device)
    if dtype == torch.bfloat16:
        return PagedCache(rows(), rows())
    scales = lambda: torch.empty(num_pages, H, page, dtype=torch.float8_e8m0fnu, device=device)
    return PagedCache(rows(), rows(), scales(), scales())


def _check_cache(c: PagedCache):
    """(cache type, device, shape) of a well-formed pool."""
    k, v = c.k, c.v
    dt, dev, shape = k.dtype, k.device, k.shape
    if not (k.is_cuda and len(shape) == 4 and k.is_contiguous() and v.is_contiguous()
            and v.shape == shape and v.dtype == dt and v.device == dev):
        raise ValueError("a cache is two contiguous CUDA tensors [num_pages,H,page,d] of one type")
    if dt == torch.bfloat16:
        if c.k_scale is not None or c.v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return C.SA_CACHE_BF16, dev, shape
    if dt != torch.float8_e4m3fn:
        raise ValueError("a cache holds bfloat16 or float8_e4m3fn rows")
    rows = shape[:3]
    for s in (c.k_scale, c.v_scale):
        if s is None or s.dtype != torch.float8_e8m0fnu or s.shape != rows \
                or not s.is_contiguous() or s.device != dev:
            raise ValueError("an e4m3 cache needs contiguous float8_e8m0fnu scales [num_pages,H,page]")
    return C.SA_CACHE_E4M3, dev, shape


def _strides(name, x, shape, device):
    """Element strides (b, h, t) of bf16 rows; a dimension of one has stride 0."""
    if x.dtype != torch.bfloat16 or x.shape != shape or x.device != device:
        raise ValueError(f"{name} must be a bf16 tensor {tuple(shape)} on {device}")
    sb, sh, st, sd = x.stride()
    if sd != 1 and x.numel():
        raise ValueError(f"the rows of {name} must be contiguous")
    B, H, T, _ = shape
    return sb if B > 1 else 0, sh if H > 1 else 0, st if T > 1 else 0


def _ints(name, x, shape, device):
    if x.dtype != torch.int32 or x.shape != shape or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}")


def _table(x, B, device):
    """(width, stride) of a page table [B, width] whose rows are contiguous."""
    shape = x.shape
    if x.dtype == torch.int32 and len(shape) == 2 and shape[0] == B and x.device == device:
        width = shape[1]
        if B * width == 0:
            return width, width
        stride, step = x.stride()
        if (width == 1 or step == 1) and (B == 1 or stride >= width):
            return width, stride if B > 1 else width
    raise ValueError(f"page_table must be an int32 tensor [{B}, width] on {device} with contiguous rows")


def _flag(err_flag, device):
    if err_flag is not None and (err_flag.dtype != torch.int32 or err_flag.device != device
                                 or err_flag.numel() < 1):
        raise ValueError(f"err_flag must be an int32 tensor on {device}")


# handle of a device's current stream (torch.cuda.current_stream builds a Stream around it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


@contextlib.contextmanager
def _guard(device, stream):
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context that makes ``device`` and ``stream`` current (nothing where they are)."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _HERE
    return _guard(device, stream)


def _apart(name, x):
    """Rows of a destination must not share memory."""
    need = x.shape[3] if x.numel() else 0     # elements from the first to the last of what is nested
    for st, n in sorted((x.stride(i), x.shape[i]) for i in range(3) if x.shape[i] > 1):
        if st < need:
            raise ValueError(f"the rows of {name} overlap")
        need += st * (n - 1)


def cache_append(cache: PagedCache, k, v, page_table, start, count=None, err_flag=None, stream=None):
    """Write rows t < count[b] (all T when ``count`` is None) of k, v [B,H,T,d] at positions
    start[b] + t of sequence b. Rows may be strided (a token-major projection seen as
    [B,H,T,d]); an e4m3 cache quantises them on the way."""
    dt, dev, (P, H, page, d) = _check_cache(cache)
    if k.dim() != 4:
        raise ValueError("k must be [B,H,T,d]")
    B, _, T, _ = k.shape
    shape = (B, H, T, d)
    ks, vs = _strides("k", k, shape, dev), _strides("v", v, shape, dev)
    width, stride = _table(page_table, B, dev)
    _ints("start", start, (B,), dev)
    if count is not None:
        _ints("count", count, (B,), dev)
    _flag(err_flag, dev)
    with _on(dev, stream):
        C.sparse_attn_cache_append(k, v, ks, vs, B, H, T, d, page_table, width, stride,
                                   start, count, cache.k, cache.v, cache.k_scale, cache.v_scale,
                                   dt, P, page, err_flag, _raw_stream(dev.index))


def cache_read(cache: PagedCache, page_table, lens, k, v, first=None, err_flag=None, stream=None):
    """Write rows first[b] <= t < lens[b] (from 0 when ``first`` is None) of every sequence
    to rows t of k, v [B,H,N,d] bf16; their other rows stay as they are."""
    dt, dev, (P, H, page, d) = _check_cache(cache)
    if k.dim() != 4:
        raise ValueError("k must be [B,H,N,d]")
    B, _, N, _ = k.shape
    shape = (B, H, N, d)
    ks, vs = _strides("k", k, shape, dev), _strides("v", v, shape, dev)
    _apart("k", k)
    _apart("v", v)
    width, stride = _table(page_table, B, dev)
    _ints("lens", lens, (B,), dev)
    if first is not None:
        _ints("first", first, (B,), dev)
    _flag(err_flag, dev)
    with _on(dev, stream):
        C.sparse_attn_cache_read(cache.k, cache.v, cache.k_scale, cache.v_scale, dt, P, page,
                                 page_table, width, stride, first, lens, B, H, N, d, k, v,
                                 ks, vs, err_flag, _raw_stream(dev.index))


@functools.lru_cache(maxsize=1024)
def _work_bytes(device, *shape):
    with torch.cuda.device(device):
        return C.sparse_attn_decode_work_bytes(*shape)


def decode(q, cache: PagedCache, page_table, lens, kv_idx=None, kv_cnt=None, scale=None,
           out_dtype=torch.float32, out=None, return_lse=False, err_flag=None, stream=None):
    """Attention of the last T tokens of every sequence over its cached rows.

    q [B,Hq,T,d] bf16 (rows may be strided), T <= 16; ``lens`` [B] counts the cached rows, the
    T new ones among them, so row t attends positions p < lens[b] - (T - 1 - t). Hq is a
    multiple of the cache's H: each kv head serves Hq / H query heads.
    ``kv_idx`` [B,H,cap] and ``kv_cnt`` [B,H] keep only the listed pages of each kv head, in
    the list format of :func:`attention.route` (its [B,H,1,cap] lists of one query block, with
    block = page, are taken as they are; a list may be empty, and cap may be 0). Routing lists per
    query head: where Hq > H the caller joins the lists of a kv head's group. A row that attends
    nothing is 0, its lse -inf. Tables and lists no wider than needed run short sequences faster.
    Returns ``out`` [B,Hq,T,d] (fp32, or bf16 by ``out_dtype``), and with ``return_lse`` also
    the fp32 log-sum-exp [B,Hq,T] of the scaled logits, by which partial results merge."""
    dt, dev, (P, H, page, d) = _check_cache(cache)
    if q.dim() != 4:
        raise ValueError("q must be [B,Hq,T,d]")
    B, Hq, T, _ = q.shape
    qs = _strides("q", q, (B, Hq, T, d), dev)
    width, stride = _table(page_table, B, dev)
    _ints("lens", lens, (B,), dev)
    cap = 0
    if (kv_idx is None) != (kv_cnt is None):
        raise ValueError("kv_idx and kv_cnt go together")
    if kv_idx is not None:
        if kv_idx.dim() == 4 and kv_idx.shape[2] == 1:
            kv_idx = kv_idx[:, :, 0]
        if kv_cnt.dim() == 3 and kv_cnt.shape[2] == 1:
            kv_cnt = kv_cnt[:, :, 0]
        cap = kv_idx.shape[-1]
        _ints("kv_idx", kv_idx, (B, H, cap), dev)
        _ints("kv_cnt", kv_cnt, (B, H), dev)
        if cap == 0:
            kv_idx = kv_cnt      # lists without room are not read, but an empty tensor has no address
    _flag(err_flag, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty(B, Hq, T, d, dtype=out_dtype, device=dev)
        elif out.device != dev or tuple(out.shape) != (B, Hq, T, d) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous tensor {(B, Hq, T, d)} on {dev}")
        if out.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("the output is float32 or bfloat16")
        lse = torch.empty(B, Hq, T, dtype=torch.float32, device=dev) if return_lse else None
        odt = C.SA_OUT_F32 if out.dtype == torch.float32 else C.SA_OUT_BF16
        need = _work_bytes(dev.index, B, Hq, H, T, d, dt, page, width, -1 if kv_idx is None else cap, odt)
        # scratch of this call alone: calls on other streams and captured graphs have their own
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        C.sparse_attn_decode(q, qs, B, Hq, H, T, d, cache.k, cache.v, cache.k_scale, cache.v_scale,
                             dt, P, page, page_table, width, stride, lens, kv_idx, kv_cnt, cap,
                             1.0 / math.sqrt(d) if scale is None else scale, work, out,
                             odt, lse, err_flag, _raw_stream(dev.index))
    return (out, lse) if return_lse else out


def check(err_flag):
    """Raise SA_ERR_INDEX if an earlier call met a page number, length or position out of
    range (synchronises). The flag is sticky: clear it with ``err_flag.zero_()``."""
    if int(err_flag.item()) & C.SA_FLAG_INDEX:
        raise C.SparseAttnError(C.SA_ERR_INDEX, "a page number, length or position of a paged "
                                "cache is out of range; the rows it stands for were left out")
