"""The key/value cache in NVFP4: keys and values of attention held as packed
E2M1 codes with Four Over Six block scales, in pages.

    cache = fos.KVCache.empty(pages, page_size, heads, head_dim, k_amax, v_amax)
    q = fos.kv_append(cache, k, v, slots, positions=pos, cos_sin=table, q=q)
    y = fos.kv_attention(cache, q, cu_q, pages, kv_len, max_q)

kv_append rotates the new keys (and queries) to their positions and
quantizes the keys and values into their slots; kv_attention reads the codes
and scales; kv_read gives them back as bf16.  This module only checks
arguments, allocates outputs and workspaces, and hands pointers to the C ABI
(include/fos.h, where layouts and semantics are).  The calls run on the
device of their tensors, on `stream` or that device's current stream.  With
`stream`, the tensors passed in must be ready on it; outputs and workspaces
that the call allocates are that stream's.

Sources: Ultralytics glossary "FP4", "Como funciona FP4" (NVFP4: 16 values,
E4M3 block scale, FP32 scale); Hugging Face transformers doc "Four Over
Six", introduction (the adaptive block scale).
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple, Union

import torch

from . import fos

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _CacheC(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_tensor_scale", "v_tensor_scale")] + \
        [(n, _I64) for n in ("num_pages", "page_size", "heads", "head_dim", "codes_page_stride",
                             "scales_page_stride")]


class _RotaryC(ctypes.Structure):
    _fields_ = [("table", _P), ("positions", _P), ("max_positions", _I64), ("dim", _I32), ("interleaved", _I32)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = fos.lib()
        CP, RP, sz = ctypes.POINTER(_CacheC), ctypes.POINTER(_RotaryC), ctypes.c_size_t
        L.fos_kv_append.restype = _I32
        L.fos_kv_append.argtypes = [CP, _I32, _P, _I64, _P, _I64, _I64, _P, RP, _P, _I64, _P, _I64, _I64, _P, _P]
        L.fos_kv_read.restype = _I32
        L.fos_kv_read.argtypes = [CP, _P, _I64, _P, _P, _P, _P]
        L.fos_kv_attention_workspace_size.restype = sz
        L.fos_kv_attention_workspace_size.argtypes = [CP, _I64, _I64, _I64, _I64, _I64]
        L.fos_kv_attention.restype = _I32
        L.fos_kv_attention.argtypes = [CP, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, ctypes.c_float, _I32,
                                       _I64, _P, _I64, _P, _P, sz, _P, _P]
        _bound = L
    return _bound


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class KVCache:
    """The pools of one layer: k_codes, v_codes uint8 [pages, heads,
    page_size, head_dim/2], k_scales, v_scales uint8 [pages, heads,
    page_size, head_dim/16], k_tensor_scale, v_tensor_scale float32 [heads],
    all on one device.  Each page is contiguous; the pages of the two codes
    (and of the two scales) pools are the same distance apart, so slices of a
    larger allocation work.  fmt: "nvfp4_46" or "nvfp4_6", for what is
    appended (reading is the same).  The fields are fixed, since the calls pass
    on their addresses: new scales, say, are copied into k_tensor_scale."""

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                 k_tensor_scale: torch.Tensor, v_tensor_scale: torch.Tensor, fmt: str = "nvfp4_46"):
        _need(fmt in ("nvfp4_46", "nvfp4_6"), "fmt must be nvfp4_46 or nvfp4_6")
        _need(k_codes.dim() == 4, "codes must be [pages, heads, page_size, head_dim/2]")
        n, h, p, half = k_codes.shape
        dev = k_codes.device
        if dev.type != "cuda":
            raise TypeError("the pools must be CUDA tensors")
        for t, last in ((k_codes, half), (v_codes, half), (k_scales, half // 8), (v_scales, half // 8)):
            if t.dtype != torch.uint8:
                raise TypeError("the pools must be uint8 tensors")
            _need(tuple(t.shape) == (n, h, p, last) and t.device == dev, "the pools' shapes or devices do not match")
            _need(t.stride()[1:] == (p * last, last, 1), "a page of a pool must be contiguous")
        _need(k_codes.stride(0) == v_codes.stride(0) and k_scales.stride(0) == v_scales.stride(0),
              "the pools of keys and values must have the same distance between pages")
        for t in (k_tensor_scale, v_tensor_scale):
            if t.dtype != torch.float32:
                raise TypeError("the tensor scales must be float32")
            _need(tuple(t.shape) == (h,) and t.is_contiguous() and t.device == dev,
                  "the tensor scales must be [heads] on the pools' device")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_tensor_scale, self.v_tensor_scale, self.fmt, self.device = k_tensor_scale, v_tensor_scale, fmt, dev
        self.pages, self.heads, self.page_size, self.head_dim = n, h, p, 2 * half
        self._c = _CacheC(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                          k_tensor_scale.data_ptr(), v_tensor_scale.data_ptr(), n, p, h, 2 * half,
                          k_codes.stride(0), k_scales.stride(0))
        self._ref = ctypes.byref(self._c)
        self._dev, self._fmt, self._scale = k_codes.get_device(), fos.FMT[fmt], 1.0 / math.sqrt(2 * half)

    def __setattr__(self, name, value):
        if name in self.__dict__:           # __init__ sets each once
            raise AttributeError("the fields of a KVCache are fixed: copy into its tensors, or make another")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, k_amax: Union[float, torch.Tensor],
              v_amax: Union[float, torch.Tensor], fmt: str = "nvfp4_46", device="cuda") -> "KVCache":
        """An uninitialised cache.  k_amax, v_amax: the largest |value| to
        expect of each head's (rotated) keys and of its values, a number or
        float32 [heads]; larger ones saturate."""
        dev = torch.device(device)
        pools = [torch.empty(pages, heads, page_size, head_dim // n, dtype=torch.uint8, device=dev)
                 for n in (2, 16, 2, 16)]
        top = 2688.0 if fmt == "nvfp4_6" else 1792.0
        # a tensor as divisor: a number would be turned into its reciprocal, which is not the library's rounding
        top = torch.full((heads,), top, dtype=torch.float32, device=dev)
        st = [torch.as_tensor(a, dtype=torch.float32, device=dev).expand(heads) / top for a in (k_amax, v_amax)]
        return cls(*pools, *st, fmt=fmt)


# The device of the tensors as the current one (left as it was), and the raw
# handle of the stream to use on it.  Decoding steps launch a few microseconds
# of work a call, so the usual case asks for nothing but two integers.
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _call(cache: "KVCache", what: str, fn, stream, args) -> None:
    dev = cache._dev
    s = _current_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != 0:
        raise fos.FosError(st, what)


def _empty(x: torch.Tensor, shape, dtype, stream, output: bool = True) -> torch.Tensor:
    """A buffer of a call on `stream`, on x's device.  It comes from that stream's own memory:
    a block of the current stream's may still be in use by work that `stream`
    does not wait for.  An output is also kept from reuse until the current
    stream's work on it at its end is done."""
    if stream is None:
        return x.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        y = x.new_empty(shape, dtype=dtype)
    if output:
        y.record_stream(torch.cuda.current_stream(x.device))
    return y


def _empty_like(x: torch.Tensor, stream) -> torch.Tensor:
    if stream is None:                     # 1 us less than new_empty of x.shape
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _empty(x, x.shape, x.dtype, stream)


def _rows(name: str, x: torch.Tensor, tokens: int, heads: int, cache: "KVCache") -> int:
    """Checks x as rows of heads; the distance between tokens in elements."""
    if x.dtype is not torch.bfloat16 or x.get_device() != cache._dev:
        raise TypeError("%s must be a bfloat16 tensor on the cache's device" % name)
    dim = cache.head_dim
    if x.shape != (tokens, heads, dim):
        raise ValueError("%s must be [tokens, heads, head_dim]" % name)
    a, b, c = x.stride()
    if (c != 1 or (b != dim and heads > 1)) and tokens:
        raise ValueError("the heads of a token of %s must be contiguous" % name)
    return a if tokens > 1 else heads * dim       # the distance of a single token is free


def _ints(name: str, x: torch.Tensor, dtype, shape, cache: "KVCache") -> int:
    if x.dtype is not dtype or x.get_device() != cache._dev:
        raise TypeError("%s must be a %s tensor on the cache's device" % (name, str(dtype).replace("torch.", "")))
    if x.shape != shape or not x.is_contiguous():
        raise ValueError("%s must be contiguous %s" % (name, list(shape)))
    return x.data_ptr()


def _status(status: Optional[torch.Tensor], cache: "KVCache"):
    if status is None:
        return None
    if status.dtype is not torch.int32 or status.get_device() != cache._dev or status.numel() < 1:
        raise TypeError("status must be an int32 tensor on the cache's device")
    return status.data_ptr()


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
              positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
              interleaved: bool = False, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Quantize k, v bf16 [tokens, heads, head_dim] into the slots (int64
    [tokens], page * page_size + position in the page; negative: skip).

    cos_sin: float32 [max_positions, dim], dim/2 cosines then dim/2 sines for
    each position; with it the first dim values of each head of k (and q
    [tokens, q_heads, head_dim]) are turned by positions (int32 [tokens]), in
    pairs (i, i + dim/2), or (2i, 2i + 1) when interleaved.  Returns the
    rotated queries (q_out when given, which may be q), or None without q.
    fos_kv_append in include/fos.h has the rounding and the errors."""
    t = k.shape[0]
    h = cache.heads
    k_ld, v_ld = _rows("k", k, t, h, cache), _rows("v", v, t, h, cache)
    at = _ints("slots", slots, torch.int64, (t,), cache)
    rot = None
    q_ptr = out_ptr = None
    q_ld = out_ld = hq = 0
    if cos_sin is not None:
        _need(positions is not None, "cos_sin needs positions")
        _need(cos_sin.dim() == 2, "cos_sin must be [max_positions, dim]")
        n, dim = cos_sin.shape
        rot = ctypes.byref(_RotaryC(_ints("cos_sin", cos_sin, torch.float32, (n, dim), cache),
                                    _ints("positions", positions, torch.int32, (t,), cache), n, dim,
                                    1 if interleaved else 0))
    else:
        _need(positions is None, "positions need cos_sin")
    if q is not None:
        _need(rot is not None, "q is rotated: it needs positions and cos_sin")
        _need(q.dim() == 3, "q must be [tokens, heads, head_dim]")
        hq = q.shape[1]
        q_ld = _rows("q", q, t, hq, cache)
        if q_out is None:
            q_out, out_ld = _empty_like(q, stream), hq * cache.head_dim
        else:
            out_ld = _rows("q_out", q_out, t, hq, cache)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    else:
        _need(q_out is None, "q_out without q")
    _call(cache, "fos_kv_append", _lib().fos_kv_append, stream,
          (cache._ref, cache._fmt, k.data_ptr(), k_ld, v.data_ptr(), v_ld, t, at, rot, q_ptr, q_ld, out_ptr, out_ld,
           hq, _status(status, cache)))
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values of slots (int64 [tokens]) as the cache holds them:
    two bf16 tensors [tokens, heads, head_dim], zeros for negative slots."""
    _need(slots.dim() == 1, "slots must be [tokens]")
    t = slots.shape[0]
    at = _ints("slots", slots, torch.int64, (t,), cache)
    if out is None:
        out = _empty(slots, (2, t, cache.heads, cache.head_dim), torch.bfloat16, stream).unbind(0)
    else:
        for x in out:
            _rows("out", x, t, cache.heads, cache)
            _need(x.is_contiguous(), "out must be contiguous")
    k, v = out
    _call(cache, "fos_kv_read", _lib().fos_kv_read, stream,
          (cache._ref, at, t, k.data_ptr(), v.data_ptr(), _status(status, cache)))
    return k, v


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(heads: int, head_dim: int, page_size: int, total_q: int, batch: int, q_heads: int, max_q: int,
                     max_pages: int) -> int:
    c = _CacheC(heads=heads, head_dim=head_dim, page_size=page_size)
    return int(_lib().fos_kv_attention_workspace_size(ctypes.byref(c), total_q, batch, q_heads, max_q, max_pages))


def kv_attention_workspace_size(cache: KVCache, total_q: int, batch: int, q_heads: int, max_q: int,
                                max_pages: int) -> int:
    """Bytes of workspace kv_attention needs."""
    return _workspace_bytes(cache.heads, cache.head_dim, cache.page_size, total_q, batch, q_heads, max_q, max_pages)


def kv_attention(cache: KVCache, q: torch.Tensor, cu_q: torch.Tensor, pages: torch.Tensor, kv_len: torch.Tensor,
                 max_q: int, causal: bool = True, window: int = 0, scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Attention of ragged queries over the cached keys and values.

    q: bf16 [total_q, q_heads, head_dim], q_heads a multiple of the cache's
    heads; cu_q int32 [batch + 1], where each sequence's queries begin; pages
    int32 [batch, max_pages]; kv_len int32 [batch]; max_q the largest number
    of queries of a sequence.  causal: the queries are the last of their
    sequence (window > 0: each sees that many keys, its own among them);
    causal=False: each query sees all keys, as over an encoder's states.
    scale: 1/sqrt(head_dim) by default.  Returns out bf16, or (out, lse) with
    return_lse (lse float32 [total_q, q_heads]).  Queries that see no key get
    zeros and -inf; rows of out and lse that belong to no sequence are left
    as they were.  fos_kv_attention in include/fos.h has the details."""
    _need(q.dim() == 3, "q must be [total_q, q_heads, head_dim]")
    t, hq = q.shape[0], q.shape[1]
    q_ld = _rows("q", q, t, hq, cache)
    _need(hq > 0 and hq % cache.heads == 0, "q_heads must be a multiple of the cache's heads")
    _need(cu_q.dim() == 1 and cu_q.shape[0] >= 1, "cu_q must be [batch + 1]")
    _need(pages.dim() == 2, "pages must be [batch, max_pages]")
    _need(window >= 0 and (causal or window == 0), "window needs causal")
    b, most = cu_q.shape[0] - 1, pages.shape[1]
    cu, table = _ints("cu_q", cu_q, torch.int32, (b + 1,), cache), _ints("pages", pages, torch.int32, (b, most), cache)
    lens = _ints("kv_len", kv_len, torch.int32, (b,), cache)
    if out is None:
        out, out_ld = _empty_like(q, stream), hq * cache.head_dim
    else:
        out_ld = _rows("out", out, t, hq, cache)
    lse_ptr = None
    if lse is not None:
        lse_ptr = _ints("lse", lse, torch.float32, (t, hq), cache)
    elif return_lse:
        lse = _empty(q, (t, hq), torch.float32, stream)
        lse_ptr = lse.data_ptr()
    L = _lib()
    need = _workspace_bytes(cache.heads, cache.head_dim, cache.page_size, t, b, hq, max_q, most)
    if workspace is None and need:
        workspace = _empty(q, (need,), torch.uint8, stream, output=False)
    elif workspace is not None:
        _need(workspace.get_device() == cache._dev and workspace.is_contiguous(),
              "workspace must be contiguous and on the cache's device")
        need = workspace.numel() * workspace.element_size()
    _call(cache, "fos_kv_attention", L.fos_kv_attention, stream,
          (cache._ref, q.data_ptr(), q_ld, t, hq, cu, b, table, most, lens, max_q,
           cache._scale if scale is None else scale, 1 if causal else 0, window, out.data_ptr(), out_ld, lse_ptr,
           None if workspace is None else workspace.data_ptr(), need, _status(status, cache)))
    return (out, lse) if return_lse else out
