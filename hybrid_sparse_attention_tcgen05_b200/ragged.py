"""Calls over ragged batches and paged caches: rotary positions, the write of
new keys and values into the pages (plain or as 8-bit floats), reading them
back, and attention of packed prompts and of new tokens over the pages.

As the rest of the package these only check and marshal torch tensors; the
work is the library's (include/hysparse.h, "Ragged batches and paged caches").
Packed tensors are [T, H, d], the rows of all sequences one after the other;
they may be slices of one projection's output (any stride between rows that
is a multiple of 16 bytes).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import HsPagedCache

__all__ = ["rope", "rope_frequencies", "cache_write", "cache_read", "packed_attn", "chunk_attn_paged",
           "ragged_workspace_size"]

# what torch.cuda.current_device() and current_stream(dev).cuda_stream return,
# without the objects they make on the way (two microseconds a call)
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

_DTYPES = {torch.float32: _lib.HS_F32, torch.bfloat16: _lib.HS_BF16}
_POOL_DTYPES = {**_DTYPES, torch.float8_e4m3fn: _lib.HS_E4M3}


def _code(t: torch.dtype, pool: bool = False) -> int:
    code = (_POOL_DTYPES if pool else _DTYPES).get(t)
    if code is None:
        raise TypeError(f"unsupported dtype {t}")
    return code


def _device(*ts: Optional[torch.Tensor]) -> int:
    """The index of the one CUDA device that all the tensors are on."""
    dev = -2
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("hysparse runs on CUDA tensors only (no CPU path)")
                if dev >= 0:
                    raise ValueError("all tensors must be on the same device")
                dev = i
    return dev


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(t: torch.Tensor, what: str) -> Tuple[int, int, int, int]:
    """(T, H, d, row stride) of a packed [T, H, d] tensor."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [T, H, d]")
    T, H, d = t.shape
    ld, sh, sd = t.stride()
    if T > 0 and ((d > 1 and sd != 1) or (H > 1 and sh != d)):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    return T, H, d, (ld if T > 1 else H * d)


def _dense(t: Optional[torch.Tensor], what: str, dtype=None, shape=None) -> None:
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _call(dev: int, fn, what: str, *args) -> None:
    """The library call on the tensors' device and that device's current stream."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    else:
        st = fn(*args, _raw_stream(dev))
    if st != _lib.HS_OK:
        _lib.check(st, what)


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 0, slow: float = 1.0, fast: float = 32.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """Angles per position of the rot_dim / 2 rotated pairs, base ** (-2 i / rot_dim),
    as a float64 tensor, and the amplitude to pass as rope's ``factor``.

    scaling, for contexts ``factor`` times longer than trained:

    * None       -- as they are.
    * "linear"   -- every angle divided by factor (positions interpolated).
    * "base"     -- the base raised by factor ** (rot_dim / (rot_dim - 2)): the
      slowest pair is slowed by factor, the fastest not at all.
    * "parts"    -- by the turns a pair makes over original_len positions: pairs
      with at least ``fast`` turns stay, pairs with at most ``slow`` are divided
      by factor, those between are mixed linearly in the pair's index; the
      amplitude is 0.1 ln(factor) + 1.
    * "bands"    -- as "parts", but mixed linearly in the number of turns and
      with amplitude 1.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 0 or not factor >= 1.0:
        raise ValueError("base must be positive and factor at least 1")
    half = rot_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    amp = 1.0
    if scaling == "base":
        if rot_dim == 2:
            raise ValueError('"base" needs rot_dim above 2')
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** (-2.0 * i / rot_dim)
    if scaling in ("parts", "bands"):
        if original_len < 1 or not 0 < slow < fast:
            raise ValueError("original_len and 0 < slow < fast are needed")
        turns = original_len * freq / (2 * math.pi)
        if scaling == "bands":
            keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        else:
            if not base > 1:
                raise ValueError('"parts" needs a base above 1')

            def index_of(t):
                return rot_dim * math.log(original_len / (t * 2 * math.pi)) / (2 * math.log(base))

            lo, hi = max(math.floor(index_of(fast)), 0), min(math.ceil(index_of(slow)), half - 1)
            keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            amp = 0.1 * math.log(factor) + 1.0
        freq = freq * keep + freq / factor * (1.0 - keep)
    elif scaling == "linear":
        freq = freq / factor
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device or "cuda"), amp


def _inv_freq(inv_freq: torch.Tensor, d: int) -> int:
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 vector")
    rot = 2 * inv_freq.numel()
    if not 2 <= rot <= d:
        raise ValueError("inv_freq holds one angle per rotated pair: 1 to d / 2 of them")
    return rot


def rope(q: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, k: Optional[torch.Tensor] = None,
         interleaved: bool = False, inverse: bool = False, factor: float = 1.0,
         out: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Rotary positions of q [T, Hq, d] and, when given, k [T, Hkv, d]
    (hysparse_rope): the first 2 * len(inv_freq) elements of each head turned
    by positions[t] * inv_freq, the rest copied.

    inverse: turn back (the gradient with respect to q and k is this call on
    the gradients).  out / out_k may be q / k themselves.  Returns out, or
    (out, out_k) with k."""
    dev = _device(q, positions, inv_freq, k, out, out_k)
    T, Hq, d, ld_q = _rows(q, "q")
    rot = _inv_freq(inv_freq, d)
    if positions.dtype != torch.int32 or positions.shape != (T,) or not positions.is_contiguous():
        raise TypeError("positions must be a contiguous int32 vector, one per row")
    if out is None:
        out, ld_o = _like(q), Hq * d
    else:
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must be like q")
        ld_o = _rows(out, "out")[3]
    Hkv, ld_k, ld_ok = 0, 0, 0
    if k is not None:
        Tk, Hkv, dk, ld_k = _rows(k, "k")
        if Tk != T or dk != d or k.dtype != q.dtype:
            raise ValueError("q and k disagree on rows, head dim or dtype")
        if out_k is None:
            out_k, ld_ok = _like(k), Hkv * d
        else:
            if out_k.shape != k.shape or out_k.dtype != k.dtype:
                raise ValueError("out_k must be like k")
            ld_ok = _rows(out_k, "out_k")[3]
    elif out_k is not None:
        raise ValueError("out_k without k")
    flags = (_lib.HS_ROPE_INTERLEAVED if interleaved else 0) | (_lib.HS_ROPE_INVERSE if inverse else 0)
    _call(dev, _lib.lib().hysparse_rope, "hysparse_rope", T, Hq, Hkv, d, _code(q.dtype), _p(q), ld_q, _p(k), ld_k,
          _p(positions), _p(inv_freq), rot, flags, float(factor), _p(out), ld_o, _p(out_k), ld_ok)
    return out if k is None else (out, out_k)


def _paged(k_pages: torch.Tensor, v_pages: torch.Tensor, cu_rows: torch.Tensor, kv_len: Optional[torch.Tensor],
           block_table: torch.Tensor, k_scale: Optional[torch.Tensor],
           v_scale: Optional[torch.Tensor]) -> Tuple[HsPagedCache, int, int]:
    """The checked hs_paged_cache of these tensors, Hkv and d."""
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages, v_pages: [num_pages, page_size, Hkv, d], alike")
    if not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("page pools must be contiguous")
    num_pages, page, Hkv, d = k_pages.shape
    code = _code(k_pages.dtype, pool=True)
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or not block_table.is_contiguous():
        raise TypeError("block_table must be a contiguous int32 [B, max_pages]")
    B, max_pages = block_table.shape
    _dense(cu_rows, "cu_seqlens", torch.int32, (B + 1,))
    _dense(kv_len, "kv_len", torch.int32, (B,))
    if code == _lib.HS_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("8-bit pages need k_scale and v_scale")
        _dense(k_scale, "k_scale", torch.uint8, (num_pages, Hkv, page))
        _dense(v_scale, "v_scale", torch.uint8, (num_pages, Hkv, page))
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to 8-bit pages")
    return HsPagedCache(_p(cu_rows), _p(kv_len), _p(block_table), B, page, max_pages, num_pages, code, _p(k_pages),
                        _p(v_pages), _p(k_scale), _p(v_scale)), Hkv, d


def _status_ws(ws: Optional[torch.Tensor]) -> None:
    if ws is not None and (not ws.is_contiguous() or ws.numel() * ws.element_size() < 256):
        raise ValueError("ws must be contiguous and hold at least 256 bytes")


def cache_write(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                cu_seqlens: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, *,
                k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, factor: float = 1.0,
                ws: Optional[torch.Tensor] = None) -> None:
    """Write the new rows k, v [T, Hkv, d] of a ragged batch into its pages
    (hysparse_cache_write): sequence b's rows cu_seqlens[b] .. cu_seqlens[b+1]-1
    become its cache's last positions, up to kv_len[b] - 1.

    Pools: bfloat16 or float32, or float8_e4m3fn with uint8 scale bytes
    [num_pages, Hkv, page_size] (an element stands for
    code * 2 ** (byte - 127)).  inv_freq: the keys are turned by rotary
    positions on the way (as rope at their cache positions, without a rounding
    in between).  ws: only its status word is used."""
    dev = _device(k, v, k_pages, v_pages, cu_seqlens, kv_len, block_table, k_scale, v_scale, inv_freq, ws)
    T, H, d, ld_k = _rows(k, "k")
    Tv, Hv, dv, ld_v = _rows(v, "v")
    c, Hkv, dp = _paged(k_pages, v_pages, cu_seqlens, kv_len, block_table, k_scale, v_scale)
    if (Tv, Hv, dv) != (T, H, d) or (H, d) != (Hkv, dp) or k.dtype != v.dtype:
        raise ValueError("k, v and the pages disagree on rows, heads, head dim or dtype")
    rot = _inv_freq(inv_freq, d) if inv_freq is not None else 0
    _status_ws(ws)
    _call(dev, _lib.lib().hysparse_cache_write, "hysparse_cache_write", ctypes.byref(c), T, Hkv, d, _code(k.dtype),
          _p(k), ld_k, _p(v), ld_v, _p(inv_freq), rot, _lib.HS_ROPE_INTERLEAVED if interleaved else 0, float(factor),
          _p(ws))


def cache_read(k_pages: torch.Tensor, v_pages: torch.Tensor, cu_rows: torch.Tensor, block_table: torch.Tensor, *,
               total: int, start: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
               v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
               out_k: Optional[torch.Tensor] = None, out_v: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read rows back out of the pages (hysparse_cache_read): packed row
    cu_rows[b] + i of the results [total, Hkv, d] is position start[b] + i
    (start: int32 [B], 0 when left out) of sequence b, widened to dtype."""
    dev = _device(k_pages, v_pages, cu_rows, block_table, start, k_scale, v_scale, out_k, out_v, ws)
    c, Hkv, d = _paged(k_pages, v_pages, cu_rows, None, block_table, k_scale, v_scale)
    _dense(start, "start", torch.int32, (c.B,))
    shape = (int(total), Hkv, d)
    if out_k is None:
        out_k = k_pages.new_empty(shape, dtype=dtype)
    if out_v is None:
        out_v = k_pages.new_empty(shape, dtype=dtype)
    _dense(out_k, "out_k", dtype, shape)
    _dense(out_v, "out_v", dtype, shape)
    _status_ws(ws)
    _call(dev, _lib.lib().hysparse_cache_read, "hysparse_cache_read", ctypes.byref(c), _p(start), shape[0], Hkv, d,
          _code(dtype), _p(out_k), _p(out_v), _p(ws))
    return out_k, out_v


def ragged_workspace_size(B: int, T: int, Hq: int, Hkv: int, d: int = 128, max_q: int = 0, max_len: int = 0) -> int:
    """Bytes of workspace of packed_attn (max_q = max_len = the longest prompt) and
    chunk_attn_paged (most new rows of a sequence; the longest cache)."""
    n = _lib.lib().hysparse_ragged_workspace_size(B, T, Hq, Hkv, d, max_q, max_len)
    if n == 0:
        raise _lib.HysparseError(_lib.HS_ERR_INVALID_ARG, "hysparse_ragged_workspace_size")
    return int(n)


def _attn_buffers(q: torch.Tensor, Hkv: int, B: int, max_q: int, max_len: int, out, lse, ws):
    T, Hq, d, ld = _rows(q, "q")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16")
    if out is None:
        out = _like(q)
    else:
        _dense(out, "out", q.dtype, (T, Hq, d))
    if lse is None:
        lse = q.new_empty((Hq, T), dtype=torch.float32)
    else:
        _dense(lse, "lse", torch.float32, (Hq, T))
    if ws is None:   # scratch for this call only: its status word is not read
        ws = q.new_empty(ragged_workspace_size(B, T, Hq, Hkv, d, max_q, max_len), dtype=torch.uint8)
    elif not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return T, Hq, d, ld, out, lse, ws


def packed_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                max_len: Optional[int] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Causal attention over whole packed prompts (hysparse_packed_attn).

    q [T, Hq, 128], k and v [T, Hkv, 128] bfloat16, cu_seqlens int32 [B + 1]
    on the device; max_len: the longest prompt (default T).  Returns
    (out [T, Hq, 128], lse [Hq, T] f32, natural log)."""
    dev = _device(q, k, v, cu_seqlens, out, lse, ws)
    Tk, Hkv, dk, ld_k = _rows(k, "k")
    Tv, Hv, dv, ld_v = _rows(v, "v")
    if (Tv, Hv, dv) != (Tk, Hkv, dk) or (Tk, dk) != (q.shape[0], q.shape[-1]):
        raise ValueError("q, k and v disagree on rows, heads or head dim")
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("k and v must be bfloat16")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold B + 1 entries")
    B = cu_seqlens.numel() - 1
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    longest = Tk if max_len is None else int(max_len)
    T, Hq, d, ld_q, out, lse, ws = _attn_buffers(q, Hkv, B, longest, longest, out, lse, ws)
    _call(dev, _lib.lib().hysparse_packed_attn, "hysparse_packed_attn", _p(cu_seqlens), B, T, Hq, Hkv, d, longest,
          float(scale or 0.0), _p(q), ld_q, _p(k), ld_k, _p(v), ld_v, _p(out), _p(lse), _p(ws),
          ws.numel() * ws.element_size())
    return out, lse


def chunk_attn_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, cu_seqlens: torch.Tensor,
                     kv_len: torch.Tensor, block_table: torch.Tensor, *, max_q: Optional[int] = None,
                     max_len: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None):
    """Attention of new tokens over a paged cache that holds them already
    (hysparse_chunk_attn_paged).

    q [T, Hq, 128] bfloat16; pages, scales, kv_len and block_table as
    cache_write takes them (bfloat16 or float8_e4m3fn pools).  max_q: most new
    rows of a sequence (default T; 1 for a decode step); max_len: the longest
    cache (default max_pages * page_size; it only plans the work).  Returns
    (out [T, Hq, 128], lse [Hq, T] f32, natural log)."""
    dev = _device(q, k_pages, v_pages, cu_seqlens, kv_len, block_table, k_scale, v_scale, out, lse, ws)
    c, Hkv, dp = _paged(k_pages, v_pages, cu_seqlens, kv_len, block_table, k_scale, v_scale)
    if dp != q.shape[-1]:
        raise ValueError("q and the pages disagree on head dim")
    most = q.shape[0] if max_q is None else int(max_q)
    longest = c.max_pages * c.page_size if max_len is None else int(max_len)
    T, Hq, d, ld_q, out, lse, ws = _attn_buffers(q, Hkv, c.B, most, longest, out, lse, ws)
    _call(dev, _lib.lib().hysparse_chunk_attn_paged, "hysparse_chunk_attn_paged", ctypes.byref(c), T, Hq, Hkv, d, most,
          longest, float(scale or 0.0), _p(q), ld_q, _p(out), _p(lse), _p(ws), ws.numel() * ws.element_size())
    return out, lse
