"""Calls over ragged batches and paged caches: rotary positions, the write of
new keys and values into the pages (plain or as 8-bit floats), reading them
back, and attention of packed prompts and of new tokens over the pages.

As the rest of the package these only check and marshal torch tensors; the
work is the library's (include/hysparse.h, "Ragged batches and paged caches").
Packed tensors are [T, H, d], the rows of all sequences one after the other;
they may be slices of one projection's output (any stride between rows that
is a multiple of 16 bytes).

Nothing here is recorded for autograd: results carry no gradient, also where
inputs require one (rope's is rope with ``inverse`` on the results' gradients).
Tensors that a call writes into (out, pages, scales ...) count as changed, so a
backward pass that saved one of them raises.
"""
from __future__ import annotations

import ctypes
import importlib
import math
from typing import Optional, Tuple

import torch

from . import _lib

__all__ = ["rope", "rope_frequencies", "cache_write", "cache_read", "packed_attn", "chunk_attn_paged",
           "ragged_workspace_size"]

_native = None


def _binding():
    """The native half (csrc/binding.cpp): checks and marshals as the rest of
    the package does in Python, in less time; raises if not built."""
    global _native
    if _native is None:
        L = _lib.lib()
        try:
            m = importlib.import_module("._binding", __package__)
        except ImportError as e:
            raise RuntimeError("the native binding is missing or was built for another torch: build it with "
                               "`python -m hybrid_sparse_attention_tcgen05_b200.build --force`") from e
        if m.TORCH_VERSION != torch.__version__.split("+")[0]:
            raise RuntimeError(f"the native binding was built for torch {m.TORCH_VERSION}: build it with "
                               "`python -m hybrid_sparse_attention_tcgen05_b200.build --force`")
        m.bind(_lib.check, *(ctypes.cast(getattr(L, "hysparse_" + n), ctypes.c_void_p).value for n in (
            "rope", "cache_write", "cache_read", "ragged_workspace_size", "packed_attn", "chunk_attn_paged")))
        _native = m
    return _native


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
      by factor, those between are mixed linearly in the pair's index (the two
      ends rounded outwards to whole indices, within 0 and rot_dim - 1); the
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

            # hi may lie beyond the last pair, which then makes more than `slow` turns
            lo, hi = max(math.floor(index_of(fast)), 0), min(math.ceil(index_of(slow)), rot_dim - 1)
            keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            amp = 0.1 * math.log(factor) + 1.0
        freq = freq * keep + freq / factor * (1.0 - keep)
    elif scaling == "linear":
        freq = freq / factor
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device or "cuda"), amp


def rope(q: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, k: Optional[torch.Tensor] = None,
         interleaved: bool = False, inverse: bool = False, factor: float = 1.0,
         out: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Rotary positions of q [T, Hq, d] and, when given, k [T, Hkv, d]
    (hysparse_rope): the first 2 * len(inv_freq) elements of each head turned
    by positions[t] * inv_freq, the rest copied.

    inverse: turn back (the gradient with respect to q and k is this call on
    the gradients).  out / out_k may be q / k themselves.  Returns out, or
    (out, out_k) with k."""
    return (_native or _binding()).rope(q, positions, inv_freq, k, interleaved, inverse, factor, out, out_k)



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
    (_native or _binding()).cache_write(k, v, k_pages, v_pages, cu_seqlens, kv_len, block_table, k_scale, v_scale,
                                        inv_freq, interleaved, factor, ws)



def cache_read(k_pages: torch.Tensor, v_pages: torch.Tensor, cu_rows: torch.Tensor, block_table: torch.Tensor, *,
               total: int, start: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
               v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
               out_k: Optional[torch.Tensor] = None, out_v: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read rows back out of the pages (hysparse_cache_read): packed row
    cu_rows[b] + i of the results [total, Hkv, d] is position start[b] + i
    (start: int32 [B], 0 when left out) of sequence b, widened to dtype."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"unsupported dtype {dtype}")
    return (_native or _binding()).cache_read(k_pages, v_pages, cu_rows, block_table, total, start, k_scale, v_scale,
                                              dtype is torch.bfloat16, out_k, out_v, ws)



def ragged_workspace_size(B: int, T: int, Hq: int, Hkv: int, d: int = 128, max_q: int = 0, max_len: int = 0) -> int:
    """Bytes of workspace of packed_attn (max_q = max_len = the longest prompt) and
    chunk_attn_paged (most new rows of a sequence; the longest cache; 0: any).
    Fewer rows can need more than many, so a loop over batches of different
    sizes keeps one workspace of the most there is, 94 << 20."""
    n = _lib.lib().hysparse_ragged_workspace_size(B, T, Hq, Hkv, d, max_q, max_len)
    if n == 0:
        raise _lib.HysparseError(_lib.HS_ERR_INVALID_ARG, "hysparse_ragged_workspace_size")
    return int(n)


def packed_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                max_len: Optional[int] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Causal attention over whole packed prompts (hysparse_packed_attn).

    q [T, Hq, 128], k and v [T, Hkv, 128] bfloat16, cu_seqlens int32 [B + 1]
    on the device; max_len: the longest prompt (default T).  Returns
    (out [T, Hq, 128], lse [Hq, T] f32, natural log)."""
    return (_native or _binding()).packed_attn(q, k, v, cu_seqlens, max_len, scale or 0.0, out, lse, ws)



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
    return (_native or _binding()).chunk_attn_paged(q, k_pages, v_pages, cu_seqlens, kv_len, block_table, max_q,
                                                    max_len, k_scale, v_scale, scale or 0.0, out, lse, ws)
