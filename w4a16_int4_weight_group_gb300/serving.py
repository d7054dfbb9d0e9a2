"""Serving operators next to the W4A16 layer: rotary positions, the quantised paged cache, attention of drafted
tokens over it, and log probabilities. Argument marshalling only: every function checks devices, dtypes and
shapes and calls the C entry point of the same name on the current CUDA stream (see the C header for what each
computes). Exported by the package itself.

A model's step between two W4A16 projections:

    cache = w4a16_kv_cache(num_pages, kv_heads, head_dim, page_size=64, bits=4)      # once
    table = w4a16_rope_table(max_positions, head_dim, base=500000.0)                 # once
    q, k, v = qkv_layer(x).view(T, heads, head_dim).split([q_heads, kv_heads, kv_heads], 1)
    q = w4a16_kv_write(k, v, cache, slots, q=q, positions=positions, table=table)
    y = w4a16_tree_attention(q, cache, page_table, kv_lens, q_start=q_start, tree_mask=mask, max_q=n)
    logprobs, entropy, ids, alternatives = w4a16_token_logprobs(lm_head(h), drafted, top_k=5)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import W4A16Error, _check, _dtype_code, _ptr, _stream, lib, workspace_for

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class Rope(ctypes.Structure):
    """w4a16_rope_t"""
    _fields_ = [("positions", _vp), ("table", _vp), ("table_rows", _i64), ("rot_dim", _i32), ("interleaved", _i32)]


class KVCache(ctypes.Structure):
    """w4a16_kv_cache_t"""
    _fields_ = [("data", _vp), ("num_pages", _i64), ("kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("bits", _i32)]


_pc, _pr = ctypes.POINTER(KVCache), ctypes.POINTER(Rope)
SIGNATURES = [
    ("w4a16_kv_tile_bytes", ctypes.c_size_t, [ctypes.c_int, ctypes.c_int]),
    ("w4a16_rope", ctypes.c_int, [_pr, _vp, _i64, _i64, _vp, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                  _vp]),
    ("w4a16_kv_write", ctypes.c_int, [_pc, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _pr, _vp, _i64, _i64, ctypes.c_int,
                                      _vp, ctypes.c_int, _vp]),
    ("w4a16_kv_read", ctypes.c_int, [_pc, _vp, _i64, _vp, _vp, ctypes.c_int, _vp]),
    ("w4a16_tree_attention", ctypes.c_int, [_pc, _vp, _i64, _i64, ctypes.c_int, _i64, _vp, _i64, ctypes.c_int, _vp, _vp,
                                            _i64, _vp, _f32, _vp, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]),
    ("w4a16_tree_attention_workspace_size", ctypes.c_size_t, [ctypes.c_int] * 4),
    ("w4a16_token_logprobs", ctypes.c_int, [_vp, _i64, _i64, _i64, ctypes.c_int, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp,
                                            _vp, _vp, _vp]),
]


def w4a16_rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                     factor: float = 1.0, original_max_positions: Optional[int] = None, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, inv_freq: Optional[torch.Tensor] = None,
                     attention_factor: Optional[float] = None, device="cuda") -> torch.Tensor:
    """float32 [max_positions, rot_dim]: cosines, then sines, of every position's angles (made once, in 64 bits).

    scaling: None; "linear" (positions divided by factor); "ntk" (the base raised so that the lowest frequency is
    divided by factor); "yarn" (by parts: frequencies that turn more than beta_fast times within
    original_max_positions stay, those under beta_slow are divided by factor, a ramp in between; the table is
    multiplied by attention_factor, 0.1 ln(factor) + 1 unless given). inv_freq: the rot_dim / 2 frequencies
    themselves, for any other rule.
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if max_positions < 1:
        raise ValueError("max_positions must be positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    mult = 1.0
    if inv_freq is not None:
        if inv_freq.numel() != rot_dim // 2:
            raise ValueError(f"inv_freq must hold rot_dim / 2 = {rot_dim // 2} frequencies")
        f = inv_freq.detach().double().cpu().flatten()
    else:
        if scaling == "ntk" and rot_dim > 2:
            base = base * factor ** (rot_dim / (rot_dim - 2))
        f = base ** (-i / rot_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            if not original_max_positions:
                raise ValueError("yarn needs original_max_positions")
            at = lambda turns: rot_dim * math.log(original_max_positions / (turns * 2 * math.pi)) / (2 * math.log(base))
            low, high = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
            ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
            f = f / factor * ramp + f * (1 - ramp)
            mult = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    if attention_factor is not None:
        mult = attention_factor
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f.to(device)
    return (torch.cat([angle.cos(), angle.sin()], 1) * mult).float().contiguous()


def w4a16_kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, bits: int = 4,
                   device="cuda") -> torch.Tensor:
    """A zeroed cache tensor: uint8 [num_pages, kv_heads, page_size / 16, tile bytes] (layout: the C header)."""
    tile = int(lib().w4a16_kv_tile_bytes(head_dim, bits))
    if not tile:
        raise W4A16Error(2, f"head_dim {head_dim} / bits {bits} not supported; supported: [64, 128, 256] / [4, 8]")
    if page_size <= 0 or page_size % 16:
        raise ValueError("page_size must be a positive multiple of 16")
    return torch.zeros(num_pages, kv_heads, page_size // 16, tile, dtype=torch.uint8, device=device)


def _cache(cache: torch.Tensor, head_dim: int) -> KVCache:
    """The C view of a cache tensor; its bits follow from the tile's bytes."""
    if cache.dtype != torch.uint8 or cache.dim() != 4 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 tensor [pages, kv_heads, page_size / 16, tile bytes]")
    pages, heads, tiles, tile = cache.shape
    for bits in (4, 8):
        if tile == 4 * head_dim * bits + 128:
            return KVCache(cache.data_ptr(), pages, heads, head_dim, tiles * 16, bits)
    raise ValueError(f"cache tiles of {tile} bytes hold neither 4- nor 8-bit heads of {head_dim} elements")


def _heads(t: torch.Tensor, name: str, dtype=None):
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype} (got {t.dtype})")
    return t


def _index(t: torch.Tensor, name: str, dtype, shape, dev):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {dev}")
    return t


def _rope(positions, table, interleaved, tokens, dev) -> Rope:
    _index(positions, "positions", torch.int64, (tokens,), dev)
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous() or table.device != dev:
        raise ValueError(f"table must be a contiguous float32 tensor [positions, rot_dim] on {dev}")
    return Rope(positions.data_ptr(), table.data_ptr(), table.shape[0], table.shape[1], int(bool(interleaved)))


def w4a16_rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [tokens, heads, head_dim] with its heads turned to `positions` (int64 [tokens]); `out` may be x itself."""
    _heads(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _heads(out, "out", x.dtype)
    if out.shape != x.shape or out.device != x.device:
        raise ValueError("out must have the shape and device of x")
    code = _dtype_code(x.dtype)
    if not x.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    T, H, D = x.shape
    r = _rope(positions, table, interleaved, T, x.device)
    _check(lib().w4a16_rope(ctypes.byref(r), x.data_ptr(), x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
                            out.stride(1), T, H, D, code, _stream(x.device)))
    return out


def w4a16_kv_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                   q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   table: Optional[torch.Tensor] = None, interleaved: bool = False,
                   q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Quantise k and v [tokens, kv_heads, head_dim] into the cache's `slots` (int64 [tokens]). With positions and
    table, k turns first, and q [tokens, q_heads, head_dim], when given, is turned into the returned q_out."""
    _heads(k, "k")
    _heads(v, "v", k.dtype)
    dev = k.device
    if not k.is_cuda or v.device != dev or cache.device != dev:
        raise ValueError("all tensors must be CUDA tensors on the same device")
    T, Hk, D = k.shape
    if v.shape != k.shape or cache.shape[1] != Hk:
        raise ValueError(f"k, v and the cache must agree: k {list(k.shape)}, v {list(v.shape)}, cache heads {cache.shape[1]}")
    code = _dtype_code(k.dtype)
    c = _cache(cache, D)
    _index(slots, "slots", torch.int64, (T,), dev)
    r = None
    if (positions is None) != (table is None):
        raise ValueError("positions and table go together")
    if positions is not None:
        r = _rope(positions, table, interleaved, T, dev)
    qp = (None, 0, 0, 0, None)
    if q is not None:
        if r is None:
            raise ValueError("q is only taken with positions and table (it is turned, not cached)")
        _heads(q, "q", k.dtype)
        if q.shape[0] != T or q.shape[2] != D or q.device != dev:
            raise ValueError("q must be [tokens, q_heads, head_dim] on the device of k")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != dev or not q_out.is_contiguous():
            raise ValueError("q_out must be a contiguous tensor like q")
        qp = (q.data_ptr(), q.stride(0), q.stride(1), q.shape[1], q_out.data_ptr())
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(lib().w4a16_kv_write(ctypes.byref(c), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                                v.stride(1), slots.data_ptr(), T, None if r is None else ctypes.byref(r), *qp, code,
                                _stream(dev)))
    return q_out


def w4a16_kv_read(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype,
                  k_out: Optional[torch.Tensor] = None,
                  v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values [tokens, kv_heads, head_dim] of the given slots, dequantised to dtype (the one written)."""
    dev = cache.device
    if not cache.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    c = _cache(cache, head_dim)
    code = _dtype_code(dtype)
    if slots.dim() != 1:
        raise ValueError("slots must be a 1-D int64 tensor")
    T = slots.shape[0]
    _index(slots, "slots", torch.int64, (T,), dev)
    shape = (T, cache.shape[1], head_dim)
    k_out = torch.empty(shape, dtype=dtype, device=dev) if k_out is None else _index(k_out, "k_out", dtype, shape, dev)
    v_out = torch.empty(shape, dtype=dtype, device=dev) if v_out is None else _index(v_out, "v_out", dtype, shape, dev)
    _check(lib().w4a16_kv_read(ctypes.byref(c), slots.data_ptr(), T, k_out.data_ptr(), v_out.data_ptr(), code, _stream(dev)))
    return k_out, v_out


_attention_ws: dict = {}  # workspace bytes per (device, max_q, q_heads, kv_heads, head_dim)


def w4a16_tree_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                         q_start: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                         softmax_scale: Optional[float] = None, max_q: Optional[int] = None,
                         out: Optional[torch.Tensor] = None, return_lse: bool = False):
    """softmax(scale q k^T) v of each sequence's query tokens over its cached tokens, the query tokens among them.

    q [total_q, q_heads, head_dim]; page_table int32 [batch, max_pages]; kv_lens int32 [batch]; q_start int32
    [batch + 1] (None: one query token for each sequence); tree_mask int64 [total_q] (bit j: sees query token j of
    its own sequence; None: a chain); softmax_scale: head_dim ** -0.5 unless given; max_q: the most query tokens of
    a sequence, at most 64 (unless given: min(total_q, 64), 1 without q_start). Returns out, or (out, lse) with lse
    float32 [total_q, q_heads]. A query that sees nothing gives zeros and -inf.
    """
    _heads(q, "q")
    dev = q.device
    if not q.is_cuda or cache.device != dev:
        raise ValueError("all tensors must be CUDA tensors on the same device")
    total, Hq, D = q.shape
    code = _dtype_code(q.dtype)
    c = _cache(cache, D)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    B, cols = page_table.shape
    _index(page_table, "page_table", torch.int32, (B, cols), dev)
    _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    if q_start is not None:
        _index(q_start, "q_start", torch.int32, (B + 1,), dev)
    if tree_mask is not None:
        _index(tree_mask, "tree_mask", torch.int64, (total,), dev)
    if max_q is None:
        max_q = 1 if q_start is None else max(1, min(total, 64))
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty((total, Hq, D), dtype=q.dtype, device=dev)
    else:
        _index(out, "out", q.dtype, (total, Hq, D), dev)
    lse = torch.empty((total, Hq), dtype=torch.float32, device=dev) if return_lse else None
    key = (dev.index, max_q, Hq, c.kv_heads, D)
    need = _attention_ws.get(key)
    if need is None:
        need = _attention_ws[key] = int(lib().w4a16_tree_attention_workspace_size(max_q, Hq, c.kv_heads, D))
    stream = _stream(dev)
    ws = workspace_for(dev, stream.value or 0, need) if need else None
    _check(lib().w4a16_tree_attention(ctypes.byref(c), q.data_ptr(), q.stride(0), q.stride(1), Hq, total, _ptr(q_start), B,
                                      max_q, kv_lens.data_ptr(), page_table.data_ptr(), cols, _ptr(tree_mask),
                                      softmax_scale, out.data_ptr(), _ptr(lse), code, _ptr(ws),
                                      0 if ws is None else ws.numel(), stream))
    return (out, lse) if return_lse else out


def w4a16_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top_k: int = 0):
    """(logprobs, entropy, top_ids, top_logprobs) of rows of logits [rows, vocab] (float16, bfloat16 or float32).

    tokens: int64 [rows] or [rows, n]; logprobs float32 of its shape; entropy float32 [rows]; top_ids int64 and
    top_logprobs float32 [rows, top_k] (top_k <= 32), descending, equal logits by ascending index. Natural logs."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [rows, vocab] with contiguous rows")
    if not logits.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    dev = logits.device
    rows, vocab = logits.shape
    code = 2 if logits.dtype == torch.float32 else _dtype_code(logits.dtype)
    if tokens is None:
        tokens = torch.empty((rows, 0), dtype=torch.int64, device=dev)
    if tokens.dim() not in (1, 2):
        raise ValueError("tokens must be [rows] or [rows, n]")
    _index(tokens, "tokens", torch.int64, (rows,) + tuple(tokens.shape[1:]), dev)
    n = 1 if tokens.dim() == 1 else tokens.shape[1]
    lp = torch.empty(tokens.shape, dtype=torch.float32, device=dev)
    entropy = torch.empty(rows, dtype=torch.float32, device=dev)
    ids = torch.empty((rows, top_k), dtype=torch.int64, device=dev)
    top = torch.empty((rows, top_k), dtype=torch.float32, device=dev)
    stride = logits.stride(0) if rows > 1 else vocab
    _check(lib().w4a16_token_logprobs(logits.data_ptr(), stride, rows, vocab, code, tokens.data_ptr(), n, top_k, lp.data_ptr(),
                                      entropy.data_ptr(), ids.data_ptr(), top.data_ptr(), _stream(dev)))
    return lp, entropy, ids, top


__all__ = ["w4a16_rope_table", "w4a16_rope", "w4a16_kv_cache", "w4a16_kv_write", "w4a16_kv_read", "w4a16_tree_attention",
           "w4a16_token_logprobs"]
