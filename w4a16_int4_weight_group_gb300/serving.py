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

For compiled models the module `ops` has them as torch.library ops.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import W4A16Error, _check, _dtype_code, _raw_stream, lib, workspace_for

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
    ("w4a16_tree_attention_fill", ctypes.c_int, [_pc, _vp, _i64, _i64, ctypes.c_int, _i64, _vp, _i64, ctypes.c_int, _vp, _vp,
                                                 _i64, _vp, _f32, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_size_t, _vp]),
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


_calls = None  # the C entry points with flat arguments (see csrc/pycall.c)


def _bind():
    """The marshalling module's calls when it was built (less host time a call than ctypes), else the same
    calls through ctypes."""
    global _calls
    L = lib()
    try:
        from . import _w4a16_call as m
    except ImportError:
        m = None
    if m is not None and hasattr(m, "bind_serving"):
        m.bind_serving(*(ctypes.cast(getattr(L, "w4a16_" + n), _vp).value
                         for n in ("rope", "kv_write", "kv_read", "tree_attention_fill", "token_logprobs")))
        _calls = m
    else:
        _calls = _Ctypes()
    return _calls


def _ints(args, at):
    """The arguments with those that are C ints (their places in `at`) brought into an int's range: past it the nearest end,
    which the library's checks refuse (ctypes would cut them to 32 bits)."""
    return [max(-2 ** 31, min(2 ** 31 - 1, int(x))) if i in at else x for i, x in enumerate(args)]


class _Ctypes:
    """The flat calls of the marshalling module through ctypes."""

    @staticmethod
    def rope(*a):
        a = _ints(a, (3, 4, 12, 13, 14))
        return lib().w4a16_rope(ctypes.byref(Rope(*a[:5])), *a[5:])

    @staticmethod
    def kv_write(*a):
        a = _ints(a, (2, 3, 4, 5, 17, 18, 22, 24))
        rope = ctypes.byref(Rope(*a[14:19])) if a[14] else None
        return lib().w4a16_kv_write(ctypes.byref(KVCache(*a[:6])), *a[6:14], rope, *a[19:])

    @staticmethod
    def kv_read(*a):
        a = _ints(a, (2, 3, 4, 5, 10))
        return lib().w4a16_kv_read(ctypes.byref(KVCache(*a[:6])), *a[6:])

    @staticmethod
    def tree_attention(*a):
        a = _ints(a, (2, 3, 4, 5, 9, 13, 21, 22))
        return lib().w4a16_tree_attention_fill(ctypes.byref(KVCache(*a[:6])), *a[6:])

    @staticmethod
    def token_logprobs(*a):
        return lib().w4a16_token_logprobs(*_ints(a, (4, 6, 7)))


# The checks below use the cheapest tensor queries and read each once: the smallest calls take a few
# microseconds, of which these are a part. The library launches on the current device and looks its size and control
# words up, so each function runs with its tensors' device as the current one.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_codes = {torch.float16: 0, torch.bfloat16: 1}
_bits = {(4 * d * b + 128, d): b for d in (64, 128, 256) for b in (4, 8)}


def _device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors")
    return t.get_device()


def _code(dtype) -> int:
    c = _codes.get(dtype)
    return _dtype_code(dtype) if c is None else c  # raises


def _current_stream(dev: int) -> int:
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _cache_fields(cache: torch.Tensor, head_dim: int, dev: int):
    """The fields of w4a16_kv_cache_t of a cache tensor; its bits follow from the tile's bytes."""
    if cache.dtype is not torch.uint8 or not cache.is_contiguous() or cache.dim() != 4:
        raise ValueError("cache must be a contiguous uint8 tensor [pages, kv_heads, page_size / 16, tile bytes]")
    if cache.get_device() != dev:
        raise ValueError("all tensors must be CUDA tensors on the same device")
    pages, heads, tiles, tile = cache.shape
    bits = _bits.get((tile, head_dim))
    if bits is None:
        raise ValueError(f"cache tiles of {tile} bytes hold neither 4- nor 8-bit heads of {head_dim} elements")
    return cache.data_ptr(), pages, heads, head_dim, tiles * 16, bits


def _cache(cache: torch.Tensor, head_dim: int) -> KVCache:
    """w4a16_kv_cache_t of a cache tensor, for calls of the C entry points."""
    return KVCache(*_cache_fields(cache, head_dim, cache.get_device()))


def _index(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this dtype, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on device {dev}")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """Address, token stride and head stride of a [tokens, heads, head_dim] tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on device {dev}")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    return t.data_ptr(), ts, hs


def _rope(positions, table, interleaved, tokens: int, dev: int):
    pp = _index(positions, "positions", torch.int64, (tokens,), dev)
    if table.dtype is not torch.float32 or table.dim() != 2 or not table.is_contiguous() or table.get_device() != dev:
        raise ValueError(f"table must be a contiguous float32 tensor [positions, rot_dim] on device {dev}")
    rows, rot = table.shape
    return pp, table.data_ptr(), rows, rot, 1 if interleaved else 0


_no_rope = (0, 0, 0, 0, 0)


def _three(t: torch.Tensor, name: str):
    s = t.shape
    if len(s) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    return s


def w4a16_rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [tokens, heads, head_dim] with its heads turned to `positions` (int64 [tokens]); `out` may be x itself."""
    shape = _three(x, "x")
    dev = _device(x)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_rope(x, positions, table, interleaved, out)
    dtype = x.dtype
    code = _code(dtype)
    T, H, D = shape
    xa = _heads(x, "x", dtype, shape, dev)
    r = _rope(positions, table, interleaved, T, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        oa = (out.data_ptr(), H * D, D)
    else:
        oa = _heads(out, "out", dtype, shape, dev)
    st = (_calls or _bind()).rope(*r, *xa, *oa, T, H, D, code, _current_stream(dev))
    if st:
        _check(st)
    return out


def w4a16_kv_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                   q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   table: Optional[torch.Tensor] = None, interleaved: bool = False,
                   q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Quantise k and v [tokens, kv_heads, head_dim] into the cache's `slots` (int64 [tokens]). With positions and
    table, k turns first, and q [tokens, q_heads, head_dim], when given, is turned into the returned q_out."""
    shape = _three(k, "k")
    dev = _device(k)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_write(k, v, cache, slots, q, positions, table, interleaved, q_out)
    dtype = k.dtype
    code = _code(dtype)
    T, Hk, D = shape
    ka, va = _heads(k, "k", dtype, shape, dev), _heads(v, "v", dtype, shape, dev)
    c = _cache_fields(cache, D, dev)
    if c[2] != Hk:
        raise ValueError(f"k and v have {Hk} heads, the cache {c[2]}")
    sp = _index(slots, "slots", torch.int64, (T,), dev)
    if (positions is None) != (table is None):
        raise ValueError("positions and table go together")
    r = _no_rope if positions is None else _rope(positions, table, interleaved, T, dev)
    qa = (0, 0, 0, 0, 0)
    if q is not None:
        if positions is None:
            raise ValueError("q is only taken with positions and table (it is turned, not cached)")
        qs = _three(q, "q")
        Hq = qs[1]
        qv = _heads(q, "q", dtype, (T, Hq, D), dev)
        if q_out is None:
            q_out = torch.empty(qs, dtype=dtype, device=k.device)
            qo = q_out.data_ptr()
        else:
            qo = _index(q_out, "q_out", dtype, qs, dev)
        qa = (*qv, Hq, qo)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    st = (_calls or _bind()).kv_write(*c, *ka, *va, sp, T, *r, *qa, code, _current_stream(dev))
    if st:
        _check(st)
    return q_out


def w4a16_kv_read(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype,
                  k_out: Optional[torch.Tensor] = None,
                  v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values [tokens, kv_heads, head_dim] of the given slots, dequantised to dtype (the one written)."""
    dev = _device(cache)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_read(cache, slots, head_dim, dtype, k_out, v_out)
    c = _cache_fields(cache, head_dim, dev)
    code = _code(dtype)
    if slots.dim() != 1:
        raise ValueError("slots must be a 1-D int64 tensor")
    T = slots.shape[0]
    sp = _index(slots, "slots", torch.int64, (T,), dev)
    shape = (T, c[2], head_dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=cache.device)
        kp = k_out.data_ptr()
    else:
        kp = _index(k_out, "k_out", dtype, shape, dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=cache.device)
        vp = v_out.data_ptr()
    else:
        vp = _index(v_out, "v_out", dtype, shape, dev)
    st = (_calls or _bind()).kv_read(*c, sp, T, kp, vp, code, _current_stream(dev))
    if st:
        _check(st)
    return k_out, v_out


_attention_ws: dict = {}  # workspace bytes: a pure function of the sizes and the device


def w4a16_tree_attention_workspace_size(max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of the workspace that a call of w4a16_tree_attention with these sizes uses on the current device."""
    return int(lib().w4a16_tree_attention_workspace_size(max_q, q_heads, kv_heads, head_dim))


def w4a16_tree_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                         q_start: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                         softmax_scale: Optional[float] = None, max_q: Optional[int] = None,
                         out: Optional[torch.Tensor] = None, return_lse: bool = False,
                         workspace: Optional[torch.Tensor] = None):
    """softmax(scale q k^T) v of each sequence's query tokens over its cached tokens, the query tokens among them.

    q [total_q, q_heads, head_dim]; page_table int32 [batch, max_pages]; kv_lens int32 [batch]; q_start int32
    [batch + 1], ascending (None: one query token for each sequence); tree_mask int64 [total_q] (bit j: sees query token j of
    its own sequence; None: a chain); softmax_scale: head_dim ** -0.5 unless given; max_q: the most query tokens of
    a sequence, at most 64 (unless given: min(total_q, 64), 1 without q_start). A length in kv_lens that is past the
    page table counts as the table's end: the query tokens are then its last tokens. Returns out, or (out, lse) with lse
    float32 [total_q, q_heads]. A query that sees nothing gives zeros and -inf. Query tokens of a sequence past its first
    max_q, and rows that no sequence owns (before q_start[0], from q_start[batch] on), are not computed: NaN in the tensors that this
    call makes, unchanged in a given `out`.

    workspace: contiguous uint8 [bytes] of the caller's own, its first 4 KiB zero before its first use, for calls of
    one stream (or one graph) at a time; with fewer bytes than w4a16_tree_attention_workspace_size no sequence is split
    over CTAs. Unless given, the binding keeps one for each stream, and one for each capture by torch.cuda.graph.
    """
    shape = _three(q, "q")
    dev = _device(q)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_tree_attention(q, cache, page_table, kv_lens, q_start, tree_mask, softmax_scale, max_q, out,
                                        return_lse, workspace)
    dtype = q.dtype
    code = _code(dtype)
    total, Hq, D = shape
    qa = _heads(q, "q", dtype, shape, dev)
    c = _cache_fields(cache, D, dev)
    pt = page_table.shape
    if len(pt) != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    B, cols = pt
    pp = _index(page_table, "page_table", torch.int32, pt, dev)
    lp = _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    sp = 0 if q_start is None else _index(q_start, "q_start", torch.int32, (B + 1,), dev)
    mp = 0 if tree_mask is None else _index(tree_mask, "tree_mask", torch.int64, (total,), dev)
    if max_q is None:
        max_q = 1 if q_start is None else max(1, min(total, 64))
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    fill = 0  # outputs made here have no row that holds whatever was in the memory before
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
        op = out.data_ptr()
        fill = 1
    else:
        op = _index(out, "out", dtype, shape, dev)
    lse, sep = None, 0
    if return_lse:
        lse = torch.empty((total, Hq), dtype=torch.float32, device=q.device)
        sep = lse.data_ptr()
        fill |= 2
    stream = _current_stream(dev)
    wp = wb = 0
    if workspace is not None:
        wb = workspace.numel()
        wp = _index(workspace, "workspace", torch.uint8, (wb,), dev)
    else:
        key = (dev, max_q, Hq, c[2], D)
        need = _attention_ws.get(key)
        if need is None:
            need = _attention_ws[key] = w4a16_tree_attention_workspace_size(max_q, Hq, c[2], D)
        if need:
            ws = workspace_for(q.device, stream, need)
            wp, wb = ws.data_ptr(), ws.numel()
    st = (_calls or _bind()).tree_attention(*c, *qa, Hq, total, sp, B, max_q, lp, pp, cols, mp, softmax_scale, op, sep, fill,
                                            code, wp, wb, stream)
    if st:
        _check(st)
    return (out, lse) if return_lse else out


def w4a16_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top_k: int = 0):
    """(logprobs, entropy, top_ids, top_logprobs) of rows of logits [rows, vocab] (float16, bfloat16 or float32).

    tokens: int64 [rows] or [rows, n]; logprobs float32 of its shape; entropy float32 [rows]; top_ids int64 and
    top_logprobs float32 [rows, top_k] (top_k <= 32), descending, equal logits by ascending index. Natural logs."""
    s = logits.shape
    if len(s) != 2:
        raise ValueError("logits must be [rows, vocab] with contiguous rows")
    rows, vocab = s
    stride, es = logits.stride()
    if es != 1 and vocab > 1:
        raise ValueError("logits must be [rows, vocab] with contiguous rows")
    dev = _device(logits)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_token_logprobs(logits, tokens, top_k)
    device = logits.device
    code = 2 if logits.dtype is torch.float32 else _code(logits.dtype)
    if tokens is None:
        shape, n, tp = (rows, 0), 0, 0
    else:
        shape = tokens.shape
        if len(shape) not in (1, 2) or shape[0] != rows:
            raise ValueError("tokens must be [rows] or [rows, n]")
        tp = _index(tokens, "tokens", torch.int64, shape, dev)
        n = 1 if len(shape) == 1 else shape[1]
    lp = torch.empty(shape, dtype=torch.float32, device=device)
    entropy = torch.empty(rows, dtype=torch.float32, device=device)
    ids = torch.empty((rows, top_k), dtype=torch.int64, device=device)
    top = torch.empty((rows, top_k), dtype=torch.float32, device=device)
    st = (_calls or _bind()).token_logprobs(logits.data_ptr(), stride if rows > 1 else vocab, rows, vocab, code, tp, n, top_k,
                                            lp.data_ptr(), entropy.data_ptr(), ids.data_ptr(), top.data_ptr(), _current_stream(dev))
    if st:
        _check(st)
    return lp, entropy, ids, top


__all__ = ["w4a16_rope_table", "w4a16_rope", "w4a16_kv_cache", "w4a16_kv_write", "w4a16_kv_read", "w4a16_tree_attention",
           "w4a16_tree_attention_workspace_size", "w4a16_token_logprobs"]
