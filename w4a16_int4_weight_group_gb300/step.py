"""Operators around a verification step of many users: low-rank adapters beside the W4A16 layer, which drafted tokens stand,
and the pages of the quantised cache. Argument marshalling only, as in the module of the serving operators: every function
checks devices, dtypes and shapes and calls the C entry point of the same name on the current CUDA stream (see the C header
for what each computes). Exported by the package itself.

    y = w4a16_lora(x, a, b, ids, layer(x), scales=s)                            # another adapter for each token
    accepted, path, tokens, probs = w4a16_verify_drafts(logits, drafted, uniforms, noise, q_start=q_start, tree_mask=mask)
    kv_lens = w4a16_kv_compact(caches, head_dim, page_table, kv_lens, path, q_start=q_start)

    refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")              # owners of each page, 0: free
    table, lens = w4a16_kv_fork(refs, page_table, kv_lens, parents, page_size)   # samples or beams that share their parents' pages
    held, copies = w4a16_kv_reserve(refs, table, lens, lens + n, page_size)      # room for n more tokens, shared pages replaced
    w4a16_kv_copy(caches, copies)                                                # .. and copied
    w4a16_kv_free(refs, table, lens, page_size)                                  # a sequence ends

A cache is the tensor of one layer, as w4a16_kv_cache makes it, or a contiguous [layers, ...] stack of such tensors
(cache[i] is then layer i's). For compiled models the module `ops` has these as torch.library ops.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _check, lib, workspace_for
from .serving import _bits, _code, _current_device, _current_stream, _device, _index, _ints, KVCache

_i64, _int, _vp, _size = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_pc = ctypes.POINTER(KVCache)
SIGNATURES = [
    ("w4a16_lora", _int, [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, _i64, _int, _vp, _size, _vp]),
    ("w4a16_lora_workspace_size", _size, [_i64, _int, _i64]),
    ("w4a16_verify_drafts", _int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _i64, _int, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _size, _vp]),
    ("w4a16_verify_drafts_workspace_size", _size, [_i64, _i64]),
    ("w4a16_kv_fork", _int, [_vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    ("w4a16_kv_reserve", _int, [_vp, _i64, _int, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp]),
    ("w4a16_kv_free", _int, [_vp, _i64, _int, _vp, _i64, _vp, _vp, _i64, _vp]),
    ("w4a16_kv_copy", _int, [_pc, _i64, _vp, _i64, _vp]),
    ("w4a16_kv_compact", _int, [_pc, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _int, _vp, _vp]),
]

_calls = None  # the C entry points with flat arguments (see csrc/pycall.c)


def _bind():
    """The marshalling module's calls when it was built, else the same calls through ctypes."""
    global _calls
    L = lib()
    try:
        from . import _w4a16_call as m
    except ImportError:
        m = None
    if m is not None and hasattr(m, "bind_step"):
        m.bind_step(*(ctypes.cast(getattr(L, "w4a16_" + n), _vp).value
                      for n in ("lora", "verify_drafts", "kv_fork", "kv_reserve", "kv_free", "kv_copy", "kv_compact")))
        _calls = m
    else:
        _calls = _Ctypes()
    return _calls


_fast = None  # the module of ordinary calls (see csrc/fastcall.cpp), False when it was not built for this torch


def _bind_fast():
    """The calls that check ordinary tensors and make them in one step of C++. Each returns None where there is something to say or
    to provide; the functions below then go their own way."""
    global _fast
    L = lib()
    try:
        from . import _w4a16_fast as m
        from .build import fast_key
        if getattr(m, "built_for", None) != fast_key():  # (another torch's layout of tensors)
            raise ImportError
        m.bind(*(ctypes.cast(getattr(L, "w4a16_" + n), _vp).value
                 for n in ("lora", "verify_drafts", "kv_fork", "kv_reserve", "kv_free", "kv_copy", "kv_compact", "lora_workspace_size")))
        _fast = m
    except ImportError:
        _fast = False
    return _fast


class _Ctypes:
    """The flat calls of the marshalling module through ctypes."""

    @staticmethod
    def lora(*a):
        return lib().w4a16_lora(*_ints(a, (13, 15)))

    @staticmethod
    def verify_drafts(*a):
        return lib().w4a16_verify_drafts(*_ints(a, (4, 8)))

    @staticmethod
    def kv_fork(*a):
        return lib().w4a16_kv_fork(*_ints(a, (2,)))

    @staticmethod
    def kv_reserve(*a):
        return lib().w4a16_kv_reserve(*_ints(a, (2,)))

    @staticmethod
    def kv_free(*a):
        return lib().w4a16_kv_free(*_ints(a, (2,)))

    @staticmethod
    def kv_copy(*a):
        a = _ints(a, (2, 3, 4, 5))
        return lib().w4a16_kv_copy(ctypes.byref(KVCache(*a[:6])), *a[6:])

    @staticmethod
    def kv_compact(*a):
        a = _ints(a, (2, 3, 4, 5, 13))
        return lib().w4a16_kv_compact(ctypes.byref(KVCache(*a[:6])), *a[6:])


def _rows(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """Address and row stride of a 2-D tensor with contiguous rows."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on device {dev}")
    stride, es = t.stride()
    if es != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.data_ptr(), stride


def w4a16_lora_workspace_size(tokens: int, rank: int, adapters: int) -> int:
    """Bytes of the workspace that a call of w4a16_lora with these sizes needs (0: none)."""
    return int(lib().w4a16_lora_workspace_size(tokens, rank, adapters))


_lora_ws: dict = {}  # workspace bytes: a pure function of the sizes
_FEW = 256           # tokens up to which none is needed


def w4a16_lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor, base: torch.Tensor,
               scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = base[t] + scales[i] * (x[t] @ a[i].T) @ b[i].T with i = ids[t]: low-rank adapters beside a shared projection.

    x [tokens, k]; a [adapters, rank, k]; b [adapters, n, rank]; ids int32 [tokens] (outside [0, adapters): no adapter, the row is
    base's); base [tokens, n], what the projection gave; scales float32 [adapters] (None: 1); `out` may be base itself. k and n
    are multiples of 8, rank one up to 128.

    workspace: contiguous uint8 of the caller's own, for calls of one stream (or one graph) at a time; unless given, the binding
    keeps one for each stream, and one for each capture by torch.cuda.graph. Calls of up to 256 tokens need none, nor those of up to 1024 tokens,
    512 adapters and rank 64.
    """
    if workspace is None:
        fast = _bind_fast() if _fast is None else _fast
        if fast:
            y = fast.lora(x, a, b, ids, base, scales, out)
            if y is not None:
                return y
    sx, sa, sb = x.shape, a.shape, b.shape
    if len(sx) != 2 or len(sa) != 3 or len(sb) != 3:
        raise ValueError("x must be [tokens, k], a [adapters, rank, k] and b [adapters, n, rank]")
    dev = _device(x)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_lora(x, a, b, ids, base, scales, out, workspace)
    dtype = x.dtype
    code = _code(dtype)
    T, K = sx
    L, r, _ = sa
    N = sb[1]
    xa = _rows(x, "x", dtype, sx, dev)
    ap = _index(a, "a", dtype, (L, r, K), dev)
    bp = _index(b, "b", dtype, (L, N, r), dev)
    ip = _index(ids, "ids", torch.int32, (T,), dev)
    sp = 0 if scales is None else _index(scales, "scales", torch.float32, (L,), dev)
    ba = _rows(base, "base", dtype, (T, N), dev)
    if out is None:
        out = torch.empty((T, N), dtype=dtype, device=x.device)
        oa = (out.data_ptr(), N)
    else:
        oa = _rows(out, "out", dtype, (T, N), dev)
    stream = _current_stream(dev)
    wp = wb = 0
    if workspace is not None:
        wb = workspace.numel()
        wp = _index(workspace, "workspace", torch.uint8, (wb,), dev)
    elif T > _FEW:
        need = _lora_ws.get((T, r, L))
        if need is None:
            need = _lora_ws[(T, r, L)] = w4a16_lora_workspace_size(T, r, L)
        if need:
            ws = workspace_for(x.device, stream, need)
            wp, wb = ws.data_ptr(), ws.numel()
    st = (_calls or _bind()).lora(*xa, ap, bp, ip, sp, *ba, *oa, T, K, N, r, L, code, wp, wb, stream)
    if st:
        _check(st)
    return out


def w4a16_verify_drafts_workspace_size(total: int, vocab: int) -> int:
    """Bytes of the workspace that a call of w4a16_verify_drafts with these sizes needs on the current device."""
    return int(lib().w4a16_verify_drafts_workspace_size(total, vocab))


_verify_ws: dict = {}  # workspace bytes: a pure function of the sizes and the device


def w4a16_verify_drafts(logits: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor, noise: torch.Tensor,
                        q_start: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                        draft_probs: Optional[torch.Tensor] = None, temperature: Optional[torch.Tensor] = None,
                        max_q: Optional[int] = None,
                        workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(accepted, path, out_tokens, out_probs): which drafted tokens stand, and the token after them, from given random numbers.

    logits [total, vocab] (float16, bfloat16 or float32): row i is the target's after token i; tokens int64 [total]: each sequence's last
    token (the root), then its drafted ones; uniforms float32 [total] in [0, 1); noise float32 [batch, vocab], exponential
    numbers (torch.empty(..).exponential_()); q_start int32 [batch + 1] (None: one token for each sequence, plain sampling); tree_mask
    int64 [total], the attention's (None: chains); draft_probs float32 [total, vocab], chains only: row i is what the token after
    token i was drawn from (None: the tokens are guesses); temperature float32 [batch], 0 for the largest logit (None: 1); max_q: the
    most tokens of a sequence, at most 64 (unless given: min(total, 64), 1 without q_start).

    accepted int32 [batch]; path int32 [batch, max_q], the root and the accepted tokens as indices within the sequence, then -1 (what
    w4a16_kv_compact takes); out_tokens int64 [batch, max_q], the accepted tokens and the one after them, then -1; out_probs float32
    [batch, max_q], the target's probabilities of these, then 0. A row without probabilities (NaN, +infinity, all
    -infinity) gives -1 and NaN. workspace: as for w4a16_lora; every call needs one.
    """
    s, sn = logits.shape, noise.shape
    if len(s) != 2 or len(sn) != 2:
        raise ValueError("logits must be [total, vocab] and noise [batch, vocab]")
    dev = _device(logits)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_verify_drafts(logits, tokens, uniforms, noise, q_start, tree_mask, draft_probs, temperature, max_q, workspace)
    dtype, device = logits.dtype, logits.device
    code = 2 if dtype is torch.float32 else _code(dtype)
    total, V = s
    B = sn[0]
    if max_q is None:
        max_q = 1 if q_start is None else max(1, min(total, 64))
    stream = _current_stream(dev)
    if workspace is not None:
        wb = workspace.numel()
        wp = _index(workspace, "workspace", torch.uint8, (wb,), dev)
    else:
        key = (dev, total, V)
        need = _verify_ws.get(key)
        if need is None:
            need = _verify_ws[key] = w4a16_verify_drafts_workspace_size(total, V)
        ws = workspace_for(device, stream, need)
        wp, wb = ws.data_ptr(), ws.numel()
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.verify_drafts(logits, tokens, uniforms, noise, q_start, tree_mask, draft_probs, temperature, max_q, wp, wb)
        if y is not None:
            return y
    la = _rows(logits, "logits", dtype, s, dev)
    na = _rows(noise, "noise", torch.float32, (B, V), dev)
    tp = _index(tokens, "tokens", torch.int64, (total,), dev)
    up = _index(uniforms, "uniforms", torch.float32, (total,), dev)
    qp = 0 if q_start is None else _index(q_start, "q_start", torch.int32, (B + 1,), dev)
    mp = 0 if tree_mask is None else _index(tree_mask, "tree_mask", torch.int64, (total,), dev)
    da = (0, 0) if draft_probs is None else _rows(draft_probs, "draft_probs", torch.float32, s, dev)
    ep = 0 if temperature is None else _index(temperature, "temperature", torch.float32, (B,), dev)
    m = max(0, min(max_q, 64))  # (a max_q out of range is refused by the call)
    accepted = torch.empty(B, dtype=torch.int32, device=device)
    path = torch.empty((B, m), dtype=torch.int32, device=device)
    out = torch.empty((B, m), dtype=torch.int64, device=device)
    probs = torch.empty((B, m), dtype=torch.float32, device=device)
    st = (_calls or _bind()).verify_drafts(*la, total, V, code, tp, qp, B, max_q, mp, up, *na, *da, ep, accepted.data_ptr(), path.data_ptr(),
                                           out.data_ptr(), probs.data_ptr(), wp, wb, stream)
    if st:
        _check(st)
    return accepted, path, out, probs


def _table(page_table: torch.Tensor, dev: int):
    s = page_table.shape
    if len(s) != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    return _index(page_table, "page_table", torch.int32, s, dev), s[0], s[1]


def _refs(refs: torch.Tensor, dev: int):
    if refs.dim() != 1:
        raise ValueError("refs must be a 1-D int32 tensor")
    n = refs.shape[0]
    return _index(refs, "refs", torch.int32, (n,), dev), n


def w4a16_kv_fork(refs: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, parents: torch.Tensor,
                  page_size: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """(new_table, new_lens): sequences that share the pages of `parents` (int32 [rows], rows of page_table [batch, max_pages]; one out
    of range: an empty sequence). refs (int32 [pages]) counts the new holders."""
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.kv_fork(refs, page_table, kv_lens, parents, page_size)
        if y is not None:
            return y
    dev = _device(refs)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_fork(refs, page_table, kv_lens, parents, page_size)
    rp, pages = _refs(refs, dev)
    pp, B, cols = _table(page_table, dev)
    lp = _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    if parents.dim() != 1:
        raise ValueError("parents must be a 1-D int32 tensor")
    n = parents.shape[0]
    ap = _index(parents, "parents", torch.int32, (n,), dev)
    table = torch.empty((n, cols), dtype=torch.int32, device=refs.device)
    lens = torch.empty(n, dtype=torch.int32, device=refs.device)
    st = (_calls or _bind()).kv_fork(rp, pages, page_size, pp, cols, lp, B, ap, n, table.data_ptr(), lens.data_ptr(), _current_stream(dev))
    if st:
        _check(st)
    return table, lens


def w4a16_kv_reserve(refs: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor,
                     page_size: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """(held, copies): free pages for the tokens up to new_lens (int32 [batch]) go into page_table, and a partly filled last page that others
    hold too is replaced by a page of the sequence's own: copies int32 [batch, 2] says {from, to} (else -1, -1), for
    w4a16_kv_copy. held int32 [batch]: the tokens that there is room for then (new_lens, unless pages ran out)."""
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.kv_reserve(refs, page_table, kv_lens, new_lens, page_size)
        if y is not None:
            return y
    dev = _device(refs)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_reserve(refs, page_table, kv_lens, new_lens, page_size)
    rp, pages = _refs(refs, dev)
    pp, B, cols = _table(page_table, dev)
    lp = _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    np_ = _index(new_lens, "new_lens", torch.int32, (B,), dev)
    held = torch.empty(B, dtype=torch.int32, device=refs.device)
    copies = torch.empty((B, 2), dtype=torch.int32, device=refs.device)
    st = (_calls or _bind()).kv_reserve(rp, pages, page_size, pp, cols, lp, np_, B, held.data_ptr(), copies.data_ptr(), _current_stream(dev))
    if st:
        _check(st)
    return held, copies


def w4a16_kv_free(refs: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, page_size: int,
                  keep: Optional[torch.Tensor] = None) -> None:
    """Gives back the pages of the tokens from keep (int32 [batch]; None: all) on: refs shrink, the table's entries become -1."""
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.kv_free(refs, page_table, kv_lens, page_size, keep)
        if y is not None:
            return
    dev = _device(refs)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_free(refs, page_table, kv_lens, page_size, keep)
    rp, pages = _refs(refs, dev)
    pp, B, cols = _table(page_table, dev)
    lp = _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    kp = 0 if keep is None else _index(keep, "keep", torch.int32, (B,), dev)
    st = (_calls or _bind()).kv_free(rp, pages, page_size, pp, cols, lp, kp, B, _current_stream(dev))
    if st:
        _check(st)


def _layers(cache: torch.Tensor, head_dim: Optional[int], dev: int):
    """The fields of w4a16_kv_cache_t of one layer, and the layers, of a cache tensor or a stack of them. head_dim None: any that fits the
    tile's bytes (a tile of 4-bit heads is as long as one of 8-bit heads of half the size)."""
    s = cache.shape
    if cache.dtype is not torch.uint8 or not cache.is_contiguous() or len(s) not in (4, 5):
        raise ValueError("cache must be a contiguous uint8 tensor [pages, kv_heads, page_size / 16, tile bytes] or [layers, ...] of such")
    if cache.get_device() != dev:
        raise ValueError("all tensors must be CUDA tensors on the same device")
    layers = s[0] if len(s) == 5 else 1
    pages, heads, tiles, tile = s[-4:]
    if head_dim is None:
        head_dim = next((d for d in (64, 128, 256) if (tile, d) in _bits), 0)
    bits = _bits.get((tile, head_dim))
    if bits is None:
        raise ValueError(f"cache tiles of {tile} bytes hold neither 4- nor 8-bit heads of {head_dim or '64, 128 or 256'} elements")
    return cache.data_ptr(), pages, heads, head_dim, tiles * 16, bits, layers


def w4a16_kv_copy(cache: torch.Tensor, copies: torch.Tensor) -> None:
    """Copies whole pages of the cache (all layers of a stack): copies int32 [n, 2], {from, to}; pairs with a page out of range (-1) are
    skipped. No page is written twice, or both read and written."""
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.kv_copy(cache, copies)
        if y is not None:
            return
    dev = _device(cache)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_copy(cache, copies)
    c = _layers(cache, None, dev)
    if copies.dim() != 2:
        raise ValueError("copies must be [n, 2]")
    n = copies.shape[0]
    cp = _index(copies, "copies", torch.int32, (n, 2), dev)
    st = (_calls or _bind()).kv_copy(*c, cp, n, _current_stream(dev))
    if st:
        _check(st)


def w4a16_kv_compact(cache: torch.Tensor, head_dim: int, page_table: torch.Tensor, kv_lens: torch.Tensor, path: torch.Tensor,
                     q_start: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the accepted tokens of each sequence's tree together (all heads and layers) and returns the new kv_lens.

    path int32 [batch, max_q] as w4a16_verify_drafts gives it; q_start int32 [batch + 1]: the sequence's drafted tokens are the last
    q_start[b + 1] - q_start[b] of kv_lens (None: 1). Their pages belong to one sequence each (see w4a16_kv_reserve)."""
    fast = _bind_fast() if _fast is None else _fast
    if fast:
        y = fast.kv_compact(cache, head_dim, page_table, kv_lens, path, q_start)
        if y is not None:
            return y
    dev = _device(cache)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return w4a16_kv_compact(cache, head_dim, page_table, kv_lens, path, q_start)
    c = _layers(cache, head_dim, dev)
    pp, B, cols = _table(page_table, dev)
    lp = _index(kv_lens, "kv_lens", torch.int32, (B,), dev)
    sp = path.shape
    if len(sp) != 2:
        raise ValueError("path must be [batch, max_q]")
    hp = _index(path, "path", torch.int32, (B, sp[1]), dev)
    qp = 0 if q_start is None else _index(q_start, "q_start", torch.int32, (B + 1,), dev)
    lens = torch.empty(B, dtype=torch.int32, device=cache.device)
    st = (_calls or _bind()).kv_compact(*c, pp, cols, lp, qp, B, hp, sp[1], lens.data_ptr(), _current_stream(dev))
    if st:
        _check(st)
    return lens


__all__ = ["w4a16_lora", "w4a16_lora_workspace_size", "w4a16_verify_drafts", "w4a16_verify_drafts_workspace_size", "w4a16_kv_fork",
           "w4a16_kv_reserve", "w4a16_kv_free", "w4a16_kv_copy", "w4a16_kv_compact"]
