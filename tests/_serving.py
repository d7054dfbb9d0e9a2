"""Plain 64-bit implementations of the serving operators, for the tests."""
import math

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# relative error of one conversion to a format of p significant bits, 2^-p: float16 has 11, bfloat16 8
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}        # half of the smallest subnormal number


def rotate(x, positions, table, interleaved):
    """float64 [T, H, D] from float64 x, and the sum of the magnitudes of each result's two terms."""
    y, mag = x.clone(), torch.zeros_like(x)
    R = table.shape[1]
    for t, p in enumerate(positions.tolist()):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            if not 0 <= p < table.shape[0]:
                y[t, :, a] = y[t, :, b] = math.nan
                continue
            c, s = float(table[p, i]), float(table[p, R // 2 + i])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
            mag[t, :, a] = (x[t, :, a] * c).abs() + (x[t, :, b] * s).abs()
            mag[t, :, b] = (x[t, :, a] * s).abs() + (x[t, :, b] * c).abs()
    return y, mag


def rotate32(x, positions, table, interleaved):
    """The same in float32 numpy, each product and sum rounded by itself (the definition's own rounding)."""
    x = x.float().numpy()
    y = x.copy()
    t = table.numpy()[positions.numpy()][:, None]
    R = t.shape[-1]
    c, s = t[..., :R // 2], t[..., R // 2:]
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return torch.from_numpy(y)


def quantise(x, bits, dtype):
    """codes [.., D] uint8, scale (dtype), zero uint8 of rows of x (dtype), step by step in float32 numpy."""
    top = np.float32(2 ** bits - 1)
    inv_top = np.float32(1) / top
    a = x.float().numpy()
    finite = np.isfinite(a).all(-1)
    b = np.where(finite[..., None], a, np.float32(0))
    lo, hi = np.minimum(b.min(-1), 0), np.maximum(b.max(-1), 0)
    s = torch.from_numpy((hi * inv_top - lo * inv_top).astype(np.float32)).to(dtype)
    s32 = s.float().numpy()
    s32 = np.where(s32 < np.float32(2.0 ** -126), np.float32(0), s32)
    with np.errstate(divide="ignore"):
        inv = np.where(s32 > 0, np.float32(1) / s32, np.float32(0)).astype(np.float32)
    z = np.clip(np.rint(-lo * inv), 0, top)
    u = np.clip(np.rint(b * inv[..., None]) + z[..., None], 0, top)
    s = torch.from_numpy(np.where(finite, s32, np.float32(np.nan)).astype(np.float32)).to(dtype)
    return u.astype(np.uint8), s, z.astype(np.uint8)


def values(u, s, z):
    """float64 (code - zero) * scale."""
    return (torch.from_numpy(u.astype(np.float64)) - torch.from_numpy(z.astype(np.float64))[..., None]) * s.double()[..., None]


def put(cache, slots, k, v, bits, dtype):
    """The oracle's own write into a CPU cache tensor, byte by byte."""
    pages, heads, tiles, _ = cache.shape
    D = k.shape[-1]
    per = D * bits // 8
    for j, x in enumerate((k, v)):
        u, s, z = quantise(x, bits, dtype)
        sb = s.view(torch.int16).numpy().view(np.uint16)
        for t, slot in enumerate(slots.tolist()):
            if not 0 <= slot < pages * tiles * 16:
                continue
            page, at = divmod(slot, tiles * 16)
            for h in range(heads):
                row = u[t, h] if bits == 8 else u[t, h, 0::2] | (u[t, h, 1::2] << 4)
                tile = cache[page, h, at // 16].numpy()
                tile[j * 16 * per + at % 16 * per:][:per] = row
                word = 0x7FFF if np.isnan(s[t, h].item()) else int(sb[t, h])
                word |= (0 if np.isnan(s[t, h].item()) else int(z[t, h])) << 16
                tile[32 * per + 64 * j + at % 16 * 4:][:4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)


def get(cache, slots, D, bits, dtype):
    """float64 keys and values [T, heads, D] of slots of a CPU cache tensor."""
    pages, heads, tiles, _ = cache.shape
    per = D * bits // 8
    out = np.zeros((2, len(slots), heads, D))
    raw = cache.numpy()
    for t, slot in enumerate(slots):
        page, at = divmod(int(slot), tiles * 16)
        for h in range(heads):
            tile = raw[page, h, at // 16]
            for j in range(2):
                row = tile[j * 16 * per + at % 16 * per:][:per]
                if bits == 4:
                    both = np.empty(D, np.uint8)
                    both[0::2], both[1::2] = row & 15, row >> 4
                    row = both
                w = int(tile[32 * per + 64 * j + at % 16 * 4:][:4].copy().view(np.uint32)[0])
                s = torch.tensor([w & 0xFFFF], dtype=torch.int32).to(torch.int16).view(dtype).double().item()
                out[j, t, h] = (row.astype(np.float64) - (w >> 16)) * s
    return torch.from_numpy(out[0]), torch.from_numpy(out[1])


def attend(q, cache, page_table, kv_lens, q_start, tree_mask, scale, D, bits, dtype, page):
    """out, lse, and the bound's ingredients: sum p |v| and the largest sum |q| |k| scale of a row (all float64)."""
    total, Hq, _ = q.shape
    Hk = cache.shape[1]
    G = Hq // Hk
    out = torch.zeros(total, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((total, Hq), -math.inf, dtype=torch.float64)
    dots = torch.zeros(total, Hq, dtype=torch.float64)
    for b, L in enumerate(kv_lens.tolist()):
        s0, s1 = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        n = s1 - s0
        place = [t for t in range(min(L, page_table.shape[1] * page)) if 0 <= int(page_table[b, t // page]) < cache.shape[0]]
        k, v = get(cache, [int(page_table[b, t // page]) * page + t % page for t in place], D, bits, dtype)
        for i in range(n):
            w = (1 << (i + 1)) - 1 if tree_mask is None else int(tree_mask[s0 + i]) & (2 ** 64 - 1)
            L_seen = min(L, page_table.shape[1] * page)
            see = [j for j, t in enumerate(place) if t < L_seen - n or (w >> (t - (L_seen - n))) & 1]
            if not see:
                continue
            for h in range(Hq):
                ks, vs = k[see, h // G], v[see, h // G]
                x = ks @ q[s0 + i, h].double() * scale
                dots[s0 + i, h] = float((ks.abs() @ q[s0 + i, h].double().abs()).max()) * abs(scale)
                m = torch.logsumexp(x, 0)
                p = torch.exp(x - m)
                out[s0 + i, h], mag[s0 + i, h], lse[s0 + i, h] = p @ vs, p @ vs.abs(), m
    return out, lse, mag, dots
