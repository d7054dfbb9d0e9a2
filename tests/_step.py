"""Plain implementations of the operators around a step of many users, for the tests: 64 bits, one token or page after another."""
import math

import torch


def lora(x, a, b, ids, scales, base):
    """float64 out, and the sum of the magnitudes of the second product's terms and of the first's through it."""
    out, mag, mag1 = base.double().clone(), torch.zeros(base.shape, dtype=torch.float64), torch.zeros(base.shape, dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if not 0 <= i < a.shape[0]:
            continue
        s = 1.0 if scales is None else float(scales[i])
        A, B, v = a[i].double(), b[i].double(), x[t].double()
        h = (A @ v) * s
        out[t] += B @ h
        mag[t] = B.abs() @ h.abs()
        mag1[t] = B.abs() @ ((A.abs() @ v.abs()) * abs(s))
    return out, mag, mag1


def probs(row, temperature):
    """float64 probabilities of a row of logits, None where it has none."""
    l = row.double()
    if torch.isnan(l).any() or bool((l == math.inf).any()) or not bool(torch.isfinite(l).any()):
        return None
    if temperature == 0:
        p = torch.zeros_like(l)
        p[int((l == l.max()).nonzero()[0])] = 1.0
        return p
    return torch.softmax(l / temperature, 0)


def verify(logits, tokens, uniforms, noise, q_start, tree_mask, draft_probs, temperature, max_q):
    """accepted, path, out tokens, probabilities (lists), and the least relative distance of a decision from its border."""
    B, V = noise.shape
    close = math.inf
    result = []
    for b in range(B):
        s, e = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        n = min(max_q, e - s)
        t = 1.0 if temperature is None else float(temperature[b])
        if n <= 0:
            result.append((0, [-1] * max_q, [-1] * max_q, [0.0] * max_q))
            continue
        up = [-1]
        for i in range(1, n):
            word = 2 ** 64 - 1 if tree_mask is None else int(tree_mask[s + i]) & (2 ** 64 - 1)
            up.append((word & ((1 << i) - 1)).bit_length() - 1)
        path, given, toks = [0], [], []
        while True:
            p = probs(logits[s + path[-1]], t)
            kids = [i for i in range(1, n) if up[i] == path[-1] and 0 <= int(tokens[s + i]) < V]
            if p is None:
                toks.append(-1)
                given.append(math.nan)
                break
            q = None if draft_probs is None else draft_probs[s + path[-1]].double()
            r, chosen = p.clone(), None
            for i in kids:
                d, u = int(tokens[s + i]), float(uniforms[s + i])
                left, right = (u * float(q[d]), float(p[d])) if q is not None else (u * float(r.sum()), float(r[d]))
                if max(left, right) > 0 and t > 0:
                    close = min(close, abs(left - right) / max(left, right))
                if left < right:
                    chosen = i
                    break
                if q is not None:
                    r = torch.clamp(p - q, min=0)
                else:
                    r[d] = 0.0
            if chosen is None:
                r = r if bool((r > 0).any()) else p
                score = torch.where(r > 0, r / noise[b].double(), torch.full_like(r, -1.0))
                j = int((score == score.max()).nonzero()[0])
                if V > 1 and t > 0:
                    two = torch.topk(score, 2).values
                    if bool(torch.isfinite(two).all()) and float(two[0]) > 0:
                        close = min(close, float((two[0] - two[1]) / two[0]))
                toks.append(j)
                given.append(float(p[j]))
                break
            path.append(chosen)
            toks.append(int(tokens[s + chosen]))
            given.append(float(p[toks[-1]]))
        k = len(path) - 1
        fill = [-1] * (max_q - k - 1)
        result.append((k, path + fill, toks + fill, given + [0.0] * len(fill)))
    return [list(x) for x in zip(*result)] if result else [[], [], [], []], close


def pages_of(n, page, cols):
    return min((max(n, 0) + page - 1) // page, cols)


def fork(refs, table, lens, parents, page):
    refs, cols = list(refs), len(table[0]) if table else 0
    rows, new = [], []
    for i in parents:
        n = max(lens[i], 0) if 0 <= i < len(lens) else 0
        have = pages_of(n, page, cols)
        row = (table[i][:have] if have else []) + [-1] * (cols - have)
        for q in row:
            if 0 <= q < len(refs):
                refs[q] += 1
        rows.append(row)
        new.append(n)
    return refs, rows, new


def reserve(refs, table, lens, new_lens, page):
    before, refs, table = list(refs), list(refs), [list(r) for r in table]
    cols = len(table[0]) if table else 0
    free = [q for q, n in enumerate(refs) if n == 0]
    held, copies, shared = [], [], {}
    for b, row in enumerate(table):
        n, new = max(lens[b], 0), new_lens[b]
        have, want = pages_of(n, page, cols), pages_of(new, page, cols)
        copy = None
        if new > n and n % page and n < cols * page:
            q = row[have - 1]
            if 0 <= q < len(refs) and before[q] > 1:
                if shared.get(q, 0) < before[q] - 1:
                    copy = q
                shared[q] = shared.get(q, 0) + 1
        pair, room = (-1, -1), have
        out = False
        if copy is not None:
            if free:
                to = free.pop(0)
                pair = (copy, to)
                refs[copy] -= 1
                refs[to] = 1
                row[have - 1] = to
            else:
                out = True
        for c in range(have, want):
            if out or not free:
                break
            row[c] = free.pop(0)
            refs[row[c]] = 1
            room = c + 1
        held.append(n if new <= n or out else max(n, min(new, room * page)))
        copies.append(pair)
    return refs, table, held, copies


def free(refs, table, lens, keep, page):
    refs, table = list(refs), [list(r) for r in table]
    for b, row in enumerate(table):
        for c in range(pages_of(keep[b] if keep else 0, page, len(row)), pages_of(lens[b], page, len(row))):
            if 0 <= row[c] < len(refs):
                refs[row[c]] = max(refs[row[c]] - 1, 0)
            row[c] = -1
    return refs, table


def compact(cache, D, bits, table, lens, path, q_start):
    """cache uint8 [layers, pages, heads, tiles, bytes] (CPU), in place; returns the new lengths."""
    L, P, H, tiles, _ = cache.shape
    page, per, out = tiles * 16, D * bits // 8, []

    def bytes_of(place, row):
        q, i = row[place // page], place % 16
        if not 0 <= q < P:
            return None
        tile = cache[:, q, :, place % page // 16]
        return [tile[..., j * 16 * per + i * per:][..., :per] for j in range(2)] + [tile[..., 32 * per + 64 * j + 4 * i:][..., :4] for j in range(2)]

    for b, row in enumerate(table):
        n = 1 if q_start is None else max(q_start[b + 1] - q_start[b], 0)
        total = min(max(lens[b], 0), len(row) * page)
        kept = []
        for i in path[b]:
            if i < 0:
                break
            kept.append(i)
        moves = []
        for k, i in enumerate(kept):
            a, z = total - n + i, total - n + k
            if i != k and i < n and k < n and a >= 0 and z >= 0:
                x, y = bytes_of(a, row), bytes_of(z, row)
                if x is not None and y is not None:
                    moves.append(([v.clone() for v in x], y))
        for x, y in moves:
            for v, w in zip(x, y):
                w.copy_(v)
        out.append(max(total - n + min(len(kept), n), 0))
    return out
