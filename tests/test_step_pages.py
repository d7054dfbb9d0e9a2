"""A page that several sequences hold is written by one of them only once the others have copies of their own, also where pages run out.

`reserve` here follows the C header's words; what it hands out is also written and read back, so that a wrong rule shows as another
sequence's overwritten tokens whatever the rule's own model says."""
import itertools

import pytest
import torch

PAGE, D, BITS = 16, 64, 4
TILE = 4 * D * BITS + 128


def reserve(refs, table, lens, new_lens):
    refs, table = list(refs), [list(r) for r in table]
    cols = len(table[0])
    grows = [b for b in range(len(table)) if new_lens[b] > lens[b]]
    tail = {b: table[b][lens[b] // PAGE] for b in grows if lens[b] % PAGE and lens[b] // PAGE < cols}
    asks = set()
    for page in set(tail.values()):
        mine = [b for b in grows if tail.get(b) == page]
        others = refs[page] - len(mine)  # sequences that the call does not grow
        asks.update(mine if others else mine[:-1])
    copies, room = [(-1, -1)] * len(table), [-(-n // PAGE) for n in lens]
    free = [q for q, n in enumerate(refs) if n == 0]
    out = False
    for b in grows:
        if b in asks and not out:
            if free:
                copies[b] = (tail[b], free.pop(0))
                refs[tail[b]] -= 1
                refs[copies[b][1]] = 1
                table[b][lens[b] // PAGE] = copies[b][1]
            else:
                out = True
        while not out and room[b] < min(-(-new_lens[b] // PAGE), cols):
            if free:
                table[b][room[b]] = free.pop(0)
                refs[table[b][room[b]]] = 1
                room[b] += 1
            else:
                out = True
    held = list(lens)
    for b in grows:
        last = table[b][lens[b] // PAGE] if b in tail else None
        if last is None or refs[last] == 1:
            held[b] = max(lens[b], min(new_lens[b], room[b] * PAGE))
    return refs, table, held, copies


def cells(table, b, lo, hi):
    """Page, tile and first byte of the K codes of tokens lo .. hi - 1 (tiles of 16 tokens, D * BITS / 8 bytes a token)."""
    return [(table[b][t // PAGE], t % PAGE // 16, t % 16 * (D * BITS // 8)) for t in range(lo, hi)]


def write(cache, table, b, lo, hi, value):
    for t, (q, tile, at) in enumerate(cells(table, b, lo, hi), lo):
        assert q >= 0
        cache[0, q, 0, tile, at:at + D * BITS // 8] = value(t)


def holders(lens, spare, cols=5):
    """One prompt, forked to sequences of these lengths (the longest whole, the others' ends given back), and `spare` free pages."""
    most = -(-max(lens) // PAGE)
    table = [[q if q < -(-n // PAGE) else -1 for q in range(cols)] for n in lens]
    refs = [sum(q in row for row in table) for q in range(most)] + [0] * spare
    cache = torch.zeros(1, len(refs), 1, PAGE // 16, TILE, dtype=torch.uint8)
    write(cache, table, lens.index(max(lens)), 0, max(lens), lambda t: t + 1)
    return refs, table, cache


def untouched(cache, table, lens, held, new_lens):
    """Every growing sequence writes what it has room for; then all tokens are those of their sequence."""
    for b, n in enumerate(lens):
        write(cache, table, b, n, held[b], lambda t: 100 + b)
    for b, n in enumerate(lens):
        for t, (q, tile, at) in enumerate(cells(table, b, 0, held[b])):
            want = t + 1 if t < n else 100 + b
            assert (cache[0, q, 0, tile, at:at + D * BITS // 8] == want).all(), (b, t)


CASES = [([25, 20], [27, 23], 0), ([20, 25], [23, 27], 0), ([25, 20], [27, 23], 1), ([25, 20], [25, 23], 0), ([20, 18], [24, 24], 0),
         ([21, 21], [24, 24], 0), ([21, 21], [24, 40], 0), ([21, 21], [24, 40], 1), ([25, 32], [30, 40], 0), ([16, 16], [20, 20], 1)]
CASES += [(list(lens), [n + 4 for n in lens], spare) for lens in itertools.permutations([25, 20, 30]) for spare in range(4)]
CASES += [([25, 20, 30], [40, 20, 50], s) for s in range(5)] + [([17, 18, 19, 20, 20], [40, 30, 19, 22, 50], s) for s in range(8)]


@pytest.mark.parametrize("lens,new_lens,spare", CASES)
def test_the_headers_rule_leaves_every_token_alone(lens, new_lens, spare):
    refs, table, cache = holders(lens, spare)
    refs, table, held, copies = reserve(refs, table, lens, new_lens)
    for a, z in copies:
        if a >= 0:
            cache[:, z] = cache[:, a]
    untouched(cache, table, lens, held, new_lens)
    for b, n in enumerate(lens):
        assert held[b] == n or n % PAGE == 0 or refs[table[b][n // PAGE]] == 1


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new_lens,spare", CASES)
def test_a_shared_page_is_not_written_where_pages_run_out(lens, new_lens, spare):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as w
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refs, table, cache = holders(lens, spare)
    tr, tt, tc = i32(refs), i32(table), cache.cuda()
    now, want, order = list(lens), list(new_lens), list(range(len(lens)))
    for _ in range(2):  # again with the rows in the other order: who was told to wait is now in front
        held, copies = w.w4a16_kv_reserve(tr, tt, i32(now), i32(want), PAGE)
        w.w4a16_kv_copy(tc, copies)
        r, t, h, c = reserve(refs, table, now, want)
        cache = tc.cpu()
        assert held.tolist() == h and tr.tolist() == r and tt.tolist() == t and copies.tolist() == [list(x) for x in c]
        untouched(cache, tt.tolist(), now, held.tolist(), want)
        order.reverse()
        refs, table, now, want, tt = r, t[::-1], now[::-1], want[::-1], tt.flip(0).contiguous()
        # (what was reserved and not used goes back)
        w.w4a16_kv_free(tr, tt, held.flip(0).contiguous(), PAGE, keep=i32(now))
        for b, n in enumerate(now):
            for col in range(-(-n // PAGE), -(-h[::-1][b] // PAGE)):
                refs[table[b][col]] -= 1
                table[b][col] = -1
        assert tr.tolist() == refs and tt.tolist() == table
        tc = cache.cuda()
