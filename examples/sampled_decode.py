"""Sampling several answers for several users at once: trees of guesses, an adapter for each user, one pool of pages.

The users' prompts are read once, each forked into a number of answers that share its pages. A step reserves pages for
the guesses (a shared page that would be written is replaced by a copy), runs the W4A16 layers with every user's low-rank adapter
beside them, decides on the device which guesses stand, moves their keys and values together in all layers and gives the
pages of the others back. Only the tokens that came out go to the host, where the next guesses are made.

    python examples/sampled_decode.py            (needs the built library and a GPU)
"""
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]
import w4a16_int4_weight_group_gb300 as w4  # noqa: E402
from speculative_decode import linear, norm  # noqa: E402


class Server:
    """`layers` pre-norm blocks of attention and a gated MLP; a paged 4-bit cache of all layers; adapters on two projections."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, layers=2, vocab=2048, pages=160, page=16, adapters=3, rank=16,
                 dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.page, self.vocab = q_heads, kv_heads, head_dim, page, vocab
        self.embedding = torch.randn(vocab, hidden, generator=g).to(dtype).cuda()
        wide = (q_heads + 2 * kv_heads) * head_dim

        def adapter(k, n):
            a = torch.randn(adapters, rank, k, generator=g) * k ** -0.5
            b = torch.randn(adapters, n, rank, generator=g) * 0.3 * rank ** -0.5
            return a.to(dtype).cuda(), b.to(dtype).cuda()

        self.layers = [dict(qkv=linear(g, hidden, wide, dtype), qkv_adapter=adapter(hidden, wide), out=linear(g, q_heads * head_dim, hidden, dtype),
                            up=linear(g, hidden, 4 * hidden, dtype), up_adapter=adapter(hidden, 4 * hidden),
                            down=linear(g, 2 * hidden, hidden, dtype)) for _ in range(layers)]
        self.head = linear(g, hidden, vocab, dtype)
        self.caches = torch.stack([w4.w4a16_kv_cache(pages, kv_heads, head_dim, page, bits=4) for _ in range(layers)])
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.max_pages = pages // 4
        self.rope = w4.w4a16_rope_table(self.max_pages * page, head_dim)

    def _project(self, layer, name, x, users):
        y = layer[name](x)
        return w4.w4a16_lora(x, *layer[name + "_adapter"], users, y, out=y)

    def give_back(self, table, lens, keep=None):
        w4.w4a16_kv_free(self.refs, table, lens, self.page, keep=keep)

    def step(self, table, lens, users, tokens, positions, q_start, mask, max_q):
        """Logits of the sequences' next tokens; these go into the cache behind the `lens` that are there. Returns the lengths too.
        MemoryError where the pool has no room for all of them: nothing was written, and what was reserved has been given back."""
        count = q_start[1:] - q_start[:-1]
        want = lens + count
        held, copies = w4.w4a16_kv_reserve(self.refs, table, lens, want, self.page)
        w4.w4a16_kv_copy(self.caches, copies)
        if bool((held < want).any()):  # (a page that others hold too, or none at all, stands where tokens would be written)
            self.give_back(table, held, keep=lens)
            raise MemoryError(f"{int((held < want).sum())} of {len(lens)} sequences have no room for their tokens")
        seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count, output_size=tokens.numel())
        place = torch.arange(tokens.numel(), device="cuda") - q_start[seq] + lens[seq]
        slots = table[seq, place // self.page].long() * self.page + place % self.page
        users, x = users[seq], self.embedding[tokens]
        for layer, cache in zip(self.layers, self.caches):
            qkv = self._project(layer, "qkv", norm(x), users).view(tokens.numel(), -1, self.head_dim)
            q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            q = w4.w4a16_kv_write(k, v, cache, slots, q=q, positions=positions, table=self.rope)
            y = w4.w4a16_tree_attention(q, cache, table, want, q_start=q_start, tree_mask=mask, max_q=max_q)
            x = x + layer["out"](y.view(tokens.numel(), -1))
            gate, up = self._project(layer, "up", norm(x), users).chunk(2, 1)
            x = x + layer["down"]((torch.nn.functional.silu(gate) * up).contiguous())
        return self.head(norm(x)), want

    def read(self, prompt, user):
        """The prompt but its last token in the cache: a table row and its length."""
        table = torch.full((1, self.max_pages), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        users = torch.tensor([user], dtype=torch.int32, device="cuda")
        try:
            for at in range(0, len(prompt) - 1, 64):
                part = torch.tensor(prompt[at:min(at + 64, len(prompt) - 1)], device="cuda")
                start = torch.tensor([0, part.numel()], dtype=torch.int32, device="cuda")
                _, lens = self.step(table, lens, users, part, torch.arange(at, at + part.numel(), device="cuda"), start, None, part.numel())
        except MemoryError:
            self.give_back(table, lens)
            raise
        return table, lens


def decode(server, prompts, users, answers, steps, draft, temperature=1.0, seed=0):
    """`answers` samples of at least `steps` tokens after each prompt (a list of lists of tokens). draft(tokens) -> guesses for what
    follows: a list of (parent, token), parent an earlier index of the list or -1. Returns the token lists and the guesses that
    were accepted. users[i]: the adapter of prompt i, or -1. MemoryError where the pages run out; all of them are given back then."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = []
    try:
        for p, u in zip(prompts, users):
            rows.append(server.read(p, u))
    except MemoryError:
        for t, n in rows:
            server.give_back(t, n)
        raise
    first, first_lens = torch.cat([t for t, _ in rows]), torch.cat([n for _, n in rows])
    parents = torch.arange(len(prompts) * answers, dtype=torch.int32, device="cuda") // answers
    table, lens = w4.w4a16_kv_fork(server.refs, first, first_lens, parents, server.page)
    server.give_back(first, first_lens)  # the answers hold the prompts' pages now
    out = [list(p) for p in prompts for _ in range(answers)]
    user = torch.tensor(users, dtype=torch.int32, device="cuda")[parents.long()].contiguous()
    temp = torch.full((len(out),), temperature, device="cuda")
    accepted = 0
    for _ in range(steps):
        if min(len(o) - len(prompts[i // answers]) for i, o in enumerate(out)) >= steps:
            break
        tokens, depth, masks, start = [], [], [], [0]
        for o in out:
            nodes = [(-1, o[-1])] + [(p + 1, t) for p, t in draft(o)]
            d, m = [], []
            for i, (p, t) in enumerate(nodes):
                d.append(0 if i == 0 else d[p] + 1)
                m.append((0 if i == 0 else m[p]) | (1 << i))
            tokens += [t for _, t in nodes]
            depth += [len(o) - 1 + x for x in d]
            masks += [x - (1 << 64) if x >> 63 else x for x in m]
            start.append(len(tokens))
        n = max(b - a for a, b in zip(start, start[1:]))
        start = torch.tensor(start, dtype=torch.int32, device="cuda")
        mask, ids = torch.tensor(masks, device="cuda"), torch.tensor(tokens, device="cuda")
        try:
            logits, want = server.step(table, lens, user, ids, torch.tensor(depth, device="cuda"), start, mask, n)
        except MemoryError:
            server.give_back(table, lens)
            raise
        uniforms = torch.rand(len(tokens), generator=g, device="cuda")
        noise = torch.empty(len(out), server.vocab, device="cuda").exponential_(generator=g)
        _, path, new, _ = w4.w4a16_verify_drafts(logits, ids, uniforms, noise, q_start=start, tree_mask=mask, temperature=temp, max_q=n)
        lens = w4.w4a16_kv_compact(server.caches, server.head_dim, table, want, path, q_start=start)
        server.give_back(table, want, keep=lens)
        for o, row in zip(out, new.tolist()):
            got = [t for t in row if t >= 0]
            o += got
            accepted += len(got) - 1
    server.give_back(table, lens)
    return out, accepted


def main():
    server = Server()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, server.vocab, (n,), generator=g).tolist() for n in (70, 23, 110)]
    plain, _ = decode(server, prompts, [0, 1, -1], 2, 24, lambda tokens: [], temperature=0.0)
    following = {tuple(o[:i]): o[i] for o in plain for i in range(20, len(o))}

    def draft(tokens):  # a stand-in for a draft model: the likeliest continuation beside a wrong one, three deep
        tree, parent, seen = [], -1, list(tokens)
        for _ in range(3):
            t = following.get(tuple(seen), 0)
            tree += [(parent, (t + 1) % server.vocab), (parent, t)]
            parent = len(tree) - 1
            seen.append(t)
        return tree

    for temperature in (0.0, 0.7):
        out, accepted = decode(server, prompts, [0, 1, -1], 2, 24, draft, temperature)
        print(f"temperature {temperature}: {sum(len(o) for o in out) - 2 * sum(map(len, prompts))} tokens, {accepted} guesses accepted")
    print(f"{int((server.refs != 0).sum())} pages held at the end")


if __name__ == "__main__":
    main()
