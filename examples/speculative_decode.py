"""Greedy decoding with trees of drafted tokens on W4A16 layers and the serving operators around them.

A small decoder (random weights) runs the step a served model runs: W4A16 QKV projection, keys and queries
turned and the cache written in one call, attention of the drafted tree over the 4-bit paged cache, W4A16
output projection and MLP, W4A16 head, log probabilities of the drafted tokens with the best alternatives.
The accepted path's keys and values are then written again at their final slots.

    python examples/speculative_decode.py            (needs the built library and a GPU)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_int4_weight_group_gb300 as w4  # noqa: E402


def linear(gen, k, n, dtype, group=128):
    """A W4A16 layer [k -> n] of random codes, of about unit gain."""
    q = torch.randint(0, 16, (k, n), generator=gen, dtype=torch.uint8).cuda()
    scales = torch.full((k // group, n), 0.22 * k ** -0.5, dtype=dtype, device="cuda")
    return w4.W4A16Linear(w4.w4a16_pack(q), scales, None, group)


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Decoder:
    """`layers` pre-norm blocks of attention and a gated MLP with a tied-free head; one sequence, paged 4-bit cache."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, layers=2, vocab=2048, pages=32, page_size=32,
                 dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.dtype, self.page_size = q_heads, kv_heads, head_dim, dtype, page_size
        self.embedding = torch.randn(vocab, hidden, generator=g).to(dtype).cuda()
        self.layers = [dict(qkv=linear(g, hidden, (q_heads + 2 * kv_heads) * head_dim, dtype), out=linear(g, q_heads * head_dim, hidden, dtype),
                            up=linear(g, hidden, 4 * hidden, dtype), down=linear(g, 2 * hidden, hidden, dtype),
                            cache=w4.w4a16_kv_cache(pages, kv_heads, head_dim, page_size, bits=4)) for _ in range(layers)]
        self.head = linear(g, hidden, vocab, dtype)
        self.table = w4.w4a16_rope_table(4 * pages * page_size, head_dim, base=10000.0, scaling="yarn", factor=4.0,
                                         original_max_positions=pages * page_size)
        # the sequence's pages, in some order
        self.pages = torch.randperm(pages, generator=g).to(torch.int32).cuda()[None]

    def slots(self, index):
        """Cache slots of the sequence's tokens `index`."""
        return self.pages[0, index // self.page_size].long() * self.page_size + index % self.page_size

    def step(self, tokens, positions, first, tree_mask):
        """Logits of `tokens` (int64 [n], n <= 64), which become the sequence's tokens first, first + 1, ..: token i sees the
        earlier ones and those of these whose bits are set in tree_mask[i]. Returns the layers' raw keys and values too."""
        n = tokens.numel()
        slots = self.slots(torch.arange(first, first + n, device="cuda"))
        kv_lens = torch.tensor([first + n], dtype=torch.int32, device="cuda")
        q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        x, kept = self.embedding[tokens], []
        for layer in self.layers:
            qkv = layer["qkv"](norm(x)).view(n, -1, self.head_dim)
            q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            q = w4.w4a16_kv_write(k, v, layer["cache"], slots, q=q, positions=positions, table=self.table)
            y = w4.w4a16_tree_attention(q, layer["cache"], self.pages, kv_lens, q_start=q_start, tree_mask=tree_mask, max_q=n)
            x = x + layer["out"](y.view(n, -1))
            gate, up = layer["up"](norm(x)).chunk(2, 1)
            x = x + layer["down"]((torch.nn.functional.silu(gate) * up).contiguous())
            kept.append((k, v))
        return self.head(norm(x)), kept

    def keep(self, kept, rows, positions, first):
        """Write the rows' keys and values again, as the sequence's tokens first, first + 1, .."""
        slots = self.slots(torch.arange(first, first + rows.numel(), device="cuda"))
        for layer, (k, v) in zip(self.layers, kept):
            w4.w4a16_kv_write(k[rows], v[rows], layer["cache"], slots, positions=positions, table=self.table)


def decode(model, prompt, steps, draft):
    """Greedy tokens after `prompt` (a list). draft(tokens) -> a tree of guesses for what follows: a list of (parent, token),
    parent an earlier index of the list or -1 for the last token. Returns the tokens and the accepted guesses of each step."""
    tokens, accepted = list(prompt), []
    at = 0
    while at < len(prompt) - 1:  # the prompt but its last token, in chains of at most 64
        part = torch.tensor(prompt[at:min(at + 64, len(prompt) - 1)], device="cuda")
        model.step(part, torch.arange(at, at + part.numel(), device="cuda"), at, None)
        at += part.numel()
    while len(tokens) < len(prompt) + steps:
        first = len(tokens) - 1  # the last token is not in the cache yet: it is the tree's root
        nodes = [(-1, tokens[-1])] + [(p + 1, t) for p, t in draft(tokens)]
        depth, masks = [], []
        for i, (p, _) in enumerate(nodes):
            depth.append(0 if i == 0 else depth[p] + 1)
            masks.append((0 if i == 0 else masks[p]) | (1 << i))
        positions = torch.tensor([first + d for d in depth], device="cuda")
        mask = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], device="cuda")
        logits, kept = model.step(torch.tensor([t for _, t in nodes], device="cuda"), positions, first, mask)
        # the guesses' own log probabilities come with the best alternative of each node
        _, _, best, _ = w4.w4a16_token_logprobs(logits, None, 1)
        best = best[:, 0].tolist()
        path, node = [0], 0
        while True:
            tokens.append(best[node])
            follow = [i for i, (p, t) in enumerate(nodes) if i and p == node and t == best[node]]
            if not follow:
                break
            node = follow[0]
            path.append(node)
        accepted.append(len(path) - 1)
        rows = torch.tensor(path, device="cuda")
        if path != list(range(len(path))):
            model.keep(kept, rows, positions[rows], first)
    return tokens[:len(prompt) + steps], accepted


def main():
    model = Decoder()
    prompt = torch.randint(0, 2048, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    plain, _ = decode(model, prompt, 48, lambda tokens: [])
    gen = torch.Generator().manual_seed(2)

    def draft(tokens):  # a stand-in for a draft model: mostly the right continuation, between wrong ones
        tree, parent = [], -1
        for i, t in enumerate(plain[len(tokens):len(tokens) + 4]):
            wrong = torch.randint(0, 2048, (2,), generator=gen).tolist()
            guesses = [(parent, wrong[0]), (parent, t if torch.rand(1, generator=gen) < 0.8 else wrong[1])]
            tree += guesses
            parent = len(tree) - 1
        return tree

    fast, accepted = decode(model, prompt, 48, draft)
    print(f"{len(accepted)} steps for {len(fast) - len(prompt)} tokens, {sum(accepted)} guesses accepted")
    print("the same tokens as one by one" if fast == plain else f"the first {next(i for i, (a, b) in enumerate(zip(fast, plain)) if a != b)} tokens agree")


if __name__ == "__main__":
    main()
