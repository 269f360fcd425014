"""Serving a small attention model with drafted trees: block plan, append, paged attention together.

Prompts go in whole, as chains. Every step after that drafts a tree of tokens for each request from
the tokens that followed the last one before (a table of successors), verifies it in one pass (each
token sees its ancestors and the context), accepts the longest branch that the model itself would
have written, and appends the accepted tokens' keys and values again at their places in a row.

    python examples/serve_attention.py [--requests 8] [--prompt 300] [--steps 16]

The weights are random. At the end the first layer's keys in the pages, which depend on their own token
only, are compared with those of one dense pass over each request's tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_ssm_gdp_gb300 as gdp  # noqa: E402

VOCAB, WIDTH, H, HKV, D, BLOCK = 64, 256, 8, 2, 64, 16


class Layer:
    def __init__(self, rng, pages, device):
        draw = lambda *s: torch.randn(*s, generator=rng, device=device)  # noqa: E731
        self.w_in = (draw(WIDTH, (H + 2 * HKV) * D) * WIDTH ** -0.5).bfloat16()
        self.w_out = (draw(H * D, WIDTH) * (H * D) ** -0.5).bfloat16()
        self.keys = torch.zeros(pages, BLOCK, HKV, D, dtype=torch.bfloat16, device=device)
        self.values = torch.zeros_like(self.keys)

    def project(self, x):
        """x [T, WIDTH] -> q [T, H, D], k, v [T, HKV, D], views of one product."""
        y = (torch.nn.functional.rms_norm(x, (WIDTH,)) @ self.w_in).unflatten(-1, (H + 2 * HKV, D))
        return y.split((H, HKV, HKV), dim=1)


class Server:
    def __init__(self, layers, embed, requests, blocks, pages, device):
        self.layers, self.embed, self.device = layers, embed, device
        i32 = dict(dtype=torch.int32, device=device)
        self.tables = torch.full((requests, blocks), -1, **i32)
        self.ctx = torch.zeros(requests, **i32)
        self.free, self.used = torch.arange(pages, **i32), torch.zeros(1, **i32)
        self.status = torch.zeros(1, **i32)
        self.frequencies, _ = gdp.gdp_rotary_frequencies(D, device=device)

    def forward(self, tokens, lens, depth=None, mask=None):
        """One pass over the packed new tokens: the next token after each, and what keep() needs. depth: places
        in the tree, counted from the context (None: a chain)."""
        i32 = dict(dtype=torch.int32, device=self.device)
        cu, req, pos, slot, self.used = gdp.gdp_block_plan(
            self.ctx, torch.tensor(lens, **i32), self.tables, self.free, self.used, BLOCK, len(tokens))
        if depth is not None:
            pos = self.ctx[req.long()] + torch.tensor(depth, **i32)
        x = self.embed[torch.tensor(tokens, device=self.device)]
        kept = []
        for a in self.layers:
            q, k, v = a.project(x)
            q = gdp.gdp_cache_append(k, v, a.keys, a.values, slot, positions=pos, frequencies=self.frequencies, q=q,
                                     status=self.status)
            o = gdp.gdp_attention_paged(q[None], a.keys, a.values, self.tables, self.ctx, cu_seqlens=cu,
                                        tree_mask=None if mask is None else torch.tensor([mask], device=self.device),
                                        status=self.status)
            x = x + o[0].flatten(1) @ a.w_out
            kept.append((k, v))
        return (x @ self.embed.T).argmax(-1).tolist(), (kept, pos)

    def keep(self, kept, paths):
        """paths: for each request the rows of its accepted tokens, which move to the places behind its context."""
        kept, pos = kept
        slot = torch.full(pos.shape, -1, dtype=torch.int64)
        tables, ctx = self.tables.cpu(), self.ctx.tolist()
        for r, path in enumerate(paths):
            for place, row in enumerate(path, ctx[r]):
                slot[row] = int(tables[r, place // BLOCK]) * BLOCK + place % BLOCK
        slot = slot.to(self.device)
        for a, (k, v) in zip(self.layers, kept):
            gdp.gdp_cache_append(k, v, a.keys, a.values, slot, positions=pos, frequencies=self.frequencies,
                                 status=self.status)
        self.ctx += torch.tensor([len(p) for p in paths], dtype=torch.int32, device=self.device)


def tree(last, seen, branches=2, most=7):
    """Tokens, parents and depths of a tree that begins with `last`: up to two of the tokens that followed each."""
    tokens, parents, depth, at = [last], [-1], [0], 0
    while at < len(tokens) and len(tokens) < most:
        for t in list(dict.fromkeys(reversed(seen.get(tokens[at], []))))[:branches]:
            if len(tokens) < most:
                tokens.append(t), parents.append(at), depth.append(depth[at] + 1)
        at += 1
    return tokens, parents, depth


def serve(requests=8, prompt=300, steps=16, seed=0, device="cuda"):
    rng = torch.Generator(device=device).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    blocks = -(-(prompt + 8 * (steps + 1)) // BLOCK) + 1
    layers = [Layer(rng, requests * blocks, device) for _ in range(2)]
    embed = torch.randn(VOCAB, WIDTH, generator=rng, device=device).bfloat16()
    s = Server(layers, embed, requests, blocks, requests * blocks, device)
    streams = [torch.randint(VOCAB, (max(1, prompt - 17 * r),), generator=host).tolist() for r in range(requests)]
    lens = [len(x) for x in streams]
    after, _ = s.forward(sum(streams, []), lens)
    s.ctx += torch.tensor(lens, dtype=torch.int32, device=device)
    ends = torch.tensor(lens).cumsum(0).tolist()
    last = [after[e - 1] for e in ends]      # written, not yet in the cache
    for _ in range(steps):
        trees = []
        for r, x in enumerate(streams):
            seen = {}
            for a, b in zip(x, x[1:] + [last[r]]):
                seen.setdefault(a, []).append(b)
            trees.append(tree(last[r], seen))
        mask, first = [], 0
        for tokens, parents, _ in trees:
            bits = []
            for i, parent in enumerate(parents):
                bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
            mask += bits
        after, kept = s.forward(sum((t for t, _, _ in trees), []), [len(t) for t, _, _ in trees],
                                sum((d for _, _, d in trees), []), mask)
        paths = []
        for r, (tokens, parents, _) in enumerate(trees):
            at, path = 0, [0]                # the root is the model's own token
            while True:
                down = [i for i, parent in enumerate(parents) if parent == at and tokens[i] == after[first + at]]
                if not down:
                    break
                at = down[0]
                path.append(at)
            streams[r] += [tokens[i] for i in path]
            last[r] = after[first + at]
            paths.append([first + i for i in path])
            first += len(tokens)
        s.keep(kept, paths)
    if int(s.status):
        raise RuntimeError(f"a step reported {int(s.status)}")
    # keys of the first layer
    off = 0.0
    for r, x in enumerate(streams):
        _, k, _ = layers[0].project(embed[torch.tensor(x, device=device)])
        want = gdp.gdp_rotary(k, torch.arange(len(x), dtype=torch.int32, device=device), s.frequencies)
        page = s.tables[r].long()[torch.arange(len(x), device=device) // BLOCK]
        got = layers[0].keys[page, torch.arange(len(x), device=device) % BLOCK]
        off = max(off, float((got.float() - want.float()).norm() / want.float().norm()))
    return streams, lens, off


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args()
    streams, lens, off = serve(a.requests, a.prompt, a.steps)
    new = sum(map(len, streams)) - sum(lens)
    print(f"{len(streams)} requests, {new} tokens in {a.steps} steps, {new / a.steps / len(streams):.2f} a step each")
    print(f"keys of the first layer in pages against a dense pass: {off:.1e} apart")


if __name__ == "__main__":
    main()
