"""Serving a small linear-attention model: block plan, paged prompts, paged decoding, output norm.

Each layer is a linear attention with a decay for each head, whose heads are normalised and
gated (gdp_group_norm) before the output projection. Requests keep their states in pages of
``block`` tokens; one gdp_block_plan per step assigns the pages of all layers. A second wave of
requests continues from the whole blocks of the first one's prompt (a shared prefix).

    python examples/serve_linear_attention.py [--requests 8] [--prompt 700] [--new 32]

The weights are random. At the end, the states in the pages are compared with those of one dense
gdp_linear_chunk_fwd over each request's whole token stream.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_ssm_gdp_gb300 as gdp  # noqa: E402


class Layer:
    """Weights of one layer: a fused projection to q, k, v, the gate and the decay, and the output's."""

    def __init__(self, width, H, HV, K, V, rng, device):
        self.H, self.HV, self.K, self.V = H, HV, K, V
        self.split = (H * K, H * K, HV * V, HV * V, HV)
        draw = lambda *shape: torch.randn(*shape, generator=rng, device=device)  # noqa: E731
        self.w_in = (draw(width, sum(self.split)) * width ** -0.5).bfloat16()
        self.w_out = (draw(HV * V, width) * (HV * V) ** -0.5).bfloat16()
        self.norm = 1 + 0.1 * draw(HV * V)
        self.decay = draw(HV)

    def project(self, x):
        """x [T, width] -> q, k [T, H, K], v [T, HV, V] (views of one product), gate [T, HV V], g [T, HV]."""
        q, k, v, gate, a = (x @ self.w_in).split_with_sizes(self.split, dim=-1)
        k = torch.nn.functional.normalize(k.reshape(-1, self.H, self.K).float(), dim=-1).to(x.dtype)
        g = torch.nn.functional.logsigmoid(a.float() + self.decay + 3)
        return q.unflatten(-1, (self.H, self.K)), k, v.unflatten(-1, (self.HV, self.V)), gate, g

    def finish(self, x, o, gate):
        """Heads of o normalised, gated, projected; the residual added."""
        y = gdp.gdp_group_norm(o.reshape(x.shape[0], -1), self.HV, self.norm, gate=gate)
        return x + y @ self.w_out


class Server:
    def __init__(self, layers, embed, n_pages, max_requests, max_blocks, block, device):
        self.layers, self.embed, self.block = layers, embed, block
        self.pools = [torch.zeros(n_pages, a.HV, a.K, a.V, device=device) for a in layers]
        self.free = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.used = torch.zeros(1, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)  # of one call
        self.seen = torch.zeros_like(self.status)  # of all
        self.tables = torch.full((max_requests, max_blocks), -1, dtype=torch.int32, device=device)
        self.ctx = torch.zeros(max_requests, dtype=torch.int32, device=device)
        self.n = 0

    def plan(self, rows, query, tokens):
        """Pages and offsets of a step in which request r of `rows` takes query[r] tokens."""
        tables, ctx = self.tables[rows], self.ctx[rows]
        cu, _, _, _, self.used = gdp.gdp_block_plan(ctx, query, tables, self.free, self.used,
                                                    self.block, tokens, status=self.status)
        self.seen |= self.status
        return cu, tables, ctx

    def attend_prompts(self, q, k, v, g, cu, pool, tables, ctx):
        o = gdp.gdp_linear_chunk_fwd_paged(q[None], k[None], v[None], g[None], cu, pool, tables, ctx,
                                           self.block, status=self.status)
        self.seen |= self.status
        return o[0]

    def errors(self):
        """What any step has reported so far (synchronises)."""
        return int(self.seen)

    def prompts(self, prompts, share=None):
        """Admits requests with these prompts (token lists); `share` = (request, blocks) of a common
        prefix that is not among the tokens given. Returns their numbers and next tokens."""
        rows = slice(self.n, self.n + len(prompts))
        if share is not None:
            r, blocks = share
            self.tables[rows, :blocks] = self.tables[r, :blocks]
            self.ctx[rows] = blocks * self.block
        dev = self.ctx.device
        query = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        x = self.embed[torch.cat([torch.as_tensor(p) for p in prompts]).to(dev)]
        cu, tables, ctx = self.plan(rows, query, x.shape[0])
        for layer, pool in zip(self.layers, self.pools):
            q, k, v, gate, g = layer.project(x)
            x = layer.finish(x, self.attend_prompts(q, k, v, g, cu, pool, tables, ctx), gate)
        self.ctx[rows] += query
        self.n += len(prompts)
        return list(range(rows.start, rows.stop)), (x[cu[1:].long() - 1] @ self.embed.T).argmax(-1)

    def decode(self, tokens):
        """One token for every request; returns the next ones."""
        rows, n = slice(0, self.n), self.n
        x = self.embed[tokens]
        _, tables, ctx = self.plan(rows, torch.ones_like(self.ctx[rows]), n)
        for layer, pool in zip(self.layers, self.pools):
            q, k, v, gate, g = layer.project(x)
            o = gdp.gdp_linear_recurrent_update_paged(
                q[:, None], k[:, None], v[:, None], g[:, None], pool, tables, ctx, self.block,
                status=self.status)
            self.seen |= self.status
            x = layer.finish(x, o[:, 0], gate)
        self.ctx[rows] += 1
        return (x @ self.embed.T).argmax(-1)

    def states(self, r):
        """States of request r after its last token, layer by layer."""
        page = int(self.tables[r, (int(self.ctx[r]) - 1) // self.block])
        return [pool[page] for pool in self.pools]


def dense_states(layers, embed, tokens):
    """The same states from the dense chunked form over a whole stream."""
    x, out = embed[tokens], []
    for layer in layers:
        q, k, v, gate, g = layer.project(x)
        o, s = gdp.gdp_linear_chunk_fwd(q[None], k[None], v[None], g[None])
        x = layer.finish(x, o[0], gate)
        out.append(s[0])
    return out


def serve(requests=8, prompt=700, new=32, block=128, width=512, H=4, HV=8, K=64, V=64, depth=2,
          vocab=1000, device="cuda", seed=0):
    """Runs both waves and the decoding; returns the token streams and, for each request, the
    largest relative difference of its paged states from the dense ones."""
    rng = torch.Generator(device=device).manual_seed(seed)
    layers = [Layer(width, H, HV, K, V, rng, device) for _ in range(depth)]
    embed = torch.randn(vocab, width, generator=rng, device=device).bfloat16()
    lens = [max(1, prompt - 37 * r) for r in range(requests)]
    host = torch.Generator().manual_seed(seed)
    first = [torch.randint(vocab, (n,), generator=host).tolist() for n in lens]
    shared = lens[0] // block  # whole blocks of request 0's prompt
    second = [torch.randint(vocab, (5 + 60 * r,), generator=host).tolist() for r in range(2)]
    blocks = -(-(prompt + 200 + new) // block)
    s = Server(layers, embed, (requests + 2) * blocks, requests + 2, blocks, block, device)
    _, next1 = s.prompts(first)
    _, next2 = s.prompts(second, share=(0, shared))
    streams = first + [first[0][:shared * block] + p for p in second]
    token = torch.cat([next1, next2])
    start = time.perf_counter()
    for _ in range(new):
        for stream, t in zip(streams, token.tolist()):
            stream.append(t)
        token = s.decode(token)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    if s.errors():
        raise RuntimeError(f"a step reported {s.errors()}")
    off = []
    for r, stream in enumerate(streams):
        want = dense_states(layers, embed, torch.tensor(stream, device=device))
        off.append(max(float((a - b).norm() / b.norm()) for a, b in zip(s.states(r), want)))
    return streams, off, took


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prompt", type=int, default=700)
    p.add_argument("--new", type=int, default=32)
    a = p.parse_args()
    streams, off, took = serve(a.requests, a.prompt, a.new)
    print(f"{len(streams)} requests, {sum(map(len, streams))} tokens, "
          f"{1e6 * took / a.new:.0f} us per decode step")
    print(f"paged against dense states: at most {max(off):.1e} apart")


if __name__ == "__main__":
    main()
