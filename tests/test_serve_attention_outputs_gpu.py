"""The attention serving example's outputs: what every accepted token got from attention, in the prompts' pass and in the
trees', is dense attention in 64 bits over its stream as the pages hold it at the end. A mask that is not used, a token
at another place or an output of zeros is far outside; tolerances are test_attention_gpu's."""
import importlib.util
import os

import pytest
import torch

from test_attention_gpu import BF, UNIT

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention_outputs", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_outputs_of_accepted_tokens(gdp, monkeypatch):
    m = load()
    calls, servers = [], []
    attention = gdp.gdp_attention_paged

    def recorded(q, *a, **kw):
        o = attention(q, *a, **kw)
        calls.append((q[0].clone(), o[0].clone()))
        return o

    class Server(m.Server):
        def __init__(self, *a):
            super().__init__(*a)
            servers.append(self)
            self.got = []                          # (layer, request, position, q, o) of accepted tokens
            self.seen = 0                          # calls whose tokens have been taken

        def take(self, paths):
            for r, path in enumerate(paths):
                for place, row in enumerate(path, int(self.ctx[r])):
                    for n in range(len(self.layers)):
                        q, o = calls[self.seen + n]
                        self.got.append((n, r, place, q[row], o[row]))
            self.seen = len(calls)

        def forward(self, tokens, lens, depth=None, mask=None):
            out = super().forward(tokens, lens, depth, mask)
            if mask is None:                       # prompts: every token stays
                ends = torch.tensor(lens).cumsum(0).tolist()
                self.take([range(e - n, e) for e, n in zip(ends, lens)])
            return out

        def keep(self, kept, paths):
            self.take(paths)
            super().keep(kept, paths)

    monkeypatch.setattr(m.gdp, "gdp_attention_paged", recorded)
    monkeypatch.setattr(m, "Server", Server)
    streams, lens, _ = m.serve(requests=4, prompt=60, steps=6)
    s, = servers
    assert len(s.got) == 2 * sum(map(len, streams))
    assert sum(map(len, streams)) > sum(lens) + 6 * len(lens)    # trees gave more than their roots
    G, D, u = m.H // m.HKV, m.D, UNIT[BF]
    for n, r, place, q, o in s.got:
        at = torch.arange(place + 1, device=q.device)
        page = s.tables[r].long()[at // m.BLOCK]
        k, v = (c[page, at % m.BLOCK].double().repeat_interleave(G, 1) for c in (s.layers[n].keys, s.layers[n].values))
        p = torch.softmax(torch.einsum("hd,jhd->hj", q.double(), k) * D ** -0.5, -1)
        size = torch.einsum("hd,jhd->hj", q.double().abs(), k.abs()).amax(-1, keepdim=True) * D ** -0.5
        want, A = (torch.einsum("hj,jhd->hd", p, x) for x in (v, v.abs()))
        tol = u * want.abs() + A * (u + 2 * (D + 4) * 2.0 ** -24 * size + 2.0 ** -20 + (80 + place / 16) * 2.0 ** -23)
        assert bool(((o.double() - want).abs() <= tol).all()), (n, r, place)
