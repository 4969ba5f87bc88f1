"""Windows, their visibility in clusters of CTAs, tokens against a window and against a 4-bit cache on two
streams at once, and captured into a graph that is replayed with other inputs: the bits of calls one by one."""

import pytest
import torch

import exact_attention_23_gb300 as fa


class _Work:
    """A step of each operator with its own inputs, workspaces and results."""

    def __init__(self, seed, d, B=2, H=8, Hkv=2, T=4500, n=3, Tmax=2600):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        self.q, self.do = new(1, H, T, d), new(1, H, T, d)
        self.k, self.v = new(1, Hkv, T, d), new(1, Hkv, T, d)
        self.ids = (torch.arange(T, dtype=torch.int32) // (700 + seed))[None].contiguous().cuda()
        self.tq, self.kc, self.vc = new(B, H, n, d), new(B, Hkv, Tmax, d), new(B, Hkv, Tmax, d)
        self.ctx = torch.tensor([Tmax - n, 900 + seed], dtype=torch.int32).cuda()
        self.cache, self.zero = fa.cache4(B, Hkv, Tmax, d), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.rest = torch.empty_like(self.q)
        self.ws = fa.bwd_mod_workspace(1, H, Hkv, T, d, window=200, sinks=4)

    def step(self):
        seen = fa.visible(1, self.q.shape[2], doc_ids=self.ids, window=200, sinks=4)
        o, lse = fa.fwd_mod(self.q, self.k, self.v, visible=seen, rest=self.rest)
        _, dk, dv = fa.bwd_mod(self.q, self.k, self.v, o, lse, self.do, visible=seen, rest=self.rest, workspace=self.ws)
        fa.append4(self.kc, self.vc, self.cache, self.zero)
        return (o, lse, self.rest, dk, dv, *fa.fwd_tree(self.tq, self.kc, self.vc, self.ctx, window=1500, sinks=4),
                *fa.fwd_tree4(self.tq, self.cache, self.ctx), *fa.fwd_tree4(self.tq, self.cache, self.ctx, window=800, sinks=130))


def _same(a, b):
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_two_streams_at_once(d):
    works = [_Work(s, d) for s in (1, 2)]
    want = [[x.clone() for x in w.step()] for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (w, s) in enumerate(zip(works, streams)):
            with torch.cuda.stream(s):
                got[i].append([x.clone() for x in w.step()])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x in a:
            _same(x, b)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_captured_and_replayed(d):
    w, other = _Work(3, d), _Work(4, d)
    want = [x.clone() for x in other.step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w.step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held = w.step()
    for name in ("q", "k", "v", "do", "ids", "tq", "kc", "vc", "ctx"):
        getattr(w, name).copy_(getattr(other, name))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        _same(held, want)
