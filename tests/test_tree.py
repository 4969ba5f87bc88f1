"""New tokens against a cache (fwd_tree): refusals on the CPU, GPU parity with the 64-bit reference
of mod_reference.py under its bounds, and the serving step rope_append → fwd_tree as it is used."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref

A, SZ = 0x7F0000000000, 1 << 34
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED


def _call(q=A, k=A + SZ, v=A + 2 * SZ, o=A + 3 * SZ, lse=A + 4 * SZ, ctx=A + 5 * SZ, tree=None,
          depths=None, cap=0.0, slopes=None, B=2, H=4, Hkv=2, Tq=8, Tmax=5000, d=64, scale=0.125,
          ws=A + 6 * SZ, ws_bytes=1 << 30):
    return fa.fa_fwd_tree(q, k, v, o, lse, ctx, tree, 1, depths, 1, cap, slopes, B, H, Hkv, Tq, Tmax,
                          d, scale, ws, ws_bytes, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(k=0), BAD), (dict(o=0), BAD), (dict(lse=0), BAD), (dict(ctx=0), BAD),
    (dict(ws=0), BAD), (dict(B=0), BAD), (dict(Tq=0), BAD), (dict(Tmax=0), BAD), (dict(Hkv=3), BAD),
    (dict(d=80), BAD), (dict(scale=math.inf), BAD), (dict(cap=-2.0), BAD), (dict(cap=math.nan), BAD),
    (dict(ws_bytes=100), BAD), (dict(Tmax=(1 << 31) - 1), BAD), (dict(Tq=1 << 25), BAD),
    (dict(B=1 << 15, H=1 << 10, Hkv=1 << 10, Tmax=1 << 20), BAD),
    (dict(q=A + 8), MIS), (dict(ws=A + 6 * SZ + 64), MIS), (dict(ctx=A + 5 * SZ + 2), MIS),
    (dict(depths=A + 7 * SZ + 1), MIS), (dict(slopes=A + 7 * SZ + 2), MIS),
    (dict(o=A), BAD), (dict(o=A + SZ), BAD), (dict(lse=A + 3 * SZ), BAD), (dict(ws=A + 2 * SZ), BAD),
    (dict(tree=A + 3 * SZ), BAD), (dict(lse=A + 5 * SZ), BAD),
])
def test_refusals(kw, want):
    assert _call(**kw) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_without_device():
    assert _call(tree=A + 7 * SZ + 1, cap=30.0) == fa.FA_ERR_UNSUPPORTED_DEVICE  # (bytes: any address)
    assert _call(B=1, H=2, Hkv=1, Tmax=100, ws=None, ws_bytes=0) == fa.FA_ERR_UNSUPPORTED_DEVICE  # a short cache needs none
    assert fa.fa_fwd_tree_workspace_size(2, 4, 2, 8, 100, 64) == 0
    with pytest.raises(ValueError):
        x = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
        fa.fwd_tree(x, x, x, torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------------------- parity (GPU)

def _trees(B, n, seed):
    """Random trees (uint8 [B, n, n], depths int32 [B, n]): a node's parent is an earlier one or
    the context."""
    g = torch.Generator().manual_seed(seed)
    vis, dep = torch.zeros(B, n, n, dtype=torch.uint8), torch.zeros(B, n, dtype=torch.int32)
    for b in range(B):
        for t in range(n):
            p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            if p >= 0:
                vis[b, t], dep[b, t] = vis[b, p], dep[b, p] + 1
            vis[b, t, t] = 1
    return vis, dep


def _seen(ctx, n, Tmax, tree):
    """([B, n, Tmax] visible rows) by the definition."""
    B = len(ctx)
    ok = torch.zeros(B, n, Tmax, dtype=torch.bool)
    for b, c in enumerate(ctx):
        if c < 0:
            continue
        ok[b, :, :min(c, Tmax)] = True
        for s in range(n):
            if c + s < Tmax:
                for t in range(n):
                    ok[b, t, c + s] = s <= t if tree is None else bool(tree[b, t, s])
    return ok


def _data(B, H, Hkv, n, Tmax, d, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, t, s=1.0: (torch.randn(B, h, t, d, generator=g) * s).to(torch.bfloat16)
    return mk(H, n, std), mk(Hkv, Tmax), mk(Hkv, Tmax)


def _check(ctx, H, Hkv, n, Tmax, d, tree=False, cap=0.0, bias=False, seed=0):
    B = len(ctx)
    q, k, v = _data(B, H, Hkv, n, Tmax, d, seed + Tmax + n, 4.0 if cap else 1.0)
    t, dep = _trees(B, n, seed) if tree else (None, None)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]) if bias else None
    qa = torch.tensor(ctx)[:, None] + (torch.arange(n) if dep is None else dep)
    ka = torch.arange(Tmax).repeat(B, 1)
    for b, c in enumerate(ctx):
        m = max(0, min(n, Tmax - c)) if c >= 0 else 0
        if m:
            ka[b, c:c + m] = qa[b, :m]
    r = ref.attention(q, k, v, _seen(ctx, n, Tmax, t), d ** -0.5, cap, sl, query_at=qa, key_at=ka)
    kc, vc = k.clone(), v.clone()
    for b, c in enumerate(ctx):               # rows behind the last new token hold anything
        kc[b, :, max(0, c + n) if c >= 0 else 0:] = math.nan
        vc[b, :, max(0, c + n) if c >= 0 else 0:] = math.nan
    o, lse = fa.fwd_tree(q.cuda(), kc.cuda(), vc.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                         tree=None if t is None else t.cuda(), depths=None if dep is None else dep.cuda(),
                         softcap=cap, slopes=None if sl is None else sl.cuda())
    torch.cuda.synchronize()
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))


# room: longer caches have their work shared out in stretches, shorter ones a CTA an entry
@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 3300])
@pytest.mark.parametrize("ctx,H,Hkv,n,Tmax,d,tree,cap,bias", [
    ([0], 1, 1, 1, 1, 64, False, 0.0, False),                    # one row in all
    ([5], 2, 2, 1, 6, 128, False, 0.0, False),
    ([63, 64, 62], 4, 4, 1, 70, 64, False, 30.0, False),         # a new token at a chunk's ends
    ([0, 200, -1, 1, 500], 8, 2, 1, 512, 64, False, 0.0, True),  # empty and inactive ones among them
    ([1000, 3, 700], 16, 1, 1, 1024, 128, False, 50.0, True),    # sixteen heads on one
    ([129, 0], 6, 2, 5, 140, 64, True, 0.0, False),
    ([300, 77], 4, 2, 16, 320, 128, True, 0.0, True),            # 32 rows
    ([100, 90, 64], 12, 12, 9, 130, 64, True, 30.0, True),
    ([511], 16, 4, 16, 600, 64, True, 5.0, False),               # 64 rows
    ([90, 400], 5, 5, 33, 450, 128, False, 0.0, True),           # a chain of 33
    ([40, 1200], 8, 2, 30, 1300, 64, True, 0.0, True),           # 120 rows: two row blocks
    ([30, 2], 8, 1, 64, 100, 128, True, 20.0, False),            # 512 rows; one runs over the end
    ([100, 95, 120], 2, 1, 4, 100, 64, False, 0.0, False),       # full caches, drafts outside
])
def test_parity(ctx, H, Hkv, n, Tmax, d, tree, cap, bias, room):
    _check(ctx, H, Hkv, n, Tmax + room, d, tree, cap, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_parity_split_over_every_cta(d):
    """Contexts long enough that each lies in several stretches, ragged by two orders."""
    _check([40000, 123, 9000, 0, 21111], 4, 2, 3, 40100, d, True, 0.0, False, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("Tmax", [210, 2500])
def test_many_sequences(Tmax):
    """More sequences than a warp has lanes, most of them short."""
    ctx = [(37 * b) % 200 - 1 for b in range(75)]
    _check(ctx, 2, 1, 2, Tmax, 64, False, 0.0, False, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("n,Tmax", [(1, 90), (1, 4000), (20, 90), (20, 4000)])
def test_nothing_active(B, n, Tmax):
    q, k, v = (x.cuda() for x in _data(B, 4, 2, n, Tmax, 64, 6))
    o, lse = fa.fwd_tree(q, k.fill_(math.nan), v.fill_(math.nan),
                         torch.full((B,), -1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [2, 16])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_depths_anywhere(H, cap):
    """Depths that put a new token in front of context keys: the bias is by distance on both sides."""
    n, ctx, Tmax, d = 5, 300, 310, 64
    q, k, v = _data(1, H, 1, n, Tmax, d, 14, 2.0)
    dep = torch.tensor([-290, -140, 0, -1, 400], dtype=torch.int32)
    tree = torch.eye(n, dtype=torch.uint8)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])
    qa = ctx + dep[None]
    ka = torch.arange(Tmax)[None].clone()
    ka[0, ctx:ctx + n] = qa[0]
    r = ref.attention(q, k, v, _seen([ctx], n, Tmax, tree[None]), d ** -0.5, cap, sl, query_at=qa, key_at=ka)
    o, lse = fa.fwd_tree(q.cuda(), k.cuda(), v.cuda(), torch.tensor([ctx], dtype=torch.int32).cuda(),
                         tree=tree.cuda(), depths=dep.cuda(), softcap=cap, slopes=sl.cuda())
    torch.cuda.synchronize()
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))


@pytest.mark.gpu
def test_rows_of_the_tree_that_see_nothing_new():
    """A tree row of zeros sees the context alone, and without a context nothing."""
    q, k, v = _data(2, 2, 2, 4, 40, 64, 9)
    tree = torch.zeros(4, 4, dtype=torch.uint8)
    tree[1, 1] = tree[3, 0] = 1
    ctx = [0, 17]
    r = ref.attention(q, k, v, _seen(ctx, 4, 40, tree.expand(2, 4, 4)), 0.125)
    for t in (tree, tree.bool()):
        o, lse = fa.fwd_tree(q.cuda(), k.cuda(), v.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                             tree=t.cuda())
        ref.check({"o": o, "lse": lse}, r, ("o", "lse"))
    assert torch.isneginf(lse[0, :, 0]).all() and not o[0, :, 0].any()


@pytest.mark.gpu
def test_chain_is_bottom_right_causal_attention():
    """A chain over an equal-length batch is what fwd_kv computes."""
    q, k, v = (x.cuda() for x in _data(2, 4, 4, 7, 333, 64, 2))
    o, lse = fa.fwd_tree(q, k, v, torch.full((2,), 326, dtype=torch.int32, device="cuda"))
    o2, lse2 = fa.fwd_kv(q, k, v)
    assert (o.float() - o2.float()).abs().max() <= 2e-2 and (lse - lse2).abs().max() <= 1e-4


@pytest.mark.gpu
def test_cache_past_32_bit_offsets():
    B, Hkv, Tmax, d = 2, 8, 1 << 20, 128              # 2³¹ elements a cache
    q, k, v = _data(B, Hkv, Hkv, 2, 300, d, 12)
    kc, vc = (torch.full((B, Hkv, Tmax, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[:, :, :300], vc[:, :, :300] = k.cuda(), v.cuda()
    ctx = [200, 298]
    o, lse = fa.fwd_tree(q.cuda(), kc, vc, torch.tensor(ctx, dtype=torch.int32).cuda())
    ref.check({"o": o, "lse": lse}, ref.attention(q, k, v, _seen(ctx, 2, 300, None), d ** -0.5),
              ("o", "lse"))


@pytest.mark.gpu
def test_serving_steps_captured_on_two_streams():
    """rope_append → fwd_tree as a server runs it: several steps of a captured graph with growing
    contexts, and the same steps on another stream with their own workspace at the same time."""
    B, H, Hkv, n, Tmax, d = 3, 8, 2, 4, 128, 64
    f = fa.rope_inv_freq(d)
    steps = 3

    class Server:
        def __init__(self, seed):
            g = torch.Generator().manual_seed(seed)
            self.x = [torch.randn(B, n, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
                      for _ in range(steps)]
            self.inp = torch.empty_like(self.x[0])
            self.kc, self.vc = (torch.full((B, Hkv, Tmax, d), math.nan, dtype=torch.bfloat16, device="cuda")
                                for _ in range(2))
            self.ctx = torch.tensor([0, 0, -100], dtype=torch.int32, device="cuda")
            self.ws = fa.fwd_tree_workspace(B, H, Hkv, n, Tmax, d)
            self.got = []

        def step(self):
            q, k, v = (self.inp[:, :, s].transpose(1, 2)
                       for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
            q = fa.rope_append(q, k, v, self.kc, self.vc, self.ctx, f)
            r = fa.fwd_tree(q, self.kc, self.vc, self.ctx, workspace=self.ws)
            self.ctx += n
            return r

        def capture(self):
            self.inp.copy_(self.x[0])
            keep = self.ctx.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step()
            torch.cuda.current_stream().wait_stream(side)
            self.ctx.copy_(keep)
            self.kc.fill_(math.nan)
            self.vc.fill_(math.nan)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self.step()
            torch.cuda.synchronize()

    servers = [Server(1), Server(2)]
    for s in servers:
        s.capture()
    streams = [torch.cuda.Stream() for _ in servers]
    for i in range(steps):
        for s, st in zip(servers, streams):
            with torch.cuda.stream(st):
                s.inp.copy_(s.x[i])
                s.graph.replay()
                s.got.append([t.clone() for t in s.out])
    torch.cuda.synchronize()
    for s in servers:
        x = torch.cat(s.x, 1).cpu()                      # every token of the run
        T = steps * n
        q, k, v = (x[:, :, a].transpose(1, 2).contiguous().cuda()
                   for a in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
        q, k = fa.rope(q, k, f)
        r = ref.attention(q.cpu(), k.cpu(), v.cpu(), ref.visible_mask(B, T, True), d ** -0.5)
        o = torch.cat([g[0] for g in s.got], 2)
        lse = torch.cat([g[1] for g in s.got], 2)
        ref.check({"o": o[:2], "lse": lse[:2]}, {a: b[:2] for a, b in r.items()}, ("o", "lse"))
        assert not o[2].any() and torch.isneginf(lse[2]).all()
        assert torch.isnan(s.kc[2].float()).all()        # the inactive sequence's cache stayed


@pytest.mark.gpu
def test_wrapper_refusals_on_device():
    q, k, v = (x.cuda() for x in _data(2, 4, 2, 3, 20, 64, 1))
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: fa.fwd_tree(q, k, v[:, :1].contiguous(), ctx),
                 lambda: fa.fwd_tree(q, k, v, ctx.long()),
                 lambda: fa.fwd_tree(q, k, v, ctx[:1]),
                 lambda: fa.fwd_tree(q, k, v, ctx.cpu()),
                 lambda: fa.fwd_tree(q, k, v, ctx, tree=torch.ones(3, 4, dtype=torch.uint8, device="cuda")),
                 lambda: fa.fwd_tree(q, k, v, ctx, tree=torch.ones(3, 3, device="cuda")),
                 lambda: fa.fwd_tree(q, k, v, ctx, depths=torch.zeros(4, dtype=torch.int32, device="cuda")),
                 lambda: fa.fwd_tree(q, k, v, ctx, slopes=torch.zeros(3, device="cuda")),
                 lambda: fa.fwd_tree(q[:, :3].contiguous(), k, v, ctx)):
        with pytest.raises(ValueError):
            call()
    q, k, v = (x.cuda() for x in _data(2, 4, 2, 3, 5000, 64, 1))
    with pytest.raises(fa.FAError):
        fa.fwd_tree(q, k, v, ctx, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert fa.fa_fwd_tree_workspace_size(2, 4, 2, 3, 20, 64) == 1
    assert fa.fa_fwd_tree_workspace_size(2, 4, 2, 3, 5000, 64) > 1
