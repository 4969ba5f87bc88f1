"""Trees and depths that a batch shares ([Tq, Tq], [Tq]) against the same ones given for each sequence, in every
kernel of new tokens with a window or over a 4-bit cache; depths below zero over the latter."""

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_cache4 import _hold, values
from tests.test_mod import _slopes
from tests.test_tree import _trees
from tests.test_window import tree_seen


def _rows(B, H, Hkv, n, Tmax, d, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, h, t, d, generator=g).to(torch.bfloat16) for h, t in ((H, n), (Hkv, Tmax), (Hkv, Tmax)))


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 6000])                   # a CTA or a cluster an entry; stretches
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("H,Hkv,n,d,bias", [
    (2, 1, 4, 64, True),      # 8 rows
    (4, 2, 8, 128, False),    # 16
    (3, 1, 8, 64, True),      # 24: the kernel of 32, or blocks of 16
    (8, 1, 9, 128, True),     # 72: the tensor-core kernel
    (4, 1, 33, 64, False),    # 132
])
def test_shared_and_own_trees(H, Hkv, n, d, bias, four, room):
    ctx = [400, 0, 77, -1, 128]
    B, Tmax, window, sinks = len(ctx), 448 + room, 60, 3
    q, k, v = _rows(B, H, Hkv, n, Tmax, d, n + d)
    tree, depths = _trees(1, n, 2)
    assert tree.shape == (1, n, n) and depths.shape == (1, n)
    many = [x.expand(B, *x.shape[1:]).contiguous().cuda() for x in (tree, depths)]
    once = [x[0].contiguous().cuda() for x in (tree, depths)]
    cache = _hold(k, v) if four else None
    kc, vc, q, at = k.cuda(), v.cuda(), q.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda()
    kw = dict(slopes=_slopes(H).cuda() if bias else None, sinks=sinks, window=window)

    def run(t, dep):
        if four:
            return fa.fwd_tree4(q, cache, at, tree=t, depths=dep, **kw)
        return fa.fwd_tree(q, kc, vc, at, tree=t, depths=dep, **kw)
    want = run(many[0], many[1])
    for t, dep in ((once[0], once[1]), (once[0], many[1]), (many[0], once[1]), (once[0].bool(), once[1])):
        got = run(t, dep)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a chain with shared depths
    got, want = run(None, once[1]), run(None, many[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 3, 20])                      # 5, 15 and 100 rows
@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("window,sinks", [(20, 4), (0, 0)])
def test_depths_below_zero_in_four_bits(H, room, window, sinks):
    """In the window's distances they count as 0; without one only the bias sees depths, as they are."""
    depths = torch.tensor([-290, 7, 0, -1, 30], dtype=torch.int32)
    ctx, n, d = [300, 40], 5, 64
    Tmax = 312 + room
    q, k, v = _rows(2, H, 1, n, Tmax, d, 8)
    ok = tree_seen(ctx, n, Tmax, None, depths.expand(2, n), window, sinks)
    sl = None if window else _slopes(H)
    qa = torch.tensor(ctx)[:, None] + depths
    ka = torch.arange(Tmax).repeat(2, 1)
    for b, c in enumerate(ctx):
        ka[b, c:c + n] = qa[b]
    r = ref.attention(q, values(k), values(v), ok, d ** -0.5, 0.0, sl, query_at=qa, key_at=ka)
    o, lse = fa.fwd_tree4(q.cuda(), _hold(k, v), torch.tensor(ctx, dtype=torch.int32).cuda(), depths=depths.cuda(),
                          slopes=None if sl is None else sl.cuda(), window=window, sinks=sinks)
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))
