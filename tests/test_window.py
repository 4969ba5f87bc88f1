"""A sliding window and sinks: training (visible, fwd_mod, bwd_mod) and serving (fwd_tree). Refusals on
the CPU, GPU parity with the 64-bit reference of mod_reference.py under its bounds."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_mod import ALL, _ids, _run, _slopes, _tensors
from tests.test_tree import _data as _tree_data, _trees

A, SZ = 0x7F0000000000, 1 << 34
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED


# ------------------------------------------------------------------------- refusals (CPU)

def test_visible_refusals():
    n = fa.fa_visible_window_size(2, 300, 50, 4)
    assert n > fa.fa_visible_size(2, 300) == fa.fa_visible_window_size(2, 300, 50, 0)
    for bad in ((0, 300, 50, 4), (2, 0, 50, 4), (2, 300, 0, 4), (2, 300, -1, 0), (2, 300, 50, -1),
                (2, 300, 50, 1025), (1, (1 << 31) - 1, 5, 1)):
        assert fa.fa_visible_window_size(*bad) == 0

    def call(ids=A, window=50, sinks=4, vis=A + 2 * SZ, nbytes=n, B=2, T=300):
        return fa.fa_visible_window(ids, window, sinks, vis, nbytes, B, T, None)
    assert call(vis=0) == BAD and call(nbytes=n - 1) == BAD and call(T=0) == BAD
    assert call(window=0) == BAD and call(sinks=-1) == BAD and call(sinks=2000) == BAD
    assert call(vis=A + 2 * SZ + 128) == MIS and call(ids=A + 2) == MIS and call(vis=A) == BAD


def _fwd(q=A, k=A + SZ, v=A + 2 * SZ, o=A + 3 * SZ, lse=A + 4 * SZ, rest=None, vis=A + 5 * SZ, window=64,
         sinks=4, cap=0.0, B=2, H=4, Hkv=2, T=300, d=64, scale=0.125):
    return fa.fa_fwd_window(q, k, v, o, lse, rest, vis, window, sinks, cap, None, B, H, Hkv, T, d, scale,
                            None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(o=0), BAD), (dict(vis=0), BAD), (dict(vis=None), BAD), (dict(window=0), BAD),
    (dict(sinks=-1), BAD), (dict(sinks=1025), BAD), (dict(Hkv=3), BAD), (dict(d=32), BAD), (dict(T=0), BAD),
    (dict(cap=-1.0), BAD), (dict(scale=math.nan), BAD), (dict(vis=A + 5 * SZ + 64), MIS),
    (dict(q=A + 8), MIS), (dict(o=A + 5 * SZ), BAD), (dict(lse=A), BAD), (dict(rest=A + 3 * SZ), BAD),
])
def test_forward_refusals(kw, want):
    assert _fwd(**kw) == want


def _bwd(q=A, k=A + SZ, v=A + 2 * SZ, o=A + 3 * SZ, do=A + 4 * SZ, lse=A + 5 * SZ, dq=A + 6 * SZ,
         dk=A + 7 * SZ, dv=A + 8 * SZ, ws=A + 9 * SZ, n=None, vis=A + 10 * SZ, window=64, sinks=4, B=2, H=4,
         Hkv=2, T=3000, d=64):
    n = fa.fa_bwd_window_workspace_size(2, 4, 2, 3000, 64, 64, 4) if n is None else n
    return fa.fa_bwd_window(q, k, v, o, do, lse, None, dq, dk, dv, ws, n, vis, window, sinks, 0.0, None, B,
                            H, Hkv, T, d, 0.125, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(do=0), BAD), (dict(ws=0), BAD), (dict(vis=None), BAD), (dict(window=0), BAD),
    (dict(sinks=2000), BAD), (dict(n=fa.fa_bwd_mod_workspace_size(2, 4, 2, 3000, 64)), BAD),
    (dict(d=96), BAD), (dict(ws=A + 9 * SZ + 16), MIS), (dict(vis=A + 10 * SZ + 8), MIS),
    (dict(dk=A + 10 * SZ), BAD), (dict(ws=A + 10 * SZ), BAD), (dict(dq=A), BAD),
])
def test_backward_refusals(kw, want):
    assert _bwd(**kw) == want


def test_workspaces():
    assert fa.fa_bwd_window_workspace_size(2, 4, 2, 3000, 64, 64, 0) == fa.fa_bwd_mod_workspace_size(2, 4, 2, 3000, 64)
    assert fa.fa_bwd_window_workspace_size(2, 4, 2, 3000, 64, 64, 4) > fa.fa_bwd_mod_workspace_size(2, 4, 2, 3000, 64)
    for bad in ((2, 4, 3, 3000, 64, 64, 4), (2, 4, 2, 3000, 64, 0, 4), (2, 4, 2, 3000, 64, 64, 1025)):
        assert fa.fa_bwd_window_workspace_size(*bad) == 0


def _tree(window=64, sinks=4, ws=A + 6 * SZ, ws_bytes=1 << 30, q=A, o=A + 3 * SZ, B=2, H=4, Hkv=2, Tq=8,
          Tmax=5000, d=64):
    return fa.fa_fwd_tree_window(q, A + SZ, A + 2 * SZ, o, A + 4 * SZ, A + 5 * SZ, None, 0, None, 0, window,
                                 sinks, 0.0, None, B, H, Hkv, Tq, Tmax, d, 0.125, ws, ws_bytes, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), BAD), (dict(window=-5), BAD), (dict(sinks=-1), BAD), (dict(q=0), BAD), (dict(d=80), BAD),
    (dict(window=4000, ws=0), BAD), (dict(window=4000, ws_bytes=64), BAD), (dict(q=A + 2), MIS),
    (dict(o=A + SZ), BAD),
])
def test_tree_refusals(kw, want):
    assert _tree(**kw) == want


def test_wrappers_reject_what_they_cannot_take():
    for kw in (dict(window=-1), dict(window=2.0), dict(sinks=3), dict(window=5, sinks=-1),
               dict(window=5, sinks=1025), dict(window=1 << 31), dict(window=5, causal=False),
               dict(window=5, prefix_len=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fa.visible(2, 300, device="cuda", **kw)
    with pytest.raises(ValueError):
        fa.fwd_tree_workspace(1, 2, 1, 1, 100, 64, device="cuda:0", sinks=3)


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_unsupported():
    none = fa.FA_ERR_UNSUPPORTED_DEVICE
    assert fa.fa_visible_window(None, 5, 1, A, 1 << 20, 1, 100, None) == none
    assert _fwd() == none and _fwd(sinks=0) == none and _bwd() == none and _bwd(sinks=0) == none
    assert _tree() == none and _tree(window=(1 << 31) - 1, sinks=(1 << 31) - 1) == none


# --------------------------------------------------------------------------- the reference

def window_mask(B, T, window, sinks, ids=None):
    """[B, T, T] by the definition, a row at a time."""
    ok = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        row = [0] * T if ids is None else ids[b].tolist()
        start = 0
        for i in range(T):
            if i and row[i] != row[i - 1]:
                start = i
            if row[i] >= 0:
                ok[b, i, max(start, i - window + 1):i + 1] = True
                ok[b, i, start:min(start + sinks, i + 1)] = True
    return ok


# ----------------------------------------------------------------------- training (GPU)

def _check(B, H, Hkv, T, d, window, sinks, cap=0.0, bias=False, lengths=None, pad=0, seed=0, with_rest=True,
           dirty=True):
    q, k, v, do = _tensors(B, H, Hkv, T, d, 29 * T + d + seed, 4.0 if cap else 1.0)
    ids = None if lengths is None else _ids(B, T, lengths, pad)
    sl = _slopes(H) if bias else None
    r = ref.attention(q, k, v, window_mask(B, T, window, sinks, ids), d ** -0.5, cap, sl, do)
    if pad and dirty:                                           # padding may hold anything
        for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, math.nan)):
            x[:, :, T - pad:] = bad
    seen = fa.visible(B, T, doc_ids=None if ids is None else ids.cuda(), window=window, sinks=sinks,
                      device="cuda")
    ref.check(_run(q, k, v, do, seen, softcap=cap, slopes=sl, with_rest=with_rest), r, ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window,sinks", [
    (1, 1, 0), (1, 5, 3), (2, 1, 1),            # one token; itself and the first
    (127, 1, 0), (129, 1, 4),                   # nothing but itself
    (300, 128, 0), (300, 129, 1), (300, 127, 4),
    (513, 100, 130),                            # sinks that reach into a second tile
    (640, 64, 600),                             # more sinks than the window
    (700, 700, 4), (700, 5000, 9),              # a window that leaves nothing out
    (1500, 33, 4),                              # the sinks' walk in pieces
])
def test_parity(T, window, sinks, d):
    _check(1, 4, 2, T, d, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (80.0, False), (0.0, True), (30.0, True), (8.0, False)])
def test_parity_with_modified_scores(cap, bias, d):
    _check(2, 4, 1, 420, d, 150, 5, cap, bias)
    _check(1, 3, 3, 260, d, 70, 0, cap, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,T,d,window,sinks,cap,bias,lengths,pad", [
    (2, 4, 2, 300, 64, 40, 4, 0.0, False, (1, 100, 27), 40),
    (2, 2, 1, 1300, 128, 50, 3, 0.0, False, (1200, 5, 90), 60),    # pieces of a document among others
    (1, 4, 4, 1000, 64, 200, 16, 30.0, True, (333, 128, 500), 33),
    (3, 2, 2, 520, 128, 16, 130, 20.0, False, (129, 3, 260), 0),
    (1, 8, 2, 2000, 64, 64, 300, 0.0, True, (1900,), 50),
])
def test_parity_with_documents(B, H, Hkv, T, d, window, sinks, cap, bias, lengths, pad):
    _check(B, H, Hkv, T, d, window, sinks, cap, bias, lengths, pad)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,window,sinks,cap,lengths,pad,with_rest", [
    (400, 64, 100, 4, 0.0, None, 0, True),
    (400, 128, 100, 4, 0.0, None, 0, False),
    (517, 64, 130, 4, 30.0, None, 0, False),
    (517, 128, 40, 200, 30.0, None, 0, True),
    (384, 64, 60, 3, 8.0, (300, 9), 70, True),                  # far scores, documents, padding
    (384, 128, 60, 3, 0.0, (130, 254), 0, True),
    (300, 64, 70, 0, 0.0, None, 0, False),
])
def test_parity_with_many_heads(T, d, window, sinks, cap, lengths, pad, with_rest):
    """320 heads: two query tiles a CTA, with sinks of their own each."""
    _check(4, 80, 10, T, d, window, sinks, cap, False, lengths, pad, with_rest=with_rest)


@pytest.mark.gpu
@pytest.mark.parametrize("d,cap,lengths", [(64, 0.0, None), (64, 30.0, (900, 200)), (128, 0.0, (1000, 3))])
def test_parity_of_wider_windows_with_many_heads(d, cap, lengths):
    """Two query tiles a CTA at either head dim, whose sinks lie in tiles before both walks."""
    _check(1, 80, 10, 1100, d, 600, 4, cap, False, lengths, 11 if lengths else 0)


@pytest.mark.gpu
def test_a_window_over_everything_is_causal_attention():
    q, k, v, do = _tensors(2, 4, 2, 500, 64, 8)
    wide = fa.visible(2, 500, window=500, sinks=4, device="cuda")
    a, b = _run(q, k, v, do, wide), _run(q, k, v, do)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("T,lengths,window,sinks", [
    (4097, (700, 1, 2048), 300, 4), (16384, (128,), 64, 1), (32768, (30000, 5), 1024, 130),  # in clusters
    (33000, (1000, 1, 2048), 300, 4), (150001, (100000, 333), 2000, 9), (140000, (139000,), 64, 1)])
def test_visible_rows(T, lengths, window, sinks):
    """Every row's two intervals, every walk's records: each visible pair lies in a tile of its query
    tile's walk and of its key tile's pieces, which cover their query tiles once."""
    B = 2
    ids = _ids(B, T, lengths, 7)
    seen = fa.visible(B, T, doc_ids=ids.cuda(), window=window, sinks=sinks)
    n_t = -(-T // 128)
    up = lambda x: -(-x // 256) * 256
    first = torch.cat((torch.ones(B, 1, dtype=torch.bool), ids[:, 1:] != ids[:, :-1]), 1)
    at = torch.arange(T).expand(B, T)
    start = torch.where(first, at, torch.zeros_like(at)).cummax(1).values
    lo = torch.maximum(start, at - window + 1)
    live = (ids >= 0)[..., None]
    want = torch.stack((lo, at + 1), -1) * live
    sink = torch.stack((start, torch.minimum(start + sinks, lo)), -1) * (live & (lo > start)[..., None])
    buf = seen.buffer.cpu()
    take = lambda off, *shape: buf[off:off + 4 * math.prod(shape)].view(torch.int32).view(shape).long()
    rows = take(0, B, n_t * 128, 2)
    assert torch.equal(rows[:, :T], want) and not rows[:, T:].any()
    piece = max(8, min(window, T) // 128 + 2)
    extra = -(-n_t * ((sinks + 126) // 128 + 1) * 8 // (7 * piece))
    off = fa.fa_visible_size(B, T)
    srows = take(off, B, n_t * 128, 2)
    assert torch.equal(srows[:, :T], sink) and not srows[:, T:].any()
    off += up(B * n_t * 128 * 8) + up(B * n_t * 8) + up(B * ((n_t + 1) // 2) * 16)
    rec = take(off, B, n_t + extra, 2, 4)
    for b in range(B):
        # the last query that sees a key: the document's last, or the window's
        nxt = torch.where(first[b], at[b], torch.full_like(at[b], T))
        end = torch.cat((nxt[1:], torch.tensor([T]))).flip(0).cummin(0).values.flip(0)
        last = torch.where(at[b] - start[b] < sinks, end - 1, torch.minimum(end - 1, at[b] + window - 1))
        far = torch.zeros(n_t, dtype=torch.int64)
        far.scatter_reduce_(0, at[b][ids[b] >= 0] // 128, last[ids[b] >= 0] // 128 + 1, "amax")
        walks = {}
        for (t, f, l, _), (slot, _, _, _) in rec[b].tolist():
            if t < n_t and l > f:
                walks.setdefault(t, []).append((f, l, slot))
        slots = []
        for t in range(n_t):
            w = sorted(walks.get(t, []))
            if far[t] == 0:
                assert not w
                continue
            assert w[0][0] <= t and w[-1][1] == far[t] and all(x[1] == y[0] for x, y in zip(w, w[1:]))
            assert all(x[1] - x[0] <= max(piece, 1) for x in w)
            assert (len(w) == 1) == (w[0][2] < 0)
            slots += [x[2] for x in w if x[2] >= 0]
        assert sorted(slots) == list(range(len(slots))) and len(slots) <= extra + min(extra, n_t)


@pytest.mark.gpu
def test_gradients_of_sinks_are_the_same_every_time():
    """dK and dV of sinks, summed over pieces and over parts of shared heads, bit for bit."""
    q, k, v, do = _tensors(1, 8, 2, 3000, 128, 5)
    seen = fa.visible(1, 3000, window=100, sinks=4, device="cuda")
    a, b = _run(q, k, v, do, seen), _run(q, k, v, do, seen)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
def test_workspaces_and_buffers_of_the_callers():
    q, k, v, do = (x.cuda() for x in _tensors(1, 4, 2, 1200, 64, 6))
    seen = fa.visible(1, 1200, window=80, sinks=4, device="cuda")
    o, lse = fa.fwd_mod(q, k, v, visible=seen)
    with pytest.raises(fa.FAError):
        fa.bwd_mod(q, k, v, o, lse, do, visible=seen, workspace=fa.bwd_mod_workspace(1, 4, 2, 1200, 64))
    ws = fa.bwd_mod_workspace(1, 4, 2, 1200, 64, window=80, sinks=4).fill_(255)   # NaN: contents are immaterial
    a = fa.bwd_mod(q, k, v, o, lse, do, visible=seen, workspace=ws)
    b = fa.bwd_mod(q, k, v, o, lse, do, visible=seen)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    again = fa.visible(1, 1200, window=80, sinks=4, buffer=seen.buffer)
    assert again.buffer is seen.buffer
    with pytest.raises(fa.FAError):
        fa.visible(1, 1200, window=80, sinks=4, buffer=torch.empty(fa.fa_visible_size(1, 1200), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.fwd_mod(q, k, v, visible=seen, causal=False)


@pytest.mark.gpu
def test_a_training_step_as_it_is_used():
    """norm_rope, the forward, the backward and norm_rope_bwd on packed documents, captured and replayed,
    against the 64-bit chain of the same functions on what each of them was given."""
    B, H, Hkv, T, d, window, sinks = 2, 4, 2, 700, 64, 120, 4
    g = torch.Generator().manual_seed(2)
    packed = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    do = torch.randn(B, H, T, d, generator=g).to(torch.bfloat16).cuda()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    ids = _ids(B, T, (300, 90, 17), 20)
    ids_gpu, f = ids.cuda(), fa.rope_inv_freq(d)

    def step():
        q, k, v = (packed[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
        seen = fa.visible(B, T, doc_ids=ids_gpu, window=window, sinks=sinks)
        tq, tk = fa.norm_rope(q, k, wq, wk, f)
        v = v.contiguous()
        rest = torch.empty_like(tq)
        o, lse = fa.fwd_mod(tq, tk, v, visible=seen, rest=rest)
        gq, gk, dv = fa.bwd_mod(tq, tk, v, o, lse, do, visible=seen, rest=rest)
        dq, dk, dwq, dwk = fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f)
        return dict(tq=tq, tk=tk, v=v, o=o, lse=lse, gq=gq, gk=gk, dv=dv, dq=dq, dk=dk, dwq=dwq, dwk=dwk)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    packed.copy_(torch.randn(packed.shape, generator=g).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    r = ref.attention(held["tq"].cpu(), held["tk"].cpu(), held["v"].cpu(),
                      window_mask(B, T, window, sinks, ids), d ** -0.5, do=do.cpu())
    got = dict(o=held["o"], lse=held["lse"], dq=held["gq"], dk=held["gk"], dv=held["dv"])
    ref.check(got, r, ALL)
    from tests.test_norm import EPS, _backward, _forward, _near
    pos = torch.arange(T).expand(B, T)
    for x, w, t, gr, dx in ((packed[:, :, :H], wq, "tq", "gq", "dq"), (packed[:, :, H:H + Hkv], wk, "tk", "gk", "dk")):
        x = x.transpose(1, 2)
        _near(held[t], _forward(x, w, pos, f, False, 1.0, EPS), t)
        rows, weight = _backward(held[gr], x, w, pos, f, False, 1.0, EPS)
        _near(held[dx], rows, dx)
        _near(held["dw" + dx[1]], weight, "dw")


# ------------------------------------------------------------------------- serving (GPU)

def tree_seen(ctx, n, Tmax, tree, depths, window, sinks):
    """([B, n, Tmax] visible rows) by the definition."""
    B = len(ctx)
    ok = torch.zeros(B, n, Tmax, dtype=torch.bool)
    for b, c in enumerate(ctx):
        if c < 0:
            continue
        for t in range(n):
            at = c + (t if depths is None else max(0, int(depths[b, t])))
            for j in range(Tmax):
                if j < c:
                    seen, place = True, j
                elif j < c + n:
                    s = j - c
                    seen = s <= t if tree is None else bool(tree[b, t, s])
                    place = c + (s if depths is None else max(0, int(depths[b, s])))
                else:
                    break
                ok[b, t, j] = seen and (not window or at - place < window or place < sinks)
    return ok


def _check_tree(ctx, H, Hkv, n, Tmax, d, window, sinks, tree=False, cap=0.0, bias=False, seed=0, depths=None,
                call=None):
    B = len(ctx)
    q, k, v = _tree_data(B, H, Hkv, n, Tmax, d, seed + Tmax + n, 4.0 if cap else 1.0)
    t, dep = _trees(B, n, seed) if tree else (None, depths)
    sl = _slopes(H) if bias else None
    qa = torch.tensor(ctx)[:, None] + (torch.arange(n) if dep is None else dep)
    ka = torch.arange(Tmax).repeat(B, 1)
    for b, c in enumerate(ctx):
        m = max(0, min(n, Tmax - c)) if c >= 0 else 0
        if m:
            ka[b, c:c + m] = qa[b, :m]
    ok = tree_seen(ctx, n, Tmax, t, dep, window, sinks)
    r = ref.attention(q, k, v, ok, d ** -0.5, cap, sl, query_at=qa, key_at=ka)
    kc, vc = k.clone(), v.clone()
    for b, c in enumerate(ctx):     # what no token can see, behind and between, holds anything
        kc[b, :, max(0, c + n) if c >= 0 else 0:] = math.nan
        vc[b, :, max(0, c + n) if c >= 0 else 0:] = math.nan
        if c >= 0:
            kc[b, :, sinks:max(sinks, c - window + 1)] = math.nan
            vc[b, :, sinks:max(sinks, c - window + 1)] = math.inf
    o, lse = fa.fwd_tree(q.cuda(), kc.cuda(), vc.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                         tree=None if t is None else t.cuda(), depths=None if dep is None else dep.cuda(),
                         softcap=cap, slopes=None if sl is None else sl.cuda(), window=window, sinks=sinks)
    torch.cuda.synchronize()
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))


# room: longer caches have their work shared out in stretches, shorter ones a CTA an entry
@pytest.mark.gpu
@pytest.mark.parametrize("ctx,H,Hkv,n,Tmax,d,window,sinks,tree,cap,bias", [
    ([0], 1, 1, 1, 1, 64, 1, 0, False, 0.0, False),
    ([5, 0, -1], 2, 2, 1, 6, 128, 1, 2, False, 0.0, False),
    ([1000, 63, 64, 400], 4, 4, 1, 1100, 64, 64, 4, False, 30.0, False),
    ([1000, 129, 700], 16, 1, 1, 1024, 128, 100, 0, False, 50.0, True),
    ([900, 300], 6, 2, 5, 920, 64, 130, 70, True, 0.0, False),
    ([300, 77, 500], 4, 2, 16, 520, 128, 40, 3, True, 0.0, True),
    ([511, 100], 16, 4, 16, 600, 64, 128, 5, True, 5.0, False),       # 64 rows
    ([90, 400], 5, 5, 33, 450, 128, 8, 2, False, 0.0, True),          # a chain longer than its window
    ([40, 1200], 8, 2, 30, 1300, 64, 12, 50, False, 0.0, False),      # the same, 120 rows
    ([400, 3], 8, 1, 64, 500, 128, 6, 10, True, 20.0, True),          # deep trees, 512 rows
    ([1500, 10], 4, 1, 64, 1600, 64, 300, 4, True, 0.0, False),
    ([100, 95, 120], 2, 1, 4, 100, 64, 30, 4, False, 0.0, False),     # full caches, drafts outside
    ([500, 300], 2, 1, 4, 100, 64, 30, 4, False, 0.0, False),         # contexts far past the cache: sinks alone
    ([500, 300], 2, 1, 4, 100, 64, 30, 0, False, 0.0, False),         # nothing
    ([700, 20], 4, 2, 3, 720, 64, 5000, 100, False, 0.0, False),      # a window over everything
])
@pytest.mark.parametrize("room", [0, 6000])
def test_tree_parity(ctx, H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, room):
    if room and max(ctx) > Tmax:
        room = 0                                             # (they are about the cache's end)
    _check_tree(ctx, H, Hkv, n, Tmax + room, d, window, sinks, tree, cap, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [2, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts_in_many_stretches(H, d):
    _check_tree([40000, 123, 9000, 0, 21111], H, 1, 3, 40100, d, 6000, 300, True, seed=3)


# Entries taken by clusters of 8, 6, 4, 3 and 2 CTAs, which need no workspace, with contexts that leave some of a
# cluster without a chunk or all of it, and long windows that go in stretches.
@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,n,Tmax,d,window,sinks,tree,cap,bias,whole", [
    (4, 4, 4, 1, 1200, 64, 1100, 3, False, 0.0, False, True),        # 16 entries
    (4, 16, 2, 4, 1200, 64, 700, 130, True, 0.0, True, True),        # 8, of 32 rows
    (5, 8, 1, 4, 900, 128, 800, 0, True, 30.0, False, True),
    (15, 4, 4, 1, 700, 64, 600, 4, False, 30.0, True, True),         # 60
    (20, 6, 3, 3, 600, 128, 300, 4, True, 0.0, False, True),
    (75, 2, 2, 1, 400, 64, 300, 1, False, 0.0, False, True),         # 150
    (66, 8, 2, 1, 500, 128, 300, 4, False, 0.0, True, True),
    (20, 4, 4, 1, 700, 64, 600, 4, False, 0.0, True, True),          # 80, by fours
    (26, 6, 3, 3, 700, 128, 600, 4, True, 30.0, False, True),        # 78, by threes
    (2, 16, 4, 16, 2600, 128, 2400, 4, True, 0.0, True, True),       # of 64 rows
    (4, 16, 4, 13, 1600, 128, 1400, 200, False, 30.0, False, True),  # 16, by sixes
    (10, 12, 4, 12, 1500, 64, 1300, 4, True, 80.0, False, True),     # 40, by threes
    (16, 16, 4, 20, 1200, 64, 1100, 4, True, 30.0, False, True),     # 64, by twos
    (1, 12, 1, 50, 2200, 64, 2000, 0, False, 30.0, True, True),      # 600 rows
    (2, 9, 1, 16, 2200, 128, 2000, 1, False, 0.0, False, True),
    (3, 4, 4, 1, 9000, 64, 8000, 4, False, 0.0, False, False),
    (3, 4, 2, 8, 9000, 128, 7000, 4, True, 0.0, False, False),
    (1, 8, 1, 16, 18000, 64, 16000, 4, False, 0.0, False, False),
])
def test_clusters(B, H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, whole):
    assert (fa.fa_fwd_tree_window_workspace_size(B, H, Hkv, n, Tmax, d, window, sinks) == 1) == whole
    ctx = [Tmax - n, -1, 0, 65, Tmax // 2, 130, Tmax, 1] * 10
    _check_tree(ctx[:B], H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, seed=B)


@pytest.mark.gpu
@pytest.mark.parametrize("Tmax", [210, 5000])
def test_many_sequences(Tmax):
    ctx = [(37 * b) % 200 - 1 for b in range(75)]
    _check_tree(ctx, 2, 1, 2, Tmax, 64, 50, 3, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [2, 20])
def test_depths_below_zero_count_as_zero(H):
    dep = torch.tensor([[-290, 7, 0, -1, 30]], dtype=torch.int32)
    _check_tree([300], H, 1, 5, 310, 64, 20, 4, depths=dep)


@pytest.mark.gpu
def test_window_into_a_cache_past_32_bit_offsets():
    B, Hkv, Tmax, d = 2, 8, 1 << 20, 128              # 2³¹ elements a cache
    kc, vc = (torch.full((B, Hkv, Tmax, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = _tree_data(B, Hkv, Hkv, 2, 104, d, 12)
    for c, x in ((kc, k), (vc, v)):
        c[:, :, :4] = x[:, :, :4].cuda()
        c[:, :, Tmax - 100:] = x[:, :, 4:].cuda()
    ctx = [Tmax - 2, Tmax - 30]
    o, lse = fa.fwd_tree(q.cuda(), kc, vc, torch.tensor(ctx, dtype=torch.int32).cuda(), window=60, sinks=4)
    ok = torch.zeros(B, 2, 104, dtype=torch.bool)
    for b, c in enumerate(ctx):
        for t in range(2):
            ok[b, t, :4] = True
            ok[b, t, c + t - 59 - Tmax + 104:c + t + 1 - Tmax + 104] = True
    ref.check({"o": o, "lse": lse}, ref.attention(q, k, v, ok, d ** -0.5), ("o", "lse"))


@pytest.mark.gpu
def test_serving_steps_with_a_window():
    """norm_rope_append → fwd_tree as a server runs it, step by step past the window, against one causal
    pass over all tokens with the same window."""
    B, H, Hkv, n, d, window, sinks, steps = 2, 8, 2, 3, 64, 20, 4, 12
    T = n * steps
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    f = fa.rope_inv_freq(d)
    kc, vc = (torch.full((B, Hkv, 64, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    outs, lses = [], []
    for i in range(steps):
        new = x[:, i * n:(i + 1) * n]
        q, k, v = (new[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
        q = fa.norm_rope_append(q, k, v, wq, wk, kc, vc, ctx, f)
        o, lse = fa.fwd_tree(q, kc, vc, ctx, window=window, sinks=sinks)
        outs.append(o)
        lses.append(lse)
        ctx += n
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    q, k = fa.norm_rope(q, k, wq, wk, f)
    r = ref.attention(q.cpu(), k.cpu(), v.cpu(), window_mask(B, T, window, sinks), d ** -0.5)
    ref.check({"o": torch.cat(outs, 2), "lse": torch.cat(lses, 2)}, r, ("o", "lse"))
