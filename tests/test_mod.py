"""Attention with modified scores (visible, fwd_mod, bwd_mod): refusals on the CPU, the reference's
own gradients against differences, and GPU parity against the 64-bit reference under the derived
bounds of mod_reference.py."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref

A, SZ = 0x7F0000000000, 1 << 32  # fake, never-dereferenced device addresses
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED


# ------------------------------------------------------------------------- refusals (CPU)

def _fwd(q=A, k=A + SZ, v=A + 2 * SZ, o=A + 3 * SZ, lse=A + 4 * SZ, rest=None, vis=None, causal=1, cap=0.0,
         slopes=None, B=2, H=4, Hkv=2, T=200, d=64, scale=0.125):
    return fa.fa_fwd_mod(q, k, v, o, lse, rest, vis, causal, cap, slopes, B, H, Hkv, T, d, scale, None, 0,
                         None)


def _bwd(q=A, k=A + SZ, v=A + 2 * SZ, o=A + 3 * SZ, do=A + 4 * SZ, lse=A + 5 * SZ, rest=None, dq=A + 6 * SZ,
         dk=A + 7 * SZ, dv=A + 8 * SZ, ws=A + 9 * SZ, ws_bytes=None, vis=None, causal=1, cap=0.0,
         slopes=None, B=2, H=4, Hkv=2, T=200, d=64, scale=0.125):
    if ws_bytes is None:
        ws_bytes = fa.fa_bwd_mod_workspace_size(B, H, Hkv, T, d) or 1 << 20
    return fa.fa_bwd_mod(q, k, v, o, do, lse, rest, dq, dk, dv, ws, ws_bytes, vis, causal, cap, slopes, B,
                         H, Hkv, T, d, scale, None, 0, None)


COMMON = [
    (dict(q=0), BAD), (dict(v=0), BAD), (dict(lse=0), BAD), (dict(T=0), BAD), (dict(B=0), BAD),
    (dict(Hkv=0), BAD), (dict(Hkv=3), BAD), (dict(Hkv=8), BAD), (dict(d=96), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=3e38), BAD), (dict(cap=-1.0), BAD),
    (dict(cap=math.nan), BAD), (dict(cap=math.inf), BAD), (dict(cap=1e-42), BAD),
    (dict(T=(1 << 31) - 1), BAD), (dict(B=1 << 20, H=1 << 11, Hkv=1), BAD),
    (dict(q=A + 8), MIS), (dict(vis=A + 20 * SZ + 16), MIS), (dict(slopes=A + 20 * SZ + 2), MIS),
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(o=0), BAD), (dict(o=A), BAD), (dict(o=A + SZ), BAD), (dict(lse=A + 3 * SZ), BAD),
    (dict(vis=A + 3 * SZ), BAD),       # o would overwrite the visibility
    (dict(slopes=A + 4 * SZ), BAD),    # lse would overwrite the slopes
    (dict(rest=A + 3 * SZ), BAD), (dict(rest=A), BAD), (dict(rest=A + 20 * SZ + 8), MIS),
])
def test_fwd_mod_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(do=0), BAD), (dict(dk=0), BAD), (dict(ws=0), BAD), (dict(ws_bytes=4096), BAD),
    (dict(dq=A), BAD), (dict(dk=A + 8 * SZ), BAD), (dict(ws=A + 5 * SZ), BAD),
    (dict(ws=A + 9 * SZ + 16), MIS), (dict(dv=A + 8 * SZ + 8), MIS), (dict(vis=A + 7 * SZ), BAD),
    (dict(rest=A + 6 * SZ), BAD), (dict(rest=A + 20 * SZ + 4), MIS),
])
def test_bwd_mod_refusals(kw, want):
    assert _bwd(**kw) == want


def test_visible_refusals():
    n = fa.fa_visible_size(2, 300)
    assert n > 0
    for bad in ((0, 5), (2, 0), (1, (1 << 31) - 1), (1 << 30, 1 << 20)):
        assert fa.fa_visible_size(*bad) == 0

    def call(ids=A, pre=A + SZ, vis=A + 2 * SZ, nbytes=n, B=2, T=300):
        return fa.fa_visible(ids, pre, 0, 1, vis, nbytes, B, T, None)
    assert call(vis=0) == BAD and call(nbytes=n - 1) == BAD and call(T=0) == BAD
    assert call(vis=A + 2 * SZ + 128) == MIS and call(ids=A + 2) == MIS and call(pre=A + SZ + 1) == MIS
    assert call(vis=A) == BAD and call(vis=A + SZ) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_unsupported():
    assert _fwd(cap=30.0, slopes=A + 20 * SZ) == fa.FA_ERR_UNSUPPORTED_DEVICE
    assert _bwd(cap=30.0, vis=A + 21 * SZ) == fa.FA_ERR_UNSUPPORTED_DEVICE
    assert fa.fa_visible(None, None, 0, 1, A, 1 << 20, 1, 100, None) == fa.FA_ERR_UNSUPPORTED_DEVICE


def test_bwd_workspace():
    """The backward's own, and, where a key head's query heads are cut into parts, their sums."""
    assert fa.fa_bwd_mod_workspace_size(4, 12, 12, 2048, 64) == fa.fa_bwd_workspace_size(4, 12, 2048, 64)
    assert fa.fa_bwd_mod_workspace_size(1, 12, 12, 128, 64) == fa.fa_bwd_workspace_size(1, 12, 128, 64)
    assert fa.fa_bwd_mod_workspace_size(1, 12, 4, 128, 128) == \
        fa.fa_bwd_workspace_size(1, 12, 128, 128) + 2 * 3 * 4 * 128 * 128 * 4
    for bad in ((0, 4, 2, 128, 64), (1, 4, 3, 128, 64), (1, 4, 2, 0, 64), (1, 4, 2, 128, 80)):
        assert fa.fa_bwd_mod_workspace_size(*bad) == 0


def test_wrappers_reject_cpu_tensors():
    x = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fwd_mod(x, x, x)
    with pytest.raises(ValueError):
        fa.bwd_mod(x, x, x, x, torch.zeros(1, 1, 8), x)
    with pytest.raises(ValueError):
        fa.visible(1, 8, device="cpu")


def test_reference_gradients_against_differences():
    """The reference's gradient formulas against central differences of its own forward."""
    g = torch.Generator().manual_seed(5)
    B, H, Hkv, T, d = 1, 4, 2, 9, 64
    q, k, v, do = (torch.randn(B, n, T, d, generator=g, dtype=torch.float64)
                   for n in (H, Hkv, Hkv, H))
    ids = torch.tensor([[0, 0, 0, 0, 4, 4, 4, -1, -1]])
    ok = ref.visible_mask(B, T, True, ids, torch.tensor([2]))
    sl = torch.tensor([0.5, 0.25, 0.125, 0.0])
    kw = dict(scale=0.125, softcap=2.0, slopes=sl)
    r = ref.attention(q, k, v, ok, do=do, **kw)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        step = torch.randn(x.shape, generator=g, dtype=torch.float64)
        at = {"dq": 0, "dk": 1, "dv": 2}[name]
        def loss(e):
            args = [q, k, v]
            args[at] = args[at] + e * step
            return float((ref.attention(*args, ok, **kw)["o"] * do).sum())
        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs(slope - float((r[name] * step).sum())) <= 1e-6 * (1 + abs(slope))


# ---------------------------------------------------------------------------- parity (GPU)

def _tensors(B, H, Hkv, T, d, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda n, s=1.0: (torch.randn(B, n, T, d, generator=g) * s).to(torch.bfloat16)
    return mk(H, std), mk(Hkv), mk(Hkv), mk(H)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def _run(q, k, v, do, seen=None, **kw):
    t = [x.cuda() for x in (q, k, v, do)]
    sl = kw.pop("slopes", None)
    sl = None if sl is None else sl.cuda()
    rest = torch.full_like(t[0], math.nan) if kw.pop("with_rest", True) else None
    o, lse = fa.fwd_mod(*t[:3], visible=seen, slopes=sl, rest=rest, **kw)
    dq, dk, dv = fa.bwd_mod(*t[:3], o, lse, t[3], visible=seen, slopes=sl, rest=rest, **kw)
    torch.cuda.synchronize()
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


ALL = ("o", "lse", "dq", "dk", "dv")


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,T,d,causal,cap,bias", [
    (1, 1, 1, 1, 64, True, 0.0, False),        # one token
    (1, 2, 1, 2, 128, False, 20.0, True),
    (2, 3, 3, 127, 64, True, 30.0, False),     # one short of a tile
    (1, 4, 2, 128, 128, True, 0.0, True),
    (1, 4, 1, 129, 64, True, 5.0, True),       # one over; a cap that bends every score
    (2, 5, 5, 300, 64, False, 0.0, True),
    (1, 6, 2, 513, 128, True, 50.0, False),
    (1, 8, 1, 640, 64, True, 0.0, False),      # eight query heads on one key head
    (1, 4, 4, 1000, 128, False, 15.0, False),
    (3, 2, 1, 65, 128, True, 30.0, True),
])
def test_parity_without_visible(B, H, Hkv, T, d, causal, cap, bias):
    q, k, v, do = _tensors(B, H, Hkv, T, d, 11 * T + d, 4.0 if cap else 1.0)
    sl = _slopes(H) if bias else None
    ok = ref.visible_mask(B, T, causal)
    r = ref.attention(q, k, v, ok, d ** -0.5, cap, sl, do)
    ref.check(_run(q, k, v, do, causal=causal, softcap=cap, slopes=sl), r, ALL)


def _ids(B, T, lengths, pad):
    """Documents of the given lengths in turn, the last `pad` tokens padding; sequences start at
    different places of the list."""
    rows = []
    for b in range(B):
        row, n = [], b
        while len(row) < T - pad:
            row += [n % 7] * lengths[n % len(lengths)]
            n += 1
        rows.append(row[:T - pad] + [-1] * pad)
    return torch.tensor(rows, dtype=torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,T,d,causal,cap,bias,lengths,pad,prefix", [
    (1, 2, 2, 5, 64, True, 0.0, False, (1, 2), 1, None),
    (2, 4, 2, 256, 64, True, 0.0, True, (128,), 0, None),        # documents end with tiles
    (2, 4, 1, 300, 128, True, 30.0, False, (1, 100, 27), 40, None),
    (3, 2, 2, 700, 64, False, 0.0, False, (300, 129, 3), 190, None),   # a whole padded tile
    (1, 4, 4, 777, 128, False, 20.0, True, (250, 64), 5, None),
    (2, 2, 1, 400, 64, True, 0.0, False, (400,), 0, "b"),
    (2, 3, 3, 513, 128, True, 0.0, True, (200, 313), 13, "b"),
    (2, 4, 2, 600, 64, True, 10.0, False, (90, 210, 17), 33, "t"),
])
def test_parity_with_visible(B, H, Hkv, T, d, causal, cap, bias, lengths, pad, prefix):
    q, k, v, do = _tensors(B, H, Hkv, T, d, 13 * T + d, 4.0 if cap else 1.0)
    ids = _ids(B, T, lengths, pad)
    pre = None
    if prefix == "b":
        pre = torch.tensor([60 * b + 7 for b in range(B)], dtype=torch.int32)
    elif prefix == "t":
        pre = ((ids + 2) * 23 - 40).to(torch.int32)               # some of them negative
    sl = _slopes(H) if bias else None
    ok = ref.visible_mask(B, T, causal, ids, pre)
    r = ref.attention(q, k, v, ok, d ** -0.5, cap, sl, do)
    seen = fa.visible(B, T, causal=causal, doc_ids=ids.cuda(),
                      prefix_len=None if pre is None else pre.cuda())
    ref.check(_run(q, k, v, do, seen, softcap=cap, slopes=sl), r, ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,causal,cap,lengths,pad,prefix,with_rest", [
    (300, 64, True, 0.0, None, 0, None, True),
    (290, 128, False, 0.0, None, 0, None, False),
    (257, 64, True, 20.0, None, 0, None, False),               # far and near scores
    (300, 128, True, 20.0, None, 0, None, True),
    (300, 64, True, 50.0, (100, 1, 47), 30, "b", True),
    (384, 128, True, 50.0, (300, 9), 140, None, False),        # a pair whose second tile sees nothing
    (300, 64, False, 0.0, (129, 3), 17, None, True),
    (280, 128, True, 0.0, (30, 128, 60), 0, "t", False),
])
def test_parity_with_many_heads(T, d, causal, cap, lengths, pad, prefix, with_rest):
    """320 heads: two query tiles a CTA (documents, prefixes, caps of up to 60)."""
    B, H, Hkv = 4, 80, 10
    q, k, v, do = _tensors(B, H, Hkv, T, d, 19 * T + d, 4.0 if cap else 1.0)
    ids = None if lengths is None else _ids(B, T, lengths, pad)
    pre = None
    if prefix == "b":
        pre = torch.tensor([60 * b + 7 for b in range(B)], dtype=torch.int32)
    elif prefix == "t":
        pre = ((ids + 2) * 23 - 40).to(torch.int32)
    ok = ref.visible_mask(B, T, causal, ids, pre)
    r = ref.attention(q, k, v, ok, d ** -0.5, cap, None, do)
    seen = None
    if ids is not None:
        seen = fa.visible(B, T, causal=causal, doc_ids=ids.cuda(),
                          prefix_len=None if pre is None else pre.cuda())
        if pad:                                                # padding may hold anything
            for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, math.nan)):
                x[:, :, T - pad:] = bad
    ref.check(_run(q, k, v, do, seen, softcap=cap, causal=causal, with_rest=with_rest), r, ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,std,with_rest", [(30.0, 9.0, False), (30.0, 9.0, True), (8.0, 3.0, False),
                                               (60.0, 40.0, True)])
def test_parity_with_many_heads_and_far_scores(d, cap, std, with_rest):
    """Scores on both sides of the polynomial's range, in the forms of the two-tile kernel."""
    B, H, Hkv, T = 4, 80, 80, 260
    q, k, v, do = _tensors(B, H, Hkv, T, d, 23 * d + int(cap), std)
    r = ref.attention(q, k, v, ref.visible_mask(B, T, True), d ** -0.5, cap, None, do)
    ref.check(_run(q, k, v, do, None, softcap=cap, with_rest=with_rest), r, ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("T,lengths,pad,causal,prefix", [
    (1, (1,), 0, True, None), (31, (4, 9), 3, True, "b"), (1000, (128, 77), 0, False, None),
    (33000, (1000, 1, 2048), 129, True, "t"), (70001, (50000, 333), 7, True, "b"),
    (200000, (100, 60000, 17), 5000, True, None),
])
def test_visible_rows(T, lengths, pad, causal, prefix):
    """Every row's interval, at lengths where a thread holds one row to several hundred."""
    B = 2
    ids = _ids(B, T, lengths, pad)
    first = torch.cat((torch.ones(B, 1, dtype=torch.bool), ids[:, 1:] != ids[:, :-1]), 1)
    at = torch.arange(T).expand(B, T)
    lo = torch.where(first, at, torch.zeros_like(at)).cummax(1).values
    nxt = torch.where(first, at, torch.full_like(at, T))
    end = torch.cat((nxt[:, 1:], torch.full((B, 1), T)), 1).flip(1).cummin(1).values.flip(1)
    pre = None
    if prefix == "b":
        pre = torch.tensor([5, 40000][:B], dtype=torch.int32)
    elif prefix == "t":
        pre = ((ids + 2) * 23 - 40).to(torch.int32)
    hi = end
    if causal:
        n = torch.zeros_like(at) if pre is None else (pre.long()[:, None] if pre.dim() == 1 else pre.long())
        hi = torch.maximum(at + 1, torch.minimum(end, lo + n.clamp(min=0)))
    want = torch.stack((lo, hi), -1) * (ids >= 0)[..., None]
    seen = fa.visible(B, T, causal=causal, doc_ids=ids.cuda(),
                      prefix_len=None if pre is None else pre.cuda())
    T_pad = -(-T // 128) * 128
    rows = seen.buffer[:B * T_pad * 8].view(torch.int32).view(B, T_pad, 2).cpu().long()
    assert torch.equal(rows[:, :T], want) and not rows[:, T:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap", [(0.0, 0.0), (0.0, 30.0), (-0.125, 0.0), (-0.125, 8.0),
                                       (0.125, 1e6)])
def test_scales_and_caps(scale, cap):
    """Uniform and reversed preferences, and a cap so large that it must change nothing."""
    q, k, v, do = _tensors(1, 2, 1, 260, 64, 3, 3.0)
    ok = ref.visible_mask(1, 260, True)
    r = ref.attention(q, k, v, ok, scale, cap, None, do)
    if cap > 1e5:  # a relative error, not one of the cap: the polynomial's 1e-6 and rounding
        r["lse_tol"] = r["lse_tol"] - cap * 2.0 ** -20
    ref.check(_run(q, k, v, do, scale=scale, softcap=cap), r, ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("d,cap", [(64, 0.0), (128, 30.0)])
def test_padding_may_hold_anything(d, cap):
    """NaN and infinities in padded rows of every input change nothing elsewhere; padded rows get
    o = 0, lse = −inf and no gradient."""
    B, H, Hkv, T, pad = 2, 4, 2, 300, 77
    q, k, v, do = _tensors(B, H, Hkv, T, d, 9)
    ids = _ids(B, T, (100, 61), pad)
    seen = fa.visible(B, T, doc_ids=ids.cuda())
    clean = _run(q, k, v, do, seen, softcap=cap)
    for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, -math.inf)):
        x[:, :, T - pad:] = bad
    dirty = _run(q, k, v, do, seen, softcap=cap)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(clean[n], dirty[n]), n
    assert (clean["dq"].float() - dirty["dq"].float()).abs().max() <= 2 * ref.U * clean["dq"].float().abs().max()
    for n in ("o", "dq", "dk", "dv"):
        assert not dirty[n][:, :, T - pad:].any(), n
    assert torch.isneginf(dirty["lse"][:, :, T - pad:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,cap", [(64, 0.0), (64, 30.0), (128, 0.0), (128, 30.0), (128, 80.0)])
def test_rest_of_the_output(d, cap):
    """o + rest is the output to the precision of its products (P in bf16), not of its own rounding,
    and the gradients of peaked rows gain by it. In the norm, a rounding to bf16 is off by 2⁻⁸/√3 of
    what it rounds at most: dQ is rounded twice (dS and itself), so within √2·2⁻⁸/√3 = 3.2e-3, and
    the rounded P's share of D may add a quarter."""
    B, H, Hkv, T = 2, 4, 2, 300
    q, k, v, do = _tensors(B, H, Hkv, T, d, 31, 4.0)
    ids = _ids(B, T, (100, 31), 20)
    seen = fa.visible(B, T, doc_ids=ids.cuda())
    r = ref.attention(q, k, v, ref.visible_mask(B, T, True, ids), d ** -0.5, cap, None, do)
    rest = torch.full_like(q, math.nan).cuda()
    o, lse = fa.fwd_mod(q.cuda(), k.cuda(), v.cuda(), visible=seen, softcap=cap, rest=rest)
    assert torch.isfinite(rest).all() and not rest[:, :, T - 20:].any()
    off = lambda x, y: float((x.double().cpu() - y).norm() / y.norm())
    both = o.double() + rest.double()
    assert off(both, r["o"]) <= 2.0 ** -8 / 3 ** 0.5 and off(both, r["o"]) < 0.7 * off(o, r["o"])
    with_it, without = (_run(q, k, v, do, seen, softcap=cap, with_rest=x) for x in (True, False))
    for n in ("dq", "dk"):
        assert off(with_it[n], r[n]) <= 4e-3 and off(with_it[n], r[n]) < off(without[n], r[n]), n
    ref.check(without, r, ALL)


@pytest.mark.gpu
def test_nothing_visible_at_all():
    q, k, v, do = _tensors(1, 2, 2, 200, 64, 4)
    seen = fa.visible(1, 200, doc_ids=torch.full((1, 200), -1, dtype=torch.int32).cuda())
    got = _run(q, k, v, do, seen)
    assert torch.isneginf(got["lse"]).all()
    assert not any(got[n].any() for n in ("o", "dq", "dk", "dv"))


@pytest.mark.gpu
def test_plain_scores_match_the_dense_kernels():
    """No cap, no bias: the same attention as fwd and bwd, within both sides' bounds."""
    q, k, v, do = (x.cuda() for x in _tensors(2, 4, 4, 600, 64, 21))
    for causal in (True, False):
        o, lse = fa.fwd(q, k, v, causal=causal)
        o2, lse2 = fa.fwd_mod(q, k, v, causal=causal)
        assert (o.float() - o2.float()).abs().max() <= 2e-2 and (lse - lse2).abs().max() <= 1e-4
        for x, y in zip(fa.bwd(q, k, v, o, lse, do, causal=causal),
                        fa.bwd_mod(q, k, v, o, lse, do, causal=causal)):
            assert (x.float() - y.float()).abs().max() <= 4 * ref.U * x.float().abs().max()


@pytest.mark.gpu
def test_captured_and_replayed():
    """visible, forward and backward captured in one graph and replayed on new data."""
    B, H, Hkv, T, d = 2, 4, 2, 300, 64
    ids = [_ids(B, T, ls, 10).cuda() for ls in ((70, 33), (150, 5))]
    data = [tuple(x.cuda() for x in _tensors(B, H, Hkv, T, d, s)) for s in (1, 2)]
    sid, st = ids[0].clone(), [x.clone() for x in data[0]]

    def step():
        seen = fa.visible(B, T, doc_ids=sid)
        o, lse = fa.fwd_mod(*st[:3], visible=seen, softcap=20.0)
        return (o, lse) + fa.bwd_mod(*st[:3], o, lse, st[3], visible=seen, softcap=20.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in (1, 0):
        sid.copy_(ids[n])
        for x, y in zip(st, data[n]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        r = ref.attention(*(x.cpu() for x in data[n][:3]), ref.visible_mask(B, T, True, ids[n].cpu()),
                          d ** -0.5, 20.0, None, data[n][3].cpu())
        ref.check(dict(zip(ALL, out)), r, ALL, f"replay {n}")


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,interleaved,cap", [(64, 64, False, 30.0), (128, 64, True, 0.0)])
def test_training_step(d, rot, interleaved, cap):
    """A layer's attention as it is trained: queries and keys of the packed projection turned, packed
    documents, forward, backward, and the gradients turned back onto the projection's."""
    B, H, Hkv, T = 2, 6, 2, 250
    g = torch.Generator().manual_seed(17)
    x = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    do = torch.randn(B, H, T, d, generator=g).to(torch.bfloat16).cuda()
    ids = _ids(B, T, (90, 41), 12)
    f = fa.rope_inv_freq(rot, scaling="linear", factor=2.0)
    sl = _slopes(H).cuda()
    seen = fa.visible(B, T, doc_ids=ids.cuda())
    q, k = fa.rope(q, k, f, interleaved=interleaved)
    v = v.contiguous()
    rest = torch.empty_like(q)
    o, lse = fa.fwd_mod(q, k, v, visible=seen, softcap=cap, slopes=sl, rest=rest)
    dq, dk, dv = fa.bwd_mod(q, k, v, o, lse, do, visible=seen, softcap=cap, slopes=sl, rest=rest)
    gq, gk = fa.rope(dq, dk, f, interleaved=interleaved, inverse=True)
    torch.cuda.synchronize()
    r = ref.attention(q.cpu(), k.cpu(), v.cpu(), ref.visible_mask(B, T, True, ids), d ** -0.5, cap,
                      sl.cpu(), do.cpu())
    ref.check({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, r, ALL)
    # turned back: the reference's gradients times e^(−i·angle), their bounds added over a pair
    angle = torch.arange(T).double()[:, None] * f.cpu()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for got, n in ((gq, "dq"), (gk, "dk")):
        want, tol = r[n].clone(), r[n + "_tol"].clone()
        z = torch.complex(r[n][..., at[0]], r[n][..., at[1]]) * torch.polar(torch.ones_like(angle), -angle)
        pair = r[n + "_tol"][..., at[0]] + r[n + "_tol"][..., at[1]]
        for s, y in zip(at, (z.real, z.imag)):
            want[..., s], tol[..., s] = y, pair + ref.U * (y.abs() + pair) + 1e-6
        ref.check({n: got}, {n: want, n + "_tol": tol}, (n,), "turned back")


@pytest.mark.gpu
def test_wrapper_refusals_on_device():
    q, k, v, do = (x.cuda() for x in _tensors(1, 4, 2, 40, 64, 8))
    seen = fa.visible(1, 40, causal=False)
    o, lse = fa.fwd_mod(q, k, v, visible=seen)
    for call in (lambda: fa.fwd_mod(q, k[:, :, :39], v[:, :, :39]),
                 lambda: fa.fwd_mod(q[:, :3].contiguous(), k, v),
                 lambda: fa.fwd_mod(q, k, v, visible=seen, causal=True),
                 lambda: fa.fwd_mod(q, k, v, visible=fa.visible(1, 41)),
                 lambda: fa.fwd_mod(q, k, v, slopes=torch.zeros(2, device="cuda")),
                 lambda: fa.fwd_mod(q.transpose(2, 3), k, v),
                 lambda: fa.fwd_mod(q, k, v, lse=torch.zeros(1, 4, 39, device="cuda")),
                 lambda: fa.bwd_mod(q, k, v, o, lse[:, :3], do),
                 lambda: fa.bwd_mod(q, k, v, o, lse, do, dk=q),
                 lambda: fa.visible(1, 40, doc_ids=torch.zeros(1, 40, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fa.FAError):
        fa.fwd_mod(q, k, v, softcap=-1.0)
    with pytest.raises(TypeError):
        fa.fwd_mod(q, k, v, visible=torch.zeros(1))
