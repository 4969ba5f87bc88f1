"""A cache held in 4 bits (cache4, append4, read4, fwd_tree4): refusals on the CPU, the format and its
rounding bit for bit against a 64-bit reference written from the definition, and attention over it under
the bounds of mod_reference.py, the keys and values being exactly what the codes stand for."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_mod import _slopes
from tests.test_tree import _trees
from tests.test_window import tree_seen

A, SZ = 0x7F0000000000, 1 << 34
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED


# ------------------------------------------------------------------------- refusals (CPU)

def _append(k=A, v=A + SZ, ks=(6400, 3200, 64), kc=A + 2 * SZ, ksc=A + 3 * SZ, vc=A + 4 * SZ, vsc=A + 5 * SZ,
            ctx=A + 6 * SZ, B=2, Hkv=2, Tq=50, Tmax=400, d=64):
    return fa.fa_append4(k, ks, v, ks, kc, ksc, vc, vsc, ctx, B, Hkv, Tq, Tmax, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(kc=0), BAD), (dict(ksc=0), BAD), (dict(vc=0), BAD),
    (dict(vsc=0), BAD), (dict(ctx=0), BAD), (dict(B=0), BAD), (dict(Hkv=0), BAD), (dict(Tq=0), BAD),
    (dict(Tmax=0), BAD), (dict(Tmax=404), BAD), (dict(d=96), BAD), (dict(B=1 << 20, Hkv=1 << 20), BAD),
    (dict(ks=(6400, 3204, 64)), BAD), (dict(ks=(-64, 64, 64)), BAD),
    (dict(k=A + 8), MIS), (dict(kc=A + 2 * SZ + 8), MIS), (dict(vsc=A + 5 * SZ + 2), MIS), (dict(ctx=A + 6 * SZ + 1), MIS),
    (dict(kc=A), BAD), (dict(vc=A + 2 * SZ), BAD), (dict(vsc=A + 2 * SZ + 64), BAD), (dict(ctx=A + 3 * SZ), BAD),
])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


def _read(kc=A + 2 * SZ, ksc=A + 3 * SZ, vc=A + 4 * SZ, vsc=A + 5 * SZ, start=A + 6 * SZ, k=A, v=A + SZ, B=2,
          Hkv=2, n=50, Tmax=400, d=64):
    return fa.fa_read4(kc, ksc, vc, vsc, start, k, v, B, Hkv, n, Tmax, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kc=0), BAD), (dict(vsc=0), BAD), (dict(start=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD),
    (dict(n=0), BAD), (dict(Tmax=10), BAD), (dict(d=32), BAD), (dict(k=A + 2), MIS), (dict(vc=A + 4 * SZ + 4), MIS),
    (dict(k=A + SZ), BAD), (dict(k=A + 2 * SZ), BAD), (dict(v=A + 5 * SZ), BAD), (dict(v=A + 6 * SZ), BAD),
])
def test_read_refusals(kw, want):
    assert _read(**kw) == want


def _fwd(q=A, kc=A + SZ, ksc=A + 2 * SZ, vc=A + 3 * SZ, vsc=A + 4 * SZ, o=A + 5 * SZ, lse=A + 6 * SZ,
         ctx=A + 7 * SZ, window=0, sinks=0, cap=0.0, B=2, H=4, Hkv=2, Tq=8, Tmax=40000, d=64, scale=0.125,
         ws=A + 8 * SZ, ws_bytes=1 << 30):
    return fa.fa_fwd_tree4(q, kc, ksc, vc, vsc, o, lse, ctx, None, 0, None, 0, window, sinks, cap, None, B,
                           H, Hkv, Tq, Tmax, d, scale, ws, ws_bytes, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(kc=0), BAD), (dict(ksc=0), BAD), (dict(vsc=0), BAD), (dict(o=0), BAD),
    (dict(ctx=0), BAD), (dict(Tmax=4004), BAD), (dict(Hkv=3), BAD), (dict(d=32), BAD), (dict(cap=-1.0), BAD),
    (dict(window=-1), BAD), (dict(sinks=3), BAD), (dict(window=5, sinks=-1), BAD), (dict(scale=math.inf), BAD),
    (dict(ws=0), BAD), (dict(ws_bytes=64), BAD), (dict(ksc=A + 2 * SZ + 8), MIS), (dict(vc=A + 3 * SZ + 8), MIS),
    (dict(ws=A + 8 * SZ + 16), MIS), (dict(o=A + SZ), BAD), (dict(lse=A + 4 * SZ), BAD), (dict(ws=A + 2 * SZ), BAD),
])
def test_forward_refusals(kw, want):
    assert _fwd(**kw) == want


def test_wrappers_reject_what_they_cannot_take():
    codes, scales = torch.zeros(1, 1, 8, 32, dtype=torch.uint8), torch.zeros(1, 1, 8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.Cache4(codes, scales, codes, scales)                  # not on a GPU
    for bad in (dict(d=96), dict(Tmax=12)):
        with pytest.raises(ValueError):
            fa.cache4(**{**dict(B=1, Hkv=1, Tmax=16, d=64, device="cpu"), **bad})
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.append4(x, x, codes, None), lambda: fa.read4(None, None, 1)):
        with pytest.raises(TypeError):
            call()
    assert fa.fa_fwd_tree4_workspace_size(1, 2, 1, 1, 12, 64, 0, 0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_unsupported():
    none = fa.FA_ERR_UNSUPPORTED_DEVICE
    assert _append() == none and _read() == none and _fwd() == none and _fwd(window=70, sinks=4) == none


# --------------------------------------------------------------------------- the reference

def _dims(d, keys):
    if keys:
        return [32 * w + 4 * c + e for c in range(4) for w in range(d // 32) for e in (0, 2, 16, 18, 1, 3, 17, 19)]
    return [64 * h + n + 8 * x for h in range(d // 64) for n in range(8) for x in range(8)]


def quantised(x):
    """(whole numbers, scales) of rows in 64 bits, by the definition; NaN scales for groups of no numbers."""
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    top = torch.where(g.isnan().any(-1), torch.full_like(top, math.inf), top)
    live = (top >= 2.0 ** -100) & (top < 2.0 ** 125)
    t = torch.where(live, top, torch.ones_like(top))
    step = torch.exp2(torch.floor(torch.log2(t / 7)) - 4)        # five significant bits
    scale = torch.ceil(t / step / 7) * step
    n = torch.where(live[..., None], torch.round(g / scale[..., None]), torch.zeros_like(g))
    scale = torch.where(live, scale, torch.where(top >= 2.0 ** 125, torch.full_like(top, math.nan), torch.zeros_like(top)))
    return n, scale


def values(x):
    n, scale = quantised(x)
    return (n * scale[..., None]).flatten(-2)


def pack(n, keys):
    """Whole numbers [..., d/32, 32] as a row's bytes."""
    c = (n.flatten(-2)[..., _dims(n.shape[-1] * n.shape[-2], keys)] + 8).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _hold(k, v):
    """A cache of these rows (CPU tensors), packed by the definition."""
    out = []
    for x, keys in ((k, True), (v, False)):
        n, s = quantised(x)
        out += [pack(n, keys).cuda(), s.to(torch.bfloat16).cuda()]
    return fa.Cache4(*out)


def _randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * std * torch.exp(torch.randn((*shape[:-1], 1), generator=g))
    return x.to(torch.bfloat16)


def test_the_values_are_near():
    """A group's values are within half a scale of what they stand for, a scale at most 17/16 of the
    largest magnitude over 7; the numbers stay within ±7."""
    x = _randn((3, 50, 128), 1)
    n, s = quantised(x)
    assert n.abs().max() <= 7
    g = x.double().unflatten(-1, (-1, 32))
    assert (s <= g.abs().amax(-1) / 7 * 17 / 16).all()
    assert ((n * s[..., None] - g).abs() <= s[..., None] / 2).all()
    y = values(x)
    assert torch.equal(y.to(torch.bfloat16).double(), y)          # every value is a bf16 number


# ------------------------------------------------------------------------ the cache (GPU)

@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,n,Tmax,d", [(1, 1, 1, 8, 64), (4, 2, 9, 64, 128), (5, 3, 33, 56, 64), (2, 4, 300, 320, 128)])
def test_append_and_read(B, Hkv, n, Tmax, d):
    packed = _randn((B, n, 2 * Hkv + 1, d), n + d).cuda()
    k, v = (packed[:, :, s].transpose(1, 2) for s in (slice(1, Hkv + 1), slice(Hkv + 1, None)))
    cache = fa.cache4(B, Hkv, Tmax, d)
    old = _randn((B, Hkv, Tmax, d), 3), _randn((B, Hkv, Tmax, d), 4)
    fa.append4(old[0].cuda(), old[1].cuda(), cache, torch.zeros(B, dtype=torch.int32, device="cuda"))
    # from the start, in the middle, running over the end, full, inactive
    ctx = torch.tensor([0, 11, Tmax - n + 1, Tmax, -1][:B], dtype=torch.int32)
    fa.append4(k, v, cache, ctx.cuda())
    torch.cuda.synchronize()
    for new, was, codes, scales, keys in ((k, old[0], cache.k_codes, cache.k_scales, True),
                                          (v, old[1], cache.v_codes, cache.v_scales, False)):
        want = was.clone()
        for b, c in enumerate(ctx.tolist()):
            m = max(0, min(n, Tmax - c)) if c >= 0 else 0
            want[b, :, max(c, 0):max(c, 0) + m] = new[b, :, :m].cpu()
        num, s = quantised(want)
        assert torch.equal(codes.cpu(), pack(num, keys)) and torch.equal(scales.cpu(), s.to(torch.bfloat16))
    # all rows back, from in front of the end to behind it, from nowhere
    start = torch.tensor([0, 5, Tmax - 3, Tmax, -2][:B], dtype=torch.int32)
    rk, rv = fa.read4(cache, start.cuda(), Tmax)
    whole = fa.read4(cache, torch.zeros(B, dtype=torch.int32, device="cuda"), Tmax)
    for got, all_, x in ((rk, whole[0], cache.k_codes), (rv, whole[1], cache.v_codes)):
        for b, c in enumerate(start.tolist()):
            m = max(0, Tmax - c) if c >= 0 else 0
            assert torch.equal(got[b, :, :m], all_[b, :, max(c, 0):max(c, 0) + m]) and not got[b, :, m:].any()
    b0 = int(min(n, Tmax))
    assert torch.equal(whole[0][0, :, :b0].cpu().double(), values(k[0, :, :b0].cpu()))
    assert torch.equal(whole[1][0, :, :b0].cpu().double(), values(v[0, :, :b0].cpu()))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_every_rounding(d):
    """Values on, half-way between and around whole multiples of scales of every five-bit significand, and
    groups of extremes."""
    rows = []
    for top in list(range(128, 256)):                            # every significand of a largest magnitude
        _, s = quantised(torch.full((1, 32), float(top)))
        half = (torch.arange(-15, 16).double() / 2 * float(s)).to(torch.bfloat16).clamp(-top, top)
        rows.append(torch.cat((half, torch.tensor([float(top)], dtype=torch.bfloat16))))
    rows = torch.stack(rows)
    extremes = torch.zeros(8, 32, dtype=torch.bfloat16)
    extremes[1, 3], extremes[2, 4], extremes[3, 5] = math.nan, math.inf, -math.inf
    extremes[4, :2] = torch.tensor([2.0 ** -100, 2.0 ** -101], dtype=torch.bfloat16)
    extremes[5, 0], extremes[6, 9] = 2.0 ** -101, 1.99 * 2.0 ** 124
    extremes[7, 1] = 2.0 ** 125
    x = torch.cat((rows, rows * 2.0 ** -20, rows * 2.0 ** 60, extremes))
    x = x.reshape(1, 1, -1, d)
    T = x.shape[2]
    cache = fa.cache4(1, 1, -(-T // 8) * 8, d)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.append4(x.cuda(), x.cuda(), cache, zero)
    want = values(x)
    for got in fa.read4(cache, zero, T):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
    n, _ = quantised(x)
    assert torch.equal(cache.k_codes[:, :, :T].cpu(), pack(n, True))


# --------------------------------------------------------------------- attention (GPU)

def _check(ctx, H, Hkv, n, Tmax, d, window=0, sinks=0, tree=False, cap=0.0, bias=False, seed=0):
    B = len(ctx)
    g = torch.Generator().manual_seed(seed + Tmax + n)
    q = (torch.randn(B, H, n, d, generator=g) * (4.0 if cap else 1.0)).to(torch.bfloat16)
    k, v = (torch.randn(B, Hkv, Tmax, d, generator=g).to(torch.bfloat16) for _ in range(2))
    t, dep = _trees(B, n, seed) if tree else (None, None)
    sl = _slopes(H) if bias else None
    qa = torch.tensor(ctx)[:, None] + (torch.arange(n) if dep is None else dep)
    ka = torch.arange(Tmax).repeat(B, 1)
    for b, c in enumerate(ctx):
        m = max(0, min(n, Tmax - c)) if c >= 0 else 0
        if m:
            ka[b, c:c + m] = qa[b, :m]
    ok = tree_seen(ctx, n, Tmax, t, dep, window, sinks)
    r = ref.attention(q, values(k), values(v), ok, d ** -0.5, cap, sl, query_at=qa, key_at=ka)
    cache = _hold(k, v)
    nan = torch.full((), math.nan, dtype=torch.bfloat16)
    for b, c in enumerate(ctx):     # what no token can see, behind and between, holds anything
        for s in (cache.k_scales, cache.v_scales):
            s[b, :, max(0, c + n) if c >= 0 else 0:] = nan
            if window and c >= 0:
                s[b, :, sinks:max(sinks, c - window + 1)] = nan
    o, lse = fa.fwd_tree4(q.cuda(), cache, torch.tensor(ctx, dtype=torch.int32).cuda(),
                          tree=None if t is None else t.cuda(), depths=None if dep is None else dep.cuda(),
                          softcap=cap, slopes=None if sl is None else sl.cuda(), window=window, sinks=sinks)
    torch.cuda.synchronize()
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))


# room: longer caches have their work shared out in stretches, shorter ones a CTA an entry
@pytest.mark.gpu
@pytest.mark.parametrize("ctx,H,Hkv,n,Tmax,d,window,sinks,tree,cap,bias", [
    ([0], 1, 1, 1, 8, 64, 0, 0, False, 0.0, False),
    ([5, -1, 0], 2, 2, 1, 8, 128, 0, 0, False, 0.0, False),
    ([127, 128, 126], 4, 4, 1, 136, 64, 0, 0, False, 30.0, False),   # a new token at a chunk's ends
    ([0, 200, -1, 1, 500], 8, 2, 1, 512, 64, 0, 0, False, 0.0, True),
    ([1000, 3, 700], 16, 1, 1, 1024, 128, 0, 0, False, 50.0, True),  # sixteen heads on one
    ([129, 0], 6, 2, 5, 144, 64, 0, 0, True, 0.0, False),
    ([300, 77], 4, 2, 16, 320, 128, 0, 0, True, 0.0, True),          # 32 rows
    ([511, 90], 16, 4, 16, 600, 64, 0, 0, True, 5.0, False),         # 64 rows: two blocks
    ([90, 400], 5, 5, 33, 448, 128, 0, 0, False, 0.0, True),
    ([30, 2], 8, 1, 40, 72, 128, 0, 0, True, 20.0, False),           # 320 rows; one runs over the end
    ([100, 97, 120], 2, 1, 4, 96, 64, 0, 0, False, 0.0, False),      # full caches, drafts outside
    ([1000, 129, 700], 4, 1, 1, 1024, 128, 100, 4, False, 0.0, False),
    ([900, 300, 4], 6, 2, 5, 920, 64, 130, 70, True, 30.0, True),
    ([90, 400], 5, 5, 33, 448, 128, 8, 2, False, 0.0, False),        # a chain longer than its window
    ([500, 300], 2, 1, 4, 104, 64, 30, 0, False, 0.0, False),        # nothing left to see
])
@pytest.mark.parametrize("room", [0, 8000])
def test_parity(ctx, H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, room):
    if room and max(ctx) + n > Tmax:
        room = 0                                             # (they are about the cache's end)
    _check(ctx, H, Hkv, n, Tmax + room, d, window, sinks, tree, cap, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [2, 24])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts_in_many_stretches(H, d):
    _check([40000, 123, 9000, 0, 21111], H, 1, 3, 40104, d, tree=True, seed=3)


# Entries taken by clusters of 8, 6, 4, 3 and 2 CTAs, as in test_window.
@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,n,Tmax,d,window,sinks,tree,cap,bias,whole", [
    (4, 4, 4, 1, 2000, 64, 0, 0, False, 0.0, False, True),           # 16 entries
    (4, 8, 4, 8, 2000, 64, 0, 0, True, 30.0, True, True),            # 16, of 16 rows
    (3, 4, 1, 2, 3200, 128, 1900, 130, False, 0.0, True, True),
    (6, 16, 2, 5, 1600, 128, 0, 0, True, 0.0, False, True),          # 40 rows: three blocks of 16
    (20, 4, 4, 1, 1400, 64, 0, 0, False, 30.0, False, True),         # 80
    (20, 4, 4, 1, 904, 128, 0, 0, False, 0.0, True, True),
    (75, 2, 2, 1, 640, 128, 500, 4, False, 0.0, False, True),        # 150
    (80, 2, 2, 1, 1040, 64, 0, 0, False, 0.0, False, True),
    (15, 2, 2, 9, 800, 64, 0, 0, True, 0.0, False, True),            # 30, of 9 rows
    (17, 4, 4, 1, 1400, 128, 0, 0, False, 30.0, False, True),        # 68, by fours
    (33, 4, 4, 1, 1040, 64, 0, 0, False, 0.0, False, True),
    (3, 4, 4, 1, 20000, 128, 15000, 4, False, 0.0, False, False),
])
def test_clusters(B, H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, whole):
    assert (fa.fa_fwd_tree4_workspace_size(B, H, Hkv, n, Tmax, d, window, sinks) == 1) == whole
    ctx = [Tmax - n, -1, 0, 129, Tmax // 2, 250, Tmax, 1] * 10
    _check(ctx[:B], H, Hkv, n, Tmax, d, window, sinks, tree, cap, bias, seed=B)


@pytest.mark.gpu
@pytest.mark.parametrize("Tmax", [208, 5000])
def test_many_sequences(Tmax):
    _check([(37 * b) % 200 - 1 for b in range(75)], 2, 1, 2, Tmax, 64, seed=4)


@pytest.mark.gpu
def test_a_nan_in_a_visible_row_shows():
    B, H, T, d = 1, 2, 40, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(B, H, n, d, generator=g).to(torch.bfloat16) for n in (1, T, T))
    k[0, 0, 7, 3] = math.inf
    cache = _hold(k, v)
    o, lse = fa.fwd_tree4(q.cuda(), cache, torch.full((1,), T - 1, dtype=torch.int32, device="cuda"))
    assert o[0, 0].isnan().all() and lse[0, 0].isnan().all() and not o[0, 1].isnan().any()


@pytest.mark.gpu
def test_cache_past_32_bit_offsets():
    B, Hkv, Tmax, d = 2, 16, 1 << 20, 128             # 2³² elements, 2³¹ bytes of codes
    cache = fa.cache4(B, Hkv, Tmax, d)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(B, Hkv, 2, d, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, Hkv, 104, d, generator=g).to(torch.bfloat16) for _ in range(2))
    at = torch.tensor([50, Tmax - 104], dtype=torch.int32, device="cuda")
    fa.append4(k.cuda(), v.cuda(), cache, at)
    rk, rv = fa.read4(cache, at, 104)
    assert torch.equal(rk.double().cpu(), values(k)) and torch.equal(rv.double().cpu(), values(v))
    ctx = (at + 102).contiguous()
    o, lse = fa.fwd_tree4(q.cuda(), cache, ctx, window=60)
    ok = torch.zeros(B, 2, 104, dtype=torch.bool)
    for t in range(2):
        ok[:, t, 102 + t - 59:102 + t + 1] = True
    ref.check({"o": o, "lse": lse}, ref.attention(q, values(k), values(v), ok, d ** -0.5), ("o", "lse"))


@pytest.mark.gpu
def test_serving_steps_captured():
    """norm_rope → append4 → fwd_tree4 as a server runs it: a captured step replayed with growing contexts
    and new inputs, on another stream than the current one, against one pass over all tokens."""
    B, H, Hkv, n, Tmax, d, steps, window, sinks = 3, 8, 2, 2, 64, 128, 9, 10, 3
    T = n * steps
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    f = fa.rope_inv_freq(d)
    inp = x[:, :n].clone()
    cache = fa.cache4(B, Hkv, Tmax, d)
    ctx = torch.tensor([0, 0, -100], dtype=torch.int32, device="cuda")
    ws = fa.fwd_tree4_workspace(B, H, Hkv, n, Tmax, d, window=window, sinks=sinks)

    def step():
        q, k, v = (inp[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
        pos = (ctx[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")).contiguous()
        q, k = fa.norm_rope(q, k, wq, wk, f, positions=pos)
        fa.append4(k, v, cache, ctx)
        r = fa.fwd_tree4(q, cache, ctx, workspace=ws, window=window, sinks=sinks)
        ctx.add_(n)
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        ctx.sub_(n)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        outs = []
        for i in range(steps):
            inp.copy_(x[:, i * n:(i + 1) * n])
            graph.replay()
            outs.append([t.clone() for t in held])
    torch.cuda.synchronize()
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    q, k = fa.norm_rope(q, k, wq, wk, f)
    from tests.test_window import window_mask
    r = ref.attention(q.cpu(), values(k.cpu()), values(v.cpu()), window_mask(B, T, window, sinks), d ** -0.5)
    got = {"o": torch.cat([y[0] for y in outs], 2), "lse": torch.cat([y[1] for y in outs], 2)}
    ref.check({a: b[:2] for a, b in got.items()}, {a: b[:2] for a, b in r.items()}, ("o", "lse"))
    assert not got["o"][2].any() and torch.isneginf(got["lse"][2]).all()
    assert (cache.k_codes[2] == 0x88).all() and not cache.k_scales[2].any()   # the inactive one's rows stayed


@pytest.mark.gpu
def test_wrapper_refusals_on_device():
    cache = fa.cache4(2, 2, 64, 64)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: fa.append4(k, k[:, :1], cache, ctx), lambda: fa.append4(k, k, cache, ctx.long()),
                 lambda: fa.append4(k[..., :32], k, cache, ctx), lambda: fa.append4(k.cpu(), k, cache, ctx),
                 lambda: fa.read4(cache, ctx[:1], 4), lambda: fa.read4(cache, ctx, 4, out_k=k),
                 lambda: fa.fwd_tree4(q[:1].contiguous(), cache, ctx), lambda: fa.fwd_tree4(q[:, :3].contiguous(), cache, ctx),
                 lambda: fa.fwd_tree4(q, cache, ctx, sinks=3), lambda: fa.fwd_tree4(q, cache, ctx, window=-2),
                 lambda: fa.Cache4(cache.k_codes, cache.k_scales[..., :1], cache.v_codes, cache.v_scales),
                 lambda: fa.Cache4(cache.k_codes, cache.k_scales.float(), cache.v_codes, cache.v_scales),
                 lambda: fa.Cache4(cache.k_codes[:, :, :60], cache.k_scales, cache.v_codes, cache.v_scales)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fa.FAError):
        # (keys and values in one place)
        fa.append4(k, k, fa.Cache4(cache.k_codes, cache.k_scales, cache.k_codes, cache.v_scales), ctx)
