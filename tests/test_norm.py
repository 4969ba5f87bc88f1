"""Head norms with rotary positions (norm_rope, norm_rope_append, norm_rope_bwd): refusals on the CPU,
GPU parity with a 64-bit reference.

Bounds (u = 2⁻⁸, half a bf16 step relative to the value).
  y    u·|y|, and before that rounding 2⁻²⁰·m·(|a| + |b|) for the turn (as rope), r's error (the sum of
       squares in at most 13 additions of one sign, halved by the root, and rsqrt's two units:
       2⁻²¹ in all) and two products: together below 2⁻¹⁹·m·(|a| + |b|), a and b the normed pair
  dx   u·|dx| + 2⁻¹⁸·M, M = r·(|h||w| + |n|·mean(|h||w||n|)) with |h| ≤ m·(|ga| + |gb|): the errors
       above for h and n, twice for the product of two of them
  dw   2⁻¹⁶·Σ|h||n|: 2⁻¹⁸ for the terms; at these sizes a sum goes through at most 16 heads a
       thread, 5 lanes, 4 warps, 19 and 32 rows of partial sums, 76 additions of 2⁻²⁴ each"""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa

A, SZ = 0x7F0000000000, 1 << 32
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED
EPS = 1e-6


# ------------------------------------------------------------------------- refusals (CPU)

def _norm(q=A, qs=(2 * 50 * 64, 50 * 64, 64), qo=A + SZ, k=A + 2 * SZ, ks=(50 * 64, 0, 64),
          ko=A + 3 * SZ, wq=A + 6 * SZ, wk=A + 7 * SZ, eps=EPS, pos=None, per=0, f=A + 4 * SZ, rot=64,
          m=1.0, B=3, H=2, Hkv=1, T=50, d=64):
    return fa.fa_norm_rope(q, qs, qo, k, ks, ko, wq, wk, eps, pos, per, f, rot, 0, m, B, H, Hkv, T, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(qo=0), BAD), (dict(f=0), BAD), (dict(wq=0), BAD), (dict(wk=0), BAD),
    (dict(k=0), BAD), (dict(ko=0), BAD), (dict(Hkv=0), BAD), (dict(B=0), BAD), (dict(T=0), BAD),
    (dict(d=96), BAD), (dict(rot=0), BAD), (dict(rot=80), BAD), (dict(m=math.inf), BAD),
    (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD),
    (dict(qs=(-64, 64, 64)), BAD), (dict(qs=(6400, 3204, 64)), BAD),
    (dict(q=A + 8), MIS), (dict(wq=A + 6 * SZ + 2), MIS), (dict(wk=A + 7 * SZ + 1), MIS),
    (dict(f=A + 4 * SZ + 4), MIS), (dict(pos=A + 5 * SZ + 2), MIS),
    (dict(qo=A + 64), BAD), (dict(ko=A), BAD), (dict(ko=A + SZ), BAD), (dict(wq=A + SZ + 256), BAD),
    (dict(wk=A + 3 * SZ), BAD), (dict(pos=A + SZ), BAD), (dict(f=A + 3 * SZ), BAD),
])
def test_refusals(kw, want):
    assert _norm(**kw) == want


def _append(q=A, qs=(256, 128, 64), qo=A + SZ, k=A + 2 * SZ, v=A + 3 * SZ, ks=(128, 0, 64), wq=A + 8 * SZ,
            wk=A + 9 * SZ, eps=EPS, kc=A + 4 * SZ, vc=A + 5 * SZ, ctx=A + 6 * SZ, pos=None, f=A + 7 * SZ,
            rot=32, B=2, H=2, Hkv=1, Tq=2, Tmax=100, d=64):
    return fa.fa_norm_rope_append(q, qs, qo, k, ks, v, ks, wq, wk, eps, kc, vc, ctx, pos, 0, f, rot, 0,
                                  1.0, B, H, Hkv, Tq, Tmax, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(v=0), BAD), (dict(kc=0), BAD), (dict(ctx=0), BAD), (dict(wk=0), BAD), (dict(Hkv=0), BAD),
    (dict(Tmax=0), BAD), (dict(eps=0.0), BAD), (dict(vc=A + 5 * SZ + 8), MIS), (dict(ctx=A + 6 * SZ + 1), MIS),
    (dict(wq=A + 8 * SZ + 2), MIS), (dict(kc=A + 5 * SZ), BAD), (dict(kc=A + 2 * SZ), BAD),
    (dict(qo=A + 4 * SZ), BAD), (dict(wq=A + 4 * SZ), BAD), (dict(ctx=A + SZ), BAD),
])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


def _bwd(gq=A, q=A + SZ, dq=A + 2 * SZ, gk=A + 3 * SZ, k=A + 4 * SZ, dk=A + 5 * SZ, wq=A + 6 * SZ,
         wk=A + 7 * SZ, dwq=A + 8 * SZ, dwk=A + 9 * SZ, eps=EPS, f=A + 10 * SZ, ws=A + 11 * SZ, n=None,
         gs=(6400, 3200, 64), B=3, H=2, Hkv=1, T=50, d=64):
    n = fa.fa_norm_rope_bwd_workspace_size(d) if n is None else n
    ks = (3200, 0, 64)
    return fa.fa_norm_rope_bwd(gq, gs, q, (6400, 3200, 64), dq, gk, ks, k, ks, dk, wq, wk, dwq, dwk, eps,
                               None, 0, f, 64, 0, 1.0, B, H, Hkv, T, d, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(gq=0), BAD), (dict(q=0), BAD), (dict(dq=0), BAD), (dict(gk=0), BAD), (dict(k=0), BAD),
    (dict(dk=0), BAD), (dict(wq=0), BAD), (dict(wk=0), BAD), (dict(dwq=0), BAD), (dict(dwk=0), BAD),
    (dict(ws=0), BAD), (dict(n=16), BAD), (dict(eps=0.0), BAD), (dict(Hkv=0), BAD), (dict(d=32), BAD),
    (dict(ws=A + 11 * SZ + 128), MIS), (dict(dq=A + 2 * SZ + 8), MIS), (dict(dwq=A + 8 * SZ + 2), MIS),
    (dict(dq=A + SZ), BAD), (dict(dk=A + 4 * SZ), BAD), (dict(dq=A, gs=(6400, 64, 128)), BAD),
    (dict(dk=A), BAD), (dict(dq=A + 3 * SZ), BAD), (dict(dwq=A + 9 * SZ + 16), BAD),
    (dict(ws=A + SZ), BAD), (dict(dwk=A + 11 * SZ), BAD), (dict(dwq=A + 6 * SZ), BAD),
    (dict(dq=A + 7 * SZ), BAD),
])
def test_backward_refusals(kw, want):
    assert _bwd(**kw) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_unsupported():
    none = fa.FA_ERR_UNSUPPORTED_DEVICE
    assert _norm() == none and _norm(qo=A) == none and _append() == none
    assert _norm(k=None, ko=None, wk=None, Hkv=0) == none
    assert _bwd() == none and _bwd(dq=A) == none
    assert _bwd(gk=None, k=None, dk=None, wk=None, dwk=None, Hkv=0) == none


def test_wrappers_reject_what_they_cannot_take():
    x, w = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.ones(64)
    f = fa.rope_inv_freq(64, device="cpu")
    with pytest.raises(ValueError):
        fa.norm_rope(x, None, w, None, f)
    with pytest.raises(ValueError):
        fa.norm_rope_bwd(x, None, x, None, w, None, f)
    with pytest.raises(ValueError):
        fa.norm_rope_append(x, x, x, w, w, x, x, torch.zeros(1, dtype=torch.int32), f)
    with pytest.raises(fa.FAError):
        fa.norm_rope_bwd_workspace(96)


# --------------------------------------------------------------------------- the reference

def _slices(rot, interleaved):
    return ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))


def _turn(y, pos, f, interleaved, m, inverse):
    """(turned rows, bound on their sizes) in 64 bits; pos [B, T]."""
    rot = 2 * f.numel()
    sa, sb = _slices(rot, interleaved)
    a, b = y[..., sa], y[..., sb]
    angle = pos.double()[:, None, :, None] * f.cpu()
    z = torch.complex(a, b) * torch.polar(torch.full_like(angle, m), -angle if inverse else angle)
    out, size = y.clone(), y.abs()
    for s, part in ((sa, z.real), (sb, z.imag)):
        out[..., s] = part
        size[..., s] = abs(m) * (a.abs() + b.abs())
    return out, size


def _forward(x, w, pos, f, interleaved, m, eps):
    x = x.double().cpu()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y, size = _turn(n * w.double().cpu(), pos, f, interleaved, m, False)
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -19 * size + 1e-30


def _backward(g, x, w, pos, f, interleaved, m, eps):
    """((dx, bound), (dw, bound))."""
    g, x, w = g.double().cpu(), x.double().cpu(), w.double().cpu()
    h, size = _turn(g, pos, f, interleaved, m, True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dx = r * (h * w - n * (h * w * n).mean(-1, keepdim=True))
    M = r * (size * w.abs() + n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True))
    dw, W = (h * n).sum((0, 1, 2)), (size * n.abs()).sum((0, 1, 2))
    return (dx, 2.0 ** -8 * dx.abs() + 2.0 ** -18 * M + 1e-30), (dw, 2.0 ** -16 * W + 1e-30)


def _near(got, ref, what=""):
    y, tol = ref
    err = (got.double().cpu() - y).abs()
    assert (err <= tol).all(), f"{what} {float((err / tol).max()):.3f} of the bound"


def test_the_reference_gradient_agrees_with_differences():
    g = torch.Generator().manual_seed(5)
    x, up = torch.randn(1, 2, 3, 64, generator=g).double(), torch.randn(1, 2, 3, 64, generator=g).double()
    w, f = torch.rand(64, generator=g).double() + 0.5, fa.rope_inv_freq(32, device="cpu")
    pos = torch.tensor([[3, 10, -7]])
    loss = lambda a, b: float((_forward(a, b, pos, f, True, 1.3, 1e-2)[0] * up).sum())
    (dx, _), (dw, _) = _backward(up, x, w, pos, f, True, 1.3, 1e-2)
    dirx, dirw = torch.randn(x.shape, generator=g).double(), torch.randn(64, generator=g).double()
    e = 1e-5
    for got, hi, lo in (((dx * dirx).sum(), loss(x + e * dirx, w), loss(x - e * dirx, w)),
                        ((dw * dirw).sum(), loss(x, w + e * dirw), loss(x, w - e * dirw))):
        # central differences: e²/6 of the third derivative, of order 1e2 here, and 1e-16/e of rounding
        assert abs(float(got) - (hi - lo) / (2 * e)) < 1e-7 * (1 + abs(float(got)))


# ---------------------------------------------------------------------------- parity (GPU)

def _packed(B, T, heads, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, heads, d, generator=g) * torch.exp(torch.randn(B, T, heads, 1, generator=g))
    return x.to(torch.bfloat16).cuda()


def _weights(d, seed):
    g = torch.Generator().manual_seed(100 + seed)
    return [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]


SIZES = [
    (1, 1, 0, 1, 64, 16, 0, False),
    (2, 3, 1, 7, 64, 64, 5, True),
    (1, 16, 4, 33, 128, 64, 100000, False),
    (3, 5, 5, 130, 128, 128, 2000000000, True),
    (2, 12, 12, 257, 64, 32, -40, False),
]


def _inputs(B, H, Hkv, T, d, rot, start, per_batch):
    x = _packed(B, T, H + 2 * Hkv, d, T + d)
    q = x[:, :, :H].transpose(1, 2)
    k = x[:, :, H:H + Hkv].transpose(1, 2) if Hkv else None
    pos = torch.arange(T, dtype=torch.int32) + start
    pos = torch.stack([pos + 3 * b for b in range(B)]) if per_batch else pos
    wq, wk = _weights(d, T)
    return q, k, wq, wk if Hkv else None, fa.rope_inv_freq(rot, scaling="by_parts", factor=4.0), pos


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_forward_parity(size, interleaved):
    q, k, wq, wk, f, pos = _inputs(*size)
    full = pos if pos.dim() == 2 else pos.expand(size[0], size[3])
    for eps in (EPS, 0.5):
        yq, yk = fa.norm_rope(q, k, wq, wk, f, positions=pos.cuda(), interleaved=interleaved,
                              mscale=1.25, eps=eps)
        _near(yq, _forward(q, wq, full, f, interleaved, 1.25, eps), "q")
        if k is None:
            assert yk is None
        else:
            _near(yk, _forward(k, wk, full, f, interleaved, 1.25, eps), "k")


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_backward_parity(size, interleaved):
    q, k, wq, wk, f, pos = _inputs(*size)
    B, H, Hkv, T, d = size[:5]
    full = pos if pos.dim() == 2 else pos.expand(B, T)
    gs = _packed(B, T, H + Hkv, d, 7)
    gq, gk = gs[:, :, :H].transpose(1, 2), gs[:, :, H:].transpose(1, 2) if Hkv else None
    kw = dict(positions=pos.cuda(), interleaved=interleaved, mscale=1.25, eps=1e-3)
    dq, dk, dwq, dwk = fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f, **kw)
    for g, x, w, dx, dw in ((gq, q, wq, dq, dwq), (gk, k, wk, dk, dwk)):
        if x is None:
            assert dx is None and dw is None
            continue
        rows, weight = _backward(g, x, w, full, f, interleaved, 1.25, 1e-3)
        _near(dx, rows, "dx")
        _near(dw, weight, "dw")
    # the same bits again, with a workspace of the caller's, in place of the gradients
    cq, ck = gq.contiguous(), gk.contiguous() if Hkv else None
    again = fa.norm_rope_bwd(cq, ck, q, k, wq, wk, f, dq=cq, dk=ck,
                             workspace=fa.norm_rope_bwd_workspace(d), **kw)
    assert again[0].data_ptr() == cq.data_ptr()
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.gpu
def test_long_weight_gradient():
    """Sums over 2.6 million rows, every block walking many tasks: against the same sum in 64 bits. A
    thread adds 2²¹·8 / (486·128) = 270 terms of the queries' or as many of the keys', then the 60
    additions behind it: 350·2⁻²⁴ of Σ|h||n|."""
    B, H, Hkv, T, d = 2, 16, 4, 65536, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, gq = (torch.randn(B, H, T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k, gk = (torch.randn(B, Hkv, T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    wq, wk = _weights(d, 1)
    f = fa.rope_inv_freq(d)
    _, _, dwq, dwk = fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f)
    for gr, x, dw in ((gq, q, dwq), (gk, k, dwk)):
        h = fa.rope(gr, None, f, inverse=True)[0].double()  # (rounded to bf16: 2⁻⁸ a term)
        n = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS)
        want = (h * n).sum((0, 1, 2))
        # the terms' roundings are independent: six deviations of 2⁻⁸/√3 a term, and the sum's
        room = 6 * 2.0 ** -8 / math.sqrt(3) * torch.sqrt(((h * n) ** 2).sum((0, 1, 2))) \
            + 350 * 2.0 ** -24 * (h * n).abs().sum((0, 1, 2))
        assert ((dw.double() - want).abs() <= room).all()


@pytest.mark.gpu
def test_defaults_in_place_and_strides():
    x = _packed(2, 40, 3, 128, 1)
    q = x.transpose(1, 2).contiguous()
    f, (w, _) = fa.rope_inv_freq(128), _weights(128, 2)
    pos = torch.arange(40).expand(2, 40)
    y, _ = fa.norm_rope(q, None, w, None, f)
    _near(y, _forward(q, w, pos, f, False, 1.0, EPS))
    same = q.clone()
    out, _ = fa.norm_rope(same, None, w, None, f, out_q=same)
    assert out.data_ptr() == same.data_ptr() and torch.equal(out, y)
    one = q[:1].expand(2, 3, 40, 128)
    _near(fa.norm_rope(one, None, w, None, f)[0], _forward(one, w, pos, f, False, 1.0, EPS))
    skip = q[:, :, ::2]
    _near(fa.norm_rope(skip, None, w, None, f)[0], _forward(skip, w, pos[:, :20], f, False, 1.0, EPS))
    part, f64, w64 = q[..., 64:], fa.rope_inv_freq(64), w[:64].contiguous()
    _near(fa.norm_rope(part, None, w64, None, f64)[0], _forward(part, w64, pos, f64, False, 1.0, EPS))
    # weights that start on any word
    _near(fa.norm_rope(part, None, w[3:67], None, f64)[0], _forward(part, w[3:67], pos, f64, False, 1.0, EPS))
    for bad in (dict(q_weight=w64), dict(q_weight=w.half()), dict(q_weight=w.cpu())):
        with pytest.raises(ValueError):
            fa.norm_rope(q, None, **bad, k_weight=None, inv_freq=f)
    with pytest.raises(ValueError):
        fa.norm_rope(q, q, w, None, f)


@pytest.mark.gpu
def test_rows_of_zeros_and_extremes():
    f, w = fa.rope_inv_freq(64), torch.ones(64, device="cuda")
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1] = 2.0 ** -60                   # far below eps
    x[0, 0, 2] = 2.0 ** 60
    x[0, 0, 3, 5] = math.nan
    y, _ = fa.norm_rope(x, None, w, None, f)
    pos = torch.arange(4).expand(1, 4)
    _near(y[:, :, :3], _forward(x[:, :, :3], w, pos[:, :3], f, False, 1.0, EPS))
    assert not y[0, 0, 0].any() and y[0, 0, 3].isnan().all()     # a NaN stays in its row
    g = torch.ones_like(x)
    dx = fa.norm_rope_bwd(g, None, x, None, w, None, f)[0]
    _near(dx[:, :, :3], tuple(t[:, :, :3] for t in _backward(g[:, :, :3], x[:, :, :3], w, pos[:, :3], f, False, 1.0, EPS)[0]))


@pytest.mark.gpu
def test_eps_whose_square_root_inverse_squared_is_no_number():
    # (1/√eps)² = 2^133 passes fp32's range, 1/√eps and the gradient do not
    eps, f, w = 2.0 ** -133, fa.rope_inv_freq(64), torch.ones(64, device="cuda")
    x = torch.zeros(1, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1], x[0, 0, 2] = 2.0 ** -64, 2.0 ** -62
    pos, g = torch.arange(3).expand(1, 3), torch.ones_like(x)
    _near(fa.norm_rope(x, None, w, None, f, eps=eps)[0], _forward(x, w, pos, f, False, 1.0, eps))
    dx, _, dw, _ = fa.norm_rope_bwd(g, None, x, None, w, None, f, eps=eps)
    rows, sums = _backward(g, x, w, pos, f, False, 1.0, eps)
    _near(dx, rows)
    _near(dw, sums)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,n,Tmax,d,rot,interleaved", [
    (1, 4, 2, 1, 20, 64, 64, False), (4, 6, 2, 9, 64, 128, 64, True), (5, 3, 3, 33, 50, 64, 16, False),
])
def test_append(B, H, Hkv, n, Tmax, d, rot, interleaved):
    x = _packed(B, n, H + 2 * Hkv, d, n + d)
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    kc, vc = (_packed(B, Hkv, Tmax, d, s) for s in (1, 2))
    k0, v0 = kc.clone(), vc.clone()
    wq, wk = _weights(d, n)
    # from the start, in the middle, running over the end, full, inactive
    ctx = torch.tensor([0, 11, Tmax - n + 1, Tmax, -1][:B], dtype=torch.int32)
    f = fa.rope_inv_freq(rot)
    for positions in (None, (ctx[:, None] + 2 * torch.arange(n)).to(torch.int32)):
        pos = ctx[:, None] + torch.arange(n) if positions is None else positions
        kc.copy_(k0)
        vc.copy_(v0)
        y = fa.norm_rope_append(q, k, v, wq, wk, kc, vc, ctx.cuda(), f, interleaved=interleaved,
                                positions=None if positions is None else positions.cuda())
        torch.cuda.synchronize()
        yq, yk = (_forward(t, w, pos, f, interleaved, 1.0, EPS) for t, w in ((q, wq), (k, wk)))
        for b in range(B):
            at, stay = int(ctx[b]), k0[b].clone()
            rows = max(0, min(n, Tmax - at)) if at >= 0 else 0
            if at < 0:
                assert not y[b].any()
            else:
                _near(y[b], (yq[0][b], yq[1][b]))
            want_v = v0[b].clone()
            if rows:
                _near(kc[b, :, at:at + rows], (yk[0][b, :, :rows], yk[1][b, :, :rows]))
                stay[:, at:at + rows] = kc[b, :, at:at + rows]
                want_v[:, at:at + rows] = v[b, :, :rows]
            assert torch.equal(kc[b], stay) and torch.equal(vc[b], want_v), f"sequence {b}"


@pytest.mark.gpu
def test_append_into_a_cache_past_32_bit_offsets():
    B, Hkv, Tmax, d = 2, 8, 1 << 20, 128            # 2³¹ elements, 4.3 GB a cache
    kc, vc = (torch.zeros(B, Hkv, Tmax, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _packed(B, 2, 3 * Hkv, d, 6)
    q, k, v = (x[:, :, i * Hkv:(i + 1) * Hkv].transpose(1, 2) for i in range(3))
    ctx = torch.tensor([5, Tmax - 2], dtype=torch.int32)
    f, (wq, wk) = fa.rope_inv_freq(d), _weights(d, 3)
    fa.norm_rope_append(q, k, v, wq, wk, kc, vc, ctx.cuda(), f)
    yk = _forward(k, wk, ctx[:, None] + torch.arange(2), f, False, 1.0, EPS)
    for b, at in enumerate(ctx.tolist()):
        _near(kc[b, :, at:at + 2], (yk[0][b], yk[1][b]))
        assert torch.equal(vc[b, :, at:at + 2], v[b])
        assert not kc[b, :, :at].any() and not kc[b, :, at + 2:].any()


@pytest.mark.gpu
def test_streams_and_captured_graphs():
    """Calls on another stream than the current one's, and replays of a captured call with new inputs."""
    B, H, Hkv, T, d = 2, 4, 2, 65, 64
    q, k, wq, wk, f, pos = _inputs(B, H, Hkv, T, d, 64, 0, False)
    q, k = q.contiguous(), k.contiguous()
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    want = fa.norm_rope(q, k, wq, wk, f) + fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f)
    ws = fa.norm_rope_bwd_workspace(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fa.norm_rope(q, k, wq, wk, f) + fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            held = fa.norm_rope(q, k, wq, wk, f) + fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    q.copy_(torch.randn_like(q))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, fa.norm_rope(q, k, wq, wk, f) + fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f)):
        assert torch.equal(a, b)
