"""Rotary positions (rope, rope_append, rope_inv_freq): refusals on the CPU, GPU parity with a
64-bit reference written as complex products.

Bound: the result's rounding to bf16, 2⁻⁸ of the value, and the fp32 arithmetic before it: cosine
and sine within 2⁻²¹ (the functions' documented error in ±π) and 2⁻²² more (the angle's rounding to
24 bits), and three roundings, together at most 2⁻²⁰·m·(|a| + |b|)."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa

A, SZ = 0x7F0000000000, 1 << 32
BAD, MIS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED


# ------------------------------------------------------------------------- refusals (CPU)

def _rope(q=A, qs=(2 * 50 * 64, 50 * 64, 64), qo=A + SZ, k=A + 2 * SZ, ks=(50 * 64, 0, 64),
          ko=A + 3 * SZ, pos=None, per=0, f=A + 4 * SZ, rot=64, m=1.0, B=3, H=2, Hkv=1, T=50, d=64):
    return fa.fa_rope(q, qs, qo, k, ks, ko, pos, per, f, rot, 0, 0, m, B, H, Hkv, T, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), BAD), (dict(qo=0), BAD), (dict(f=0), BAD), (dict(k=0), BAD), (dict(ko=0), BAD),
    (dict(Hkv=0), BAD), (dict(B=0), BAD), (dict(T=0), BAD), (dict(d=96), BAD), (dict(rot=0), BAD),
    (dict(rot=8), BAD), (dict(rot=80), BAD), (dict(m=math.inf), BAD),
    (dict(qs=(-64, 64, 64)), BAD), (dict(qs=(6400, 3204, 64)), BAD),
    (dict(qs=(1 << 61, 3200, 64)), BAD),
    (dict(q=A + 8), MIS), (dict(qo=A + SZ + 2), MIS), (dict(pos=A + 5 * SZ + 2), MIS),
    (dict(f=A + 4 * SZ + 4), MIS),
    (dict(qo=A + 64), BAD), (dict(qo=A, qs=(6400, 64, 128)), BAD),   # in place needs its own layout
    (dict(ko=A), BAD), (dict(ko=A + SZ), BAD), (dict(qo=A + 2 * SZ), BAD),
])
def test_rope_refusals(kw, want):
    assert _rope(**kw) == want


def _append(q=A, qs=(256, 128, 64), qo=A + SZ, k=A + 2 * SZ, v=A + 3 * SZ, ks=(128, 0, 64),
            kc=A + 4 * SZ, vc=A + 5 * SZ, ctx=A + 6 * SZ, pos=None, f=A + 7 * SZ, rot=32, B=2, H=2,
            Hkv=1, Tq=2, Tmax=100, d=64):
    return fa.fa_rope_append(q, qs, qo, k, ks, v, ks, kc, vc, ctx, pos, 0, f, rot, 0, 1.0, B, H, Hkv,
                             Tq, Tmax, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(v=0), BAD), (dict(kc=0), BAD), (dict(ctx=0), BAD), (dict(Hkv=0), BAD), (dict(Tmax=0), BAD),
    (dict(rot=24), BAD), (dict(vc=A + 5 * SZ + 8), MIS), (dict(ctx=A + 6 * SZ + 1), MIS),
    (dict(kc=A + 5 * SZ), BAD), (dict(kc=A + 2 * SZ), BAD), (dict(qo=A + 4 * SZ), BAD),
])
def test_rope_append_refusals(kw, want):
    assert _append(**kw) == want


@pytest.mark.parametrize("call,kw", [
    (_rope, dict(pos=A + SZ)), (_rope, dict(pos=A + 3 * SZ + 256, per=1)), (_rope, dict(f=A + 3 * SZ)),
    (_append, dict(pos=A + SZ)), (_append, dict(f=A + 4 * SZ)), (_append, dict(ctx=A + 5 * SZ)),
])
def test_outputs_over_the_small_inputs_are_refused(call, kw):
    assert call(**kw) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_unsupported():
    assert _rope() == fa.FA_ERR_UNSUPPORTED_DEVICE
    assert _rope(k=None, ko=None, Hkv=0) == fa.FA_ERR_UNSUPPORTED_DEVICE
    assert _rope(qo=A) == fa.FA_ERR_UNSUPPORTED_DEVICE               # in place
    assert _append() == fa.FA_ERR_UNSUPPORTED_DEVICE


def test_frequencies():
    f = fa.rope_inv_freq(32, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (16,)
    assert f[0] == 1.0 and abs(float(f[8]) - 1e-2) < 1e-16
    assert torch.equal(fa.rope_inv_freq(32, scaling="linear", factor=4.0, device="cpu"), f / 4)
    g = fa.rope_inv_freq(32, scaling="by_parts", factor=8.0, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.equal(g[turns < 1], f[turns < 1] / 8)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (g[between] < f[between]).all() and (g[between] > f[between] / 8).all()
    for bad in (dict(rot_dim=20), dict(rot_dim=0), dict(rot_dim=32, base=0.0),
                dict(rot_dim=32, scaling="no"), dict(rot_dim=32, scaling="by_parts", low_turns=40.0)):
        with pytest.raises(ValueError):
            fa.rope_inv_freq(device="cpu", **bad)


def test_wrapper_rejects_cpu_tensors():
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.rope(x, None, fa.rope_inv_freq(64, device="cpu"))


# ---------------------------------------------------------------------------- parity (GPU)

def _turned(x, pos, f, interleaved, m, inverse):
    """(value, bound) of the turned rows in 64 bits; x [B, n, T, d], pos [B, T]."""
    x, rot = x.double().cpu(), 2 * f.numel()
    a, b = ((x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved
            else (x[..., :rot // 2], x[..., rot // 2:rot]))
    angle = pos.double().cpu()[:, None, :, None] * f.cpu()
    z = torch.complex(a, b) * torch.polar(torch.full_like(angle, m), -angle if inverse else angle)
    y, tol = x.clone(), torch.zeros_like(x)
    slack = 2.0 ** -20 * abs(m) * (a.abs() + b.abs())
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for s, part in zip(at, (z.real, z.imag)):
        y[..., s] = part
        tol[..., s] = 2.0 ** -8 * part.abs() + slack + 1e-30
    return y, tol


def _near(got, ref):
    y, tol = ref
    err = (got.double().cpu() - y).abs()
    assert (err <= tol).all(), float((err - tol).max())


def _packed(B, T, heads, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, T, heads, d, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hkv,T,d,rot,start,per_batch", [
    (1, 1, 0, 1, 64, 16, 0, False),
    (2, 3, 1, 7, 64, 64, 5, True),
    (1, 16, 4, 33, 128, 64, 100000, False),
    (3, 5, 5, 130, 128, 128, 2000000000, True),     # far positions keep their angle
    (2, 12, 12, 257, 64, 32, -40, False),           # negative positions turn backwards
])
def test_rope_parity(B, H, Hkv, T, d, rot, start, per_batch, interleaved):
    x = _packed(B, T, H + 2 * Hkv, d, T + d)
    q = x[:, :, :H].transpose(1, 2)
    k = x[:, :, H:H + Hkv].transpose(1, 2) if Hkv else None
    f = fa.rope_inv_freq(rot, scaling="by_parts", factor=4.0)
    pos = torch.arange(T, dtype=torch.int32) + start
    pos = torch.stack([pos + 3 * b for b in range(B)]) if per_batch else pos
    full = pos if per_batch else pos.expand(B, T)
    for inverse in (False, True):
        yq, yk = fa.rope(q, k, f, positions=pos.cuda(), interleaved=interleaved, inverse=inverse,
                         mscale=1.25)
        _near(yq, _turned(q, full, f, interleaved, 1.25, inverse))
        if Hkv:
            _near(yk, _turned(k, full, f, interleaved, 1.25, inverse))
        else:
            assert yk is None


@pytest.mark.gpu
def test_default_positions_in_place_and_strides():
    x = _packed(2, 40, 3, 128, 1)
    q = x.transpose(1, 2).contiguous()
    f = fa.rope_inv_freq(128)
    pos = torch.arange(40).expand(2, 40)
    want = _turned(q, pos, f, False, 1.0, False)
    y, _ = fa.rope(q, None, f)
    _near(y, want)
    same = q.clone()
    out, _ = fa.rope(same, None, f, out_q=same)
    assert out.data_ptr() == same.data_ptr() and torch.equal(out, y)
    # a broadcast batch (stride 0), every other token, a narrower slice of wider heads
    one = q[:1].expand(2, 3, 40, 128)
    _near(fa.rope(one, None, f)[0], _turned(one, pos, f, False, 1.0, False))
    skip = q[:, :, ::2]
    _near(fa.rope(skip, None, f)[0], _turned(skip, pos[:, :20], f, False, 1.0, False))
    part, f64 = q[..., 64:], fa.rope_inv_freq(64)
    _near(fa.rope(part, None, f64)[0], _turned(part, pos, f64, False, 1.0, False))
    with pytest.raises(fa.FAError):
        fa.rope(q[..., 4:68], None, f64)      # not on a 16-byte boundary: refused


@pytest.mark.gpu
def test_gradient_is_the_inverse_turn():
    """<rope(x), g> = <x, rope(g, inverse)> within the roundings of both sides."""
    x, g = (_packed(2, 50, 4, 64, s).transpose(1, 2).contiguous() for s in (3, 4))
    f = fa.rope_inv_freq(64)
    a = (fa.rope(x, None, f, mscale=1.1)[0].double() * g.double())
    b = (x.double() * fa.rope(g, None, f, inverse=True, mscale=1.1)[0].double())
    room = 2.0 ** -8 * (a.abs().sum() + b.abs().sum())
    assert (a.sum() - b.sum()).abs() <= room


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,n,Tmax,d,rot,interleaved", [
    (1, 4, 2, 1, 20, 64, 64, False), (4, 6, 2, 9, 64, 128, 64, True), (5, 3, 3, 33, 50, 64, 16, False),
])
def test_append(B, H, Hkv, n, Tmax, d, rot, interleaved):
    x = _packed(B, n, H + 2 * Hkv, d, n + d)
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    kc, vc = (_packed(B, Hkv, Tmax, d, s) for s in (1, 2))
    k0, v0 = kc.clone(), vc.clone()
    # from the start, in the middle, running over the end, full, inactive
    ctx = torch.tensor([0, 11, Tmax - n + 1, Tmax, -1][:B], dtype=torch.int32)
    f = fa.rope_inv_freq(rot)
    for positions in (None, (ctx[:, None] + 2 * torch.arange(n)).to(torch.int32)):
        pos = ctx[:, None] + torch.arange(n) if positions is None else positions
        kc.copy_(k0)
        vc.copy_(v0)
        y = fa.rope_append(q, k, v, kc, vc, ctx.cuda(), f, interleaved=interleaved,
                           positions=None if positions is None else positions.cuda())
        torch.cuda.synchronize()
        yq, yk = (_turned(t, pos, f, interleaved, 1.0, False) for t in (q, k))
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
    """The last sequence's rows lie beyond 2³¹ elements."""
    B, Hkv, Tmax, d = 2, 8, 1 << 20, 128            # 2³¹ elements, 4.3 GB a cache
    kc, vc = (torch.zeros(B, Hkv, Tmax, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _packed(B, 2, 3 * Hkv, d, 6)
    q, k, v = (x[:, :, i * Hkv:(i + 1) * Hkv].transpose(1, 2) for i in range(3))
    ctx = torch.tensor([5, Tmax - 2], dtype=torch.int32)
    f = fa.rope_inv_freq(d)
    fa.rope_append(q, k, v, kc, vc, ctx.cuda(), f)
    pos = ctx[:, None] + torch.arange(2)
    yk = _turned(k, pos, f, False, 1.0, False)
    for b, at in enumerate(ctx.tolist()):
        _near(kc[b, :, at:at + 2], (yk[0][b], yk[1][b]))
        assert torch.equal(vc[b, :, at:at + 2], v[b])
        assert not kc[b, :, :at].any() and not kc[b, :, at + 2:].any()
