"""Head norms on batches whose blocks walk several heads and several tasks: every row against the 64-bit
reference, and bit for bit against calls on short stretches of tokens, whose blocks take one head each.
Bounds as in test_norm.py; a weight's sum goes, at these sizes, through at most 10 tasks of 3 heads a thread, 3
lanes, 4 warps, 14 and 32 rows of partial sums, 83 additions: 83·2⁻²⁴ and the terms' 2⁻¹⁸ stay below 2⁻¹⁶."""

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests.test_norm import EPS, _backward, _forward, _near, _packed, _weights

SIZES = [(1, 5, 2, 65536, 64, 64), (3, 6, 3, 9000, 128, 64)]


def _batch(B, H, Hkv, T, d, rot):
    x, g = _packed(B, T, H + Hkv, d, T), _packed(B, T, H + Hkv, d, 7)
    pos = torch.stack([torch.arange(T, dtype=torch.int32) * (1 + b) - 50 * b for b in range(B)])
    parts = [t[:, :, s].transpose(1, 2) for t in (x, g) for s in (slice(0, H), slice(H, None))]
    return parts, _weights(d, T), fa.rope_inv_freq(rot), pos


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_blocks_of_several_heads(size, interleaved):
    (q, k, gq, gk), (wq, wk), f, pos = _batch(*size)
    at = pos.cuda()
    kw = dict(interleaved=interleaved, mscale=1.25)
    yq, yk = fa.norm_rope(q, k, wq, wk, f, positions=at, **kw)
    dq, dk, dwq, dwk = fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f, positions=at, **kw)
    for b in range(size[0]):
        for x, g, w, y, dx in ((q, gq, wq, yq, dq), (k, gk, wk, yk, dk)):
            _near(y[b:b + 1], _forward(x[b:b + 1], w, pos[b:b + 1], f, interleaved, 1.25, EPS), "y")
            _near(dx[b:b + 1], _backward(g[b:b + 1], x[b:b + 1], w, pos[b:b + 1], f, interleaved, 1.25, EPS)[0], "dx")
    for g, x, w, dw in ((gq, q, wq, dwq), (gk, k, wk, dwk)):
        _near(dw, _backward(g, x, w, pos, f, interleaved, 1.25, EPS)[1], "dw")
    n = 120                                                     # (of the last stretch, what is left)
    for a in (0, 31 * n, size[3] - 65):
        s = slice(a, a + n)
        kw["positions"] = at[:, s].contiguous()
        few = fa.norm_rope(q[:, :, s], k[:, :, s], wq, wk, f, **kw)
        few += fa.norm_rope_bwd(gq[:, :, s], gk[:, :, s], q[:, :, s], k[:, :, s], wq, wk, f, **kw)[:2]
        for part, whole in zip(few, (yq, yk, dq, dk)):
            assert torch.equal(part, whole[:, :, s])


@pytest.mark.gpu
def test_weight_gradients_and_rows_of_many_tasks():
    """B2 H16+4 T65536 d128, 17 tasks a block: the rows, too, are those of short calls."""
    B, H, Hkv, T, d = 2, 16, 4, 65536, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, gq = (torch.randn(B, H, T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k, gk = (torch.randn(B, Hkv, T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    (wq, wk), f = _weights(d, 1), fa.rope_inv_freq(d)
    dq, dk = fa.norm_rope_bwd(gq, gk, q, k, wq, wk, f)[:2]
    yq, yk = fa.norm_rope(q, k, wq, wk, f)
    for a in range(0, T, 4096):
        s = slice(a, a + 40)
        at = torch.arange(a, a + 40, dtype=torch.int32, device="cuda")
        few = fa.norm_rope_bwd(gq[:, :, s], gk[:, :, s], q[:, :, s], k[:, :, s], wq, wk, f, positions=at)[:2]
        few += fa.norm_rope(q[:, :, s], k[:, :, s], wq, wk, f, positions=at)
        for part, whole in zip(few, (dq, dk, yq, yk)):
            assert torch.equal(part, whole[:, :, s])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_with_all_heads_in_a_block(interleaved):
    """40000 new rows: a block walks queries, keys and values in turn; caches that end before them, a full one
    and an inactive sequence among them."""
    B, H, Hkv, n, Tmax, d = 5, 3, 2, 8000, 9000, 64
    x = _packed(B, n, H + 2 * Hkv, d, 11)
    q, k, v = (x[:, :, s].transpose(1, 2) for s in (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, None)))
    kc, vc = (_packed(B, Hkv, Tmax, d, s) for s in (1, 2))
    k0, v0 = kc.clone(), vc.clone()
    (wq, wk), f = _weights(d, 4), fa.rope_inv_freq(32)
    ctx = torch.tensor([0, 1000, 1001, Tmax, -3], dtype=torch.int32)
    y = fa.norm_rope_append(q, k, v, wq, wk, kc, vc, ctx.cuda(), f, interleaved=interleaved)
    for b, c in enumerate(ctx.tolist()):
        pos = (c + torch.arange(n))[None]
        if c < 0:
            assert not y[b].any()
        else:
            _near(y[b:b + 1], _forward(q[b:b + 1], wq, pos, f, interleaved, 1.0, EPS), f"q {b}")
        m = max(0, min(n, Tmax - c)) if c >= 0 else 0
        if m:
            yk, tol = _forward(k[b:b + 1], wk, pos, f, interleaved, 1.0, EPS)
            _near(kc[b:b + 1, :, c:c + m], (yk[:, :, :m], tol[:, :, :m]), f"k {b}")
            k0[b, :, c:c + m], v0[b, :, c:c + m] = kc[b, :, c:c + m], v[b, :, :m]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
