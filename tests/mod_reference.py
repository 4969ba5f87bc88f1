"""Plain 64-bit reference of attention with modified scores and its gradients, with the error
bounds that the tests compare under. Elementary torch operations in float64; shares no code with
the kernels.

Bounds (u = 2⁻⁸, half a bf16 step relative to the value):
  o    the output's rounding, u·|o|, and P rounded to bf16 before its product: u·Σ_j p_j|v_j|
       (twice that, for the fp32 arithmetic in between)
  lse  fp32: a dot product of d terms, d·2⁻²⁴·Σ|q_c k_c|·|scale|; the cap's error, at most
       1.0e-6·tanh(0.8)·cap = 2⁻²⁰·⁵ of the cap where it is a polynomial (relative error 1.0e-6)
       and 2⁻²¹ beyond, with three fp32 roundings at most 2⁻²⁰ in all; the bias, 2⁻²¹ of its size; the sum of exponentials and its logarithm
  dV   u·|dV| + 2u·Pᵀ|dO|
  dQ   u·|dQ| + 2u·|scale|·M|K|, dK likewise with Mᵀ|Q|, where M = P·(1 − tanh²)·(|dP − D| +
       Σ_c|dO_c O_c|) bounds dS's own rounding and D's error, made from the rounded o
Gradients get 1e-6 on top (values that cancel to nothing).
"""

import math

import torch

U = 2.0 ** -8


def visible_mask(B, T, causal, doc_ids=None, prefix_len=None):
    """[B, T, T] truth values by the definition, one pair at a time in spirit: same maximal run of
    equal non-negative ids, and (causal) at or before the query or in its document's prefix."""
    ok = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        ids = [0] * T if doc_ids is None else doc_ids[b].tolist()
        s = 0
        while s < T:
            e = s
            while e < T and ids[e] == ids[s]:
                e += 1
            if ids[s] >= 0:
                for i in range(s, e):
                    if not causal:
                        ok[b, i, s:e] = True
                    else:
                        n = 0
                        if prefix_len is not None:
                            n = int(prefix_len[b]) if prefix_len.dim() == 1 else int(prefix_len[b, i])
                        ok[b, i, s:max(i + 1, min(e, s + max(0, n)))] = True
            s = e
    return ok


def attention(q, k, v, ok, scale, softcap=0.0, slopes=None, do=None, query_at=None, key_at=None):
    """q [B, H, Tq, d], k, v [B, Hkv, Tk, d] (any float type), ok [B, Tq, Tk]; query_at and key_at
    ([B, Tq], [B, Tk]) are the positions the bias measures between (default: the indices).
    Returns a dict of float64 results and of bounds under the same names with "_tol"."""
    q, k, v = q.double(), k.double(), v.double()
    B, H, Tq, d = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    G = H // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    raw = q @ kk.transpose(-1, -2)
    mag = q.abs() @ kk.abs().transpose(-1, -2) * abs(scale)
    z = raw * scale
    bend = torch.ones_like(z)
    if softcap:
        th = torch.tanh(z / softcap)
        z, bend = softcap * th, 1 - th * th
    dist = torch.zeros_like(z)
    if slopes is not None:
        qa = torch.arange(Tq).expand(B, Tq) if query_at is None else query_at
        ka = torch.arange(Tk).expand(B, Tk) if key_at is None else key_at
        dist = slopes.double().view(1, H, 1, 1) * (qa[:, :, None] - ka[:, None, :]).abs()[:, None].double()
        z = z - dist
    ok = ok[:, None].expand(B, H, Tq, Tk)
    z = torch.where(ok, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    live = m > -math.inf
    p = torch.where(ok, torch.exp(z - torch.where(live, m, torch.zeros_like(m))), torch.zeros_like(z))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(live, l, torch.ones_like(l))
    lse = torch.where(live, m + torch.log(torch.where(live, l, torch.ones_like(l))), m).squeeze(-1)
    o = p @ vv
    r = {"o": o, "lse": lse, "o_tol": U * o.abs() + 2 * U * (p @ vv.abs()) + 1e-7}
    zero = torch.zeros_like(mag)
    worst = torch.where(ok, mag, zero).amax(-1)
    r["lse_tol"] = (d * 2.0 ** -24 + 2.0 ** -21) * worst + softcap * 2.0 ** -20 + 1e-5 \
        + 2.0 ** -21 * torch.where(ok, dist.abs(), zero).amax(-1)
    if do is None:
        return r
    do = do.double()
    dp = do @ vv.transpose(-1, -2)
    D = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - D) * bend
    M = p * bend * ((dp - D).abs() + (do * o).abs().sum(-1, keepdim=True))
    sq = lambda x: x.view(B, Hkv, G, Tk, d).sum(2)
    r["dv"] = sq(p.transpose(-1, -2) @ do)
    r["dv_tol"] = U * r["dv"].abs() + 2 * U * sq(p.transpose(-1, -2) @ do.abs()) + 1e-6
    r["dq"] = scale * (ds @ kk)
    r["dq_tol"] = U * r["dq"].abs() + 2 * U * abs(scale) * (M @ kk.abs()) + 1e-6
    r["dk"] = scale * sq(ds.transpose(-1, -2) @ q)
    r["dk_tol"] = U * r["dk"].abs() + 2 * U * abs(scale) * sq(M.transpose(-1, -2) @ q.abs()) + 1e-6
    return r


def check(got, ref, names, what=""):
    for n in names:
        x = got[n].double().cpu()
        y, tol = ref[n], ref[n + "_tol"]
        fine = torch.isfinite(y)
        assert torch.equal(torch.isfinite(x), fine), f"{what} {n}: where it is finite"
        assert torch.equal(x[~fine], y[~fine]), f"{what} {n}: infinities"
        ratio = ((x[fine] - y[fine]).abs() / tol[fine])
        worst = float(ratio.max()) if ratio.numel() else 0.0
        assert worst <= 1.0, f"{what} {n}: error / bound {worst:.3f}"
