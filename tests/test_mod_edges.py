"""Modified scores and cached contexts at their edges, on the GPU: keys behind a length that is no
multiple of a tile, rows that see one key, padding of any value anywhere, values that are not
numbers, far positions, forms that the other files' sizes do not reach, records of long batches.
Bounds: those of mod_reference.py."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_mod import ALL, _ids, _run, _slopes, _tensors
from tests.test_tree import _check as _check_tree, _data as _tree_data

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- keys behind the sequence's end

def _opposed(B, H, Hkv, T, d, seed):
    """Queries and keys around opposed vectors: every scaled score near −120, of deviation 1."""
    q, k, v, do = (x.float() for x in _tensors(B, H, Hkv, T, d, seed))
    g = torch.Generator().manual_seed(seed + 1)
    u = torch.randint(0, 2, (d,), generator=g) * 2.0 - 1.0        # |u|² = d
    c = 120.0 * d ** -0.5                                         # d^−½ · u·(c·u) = 120
    return [x.to(torch.bfloat16) for x in (u + 0.08 * q, -c * u + 0.5 * k, v, do)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 129, 130, 300])
@pytest.mark.parametrize("cap,slope", [(0.0, None), (200.0, None), (0.0, 0.01), (200.0, 0.01)])
def test_far_below_zero_without_visible(T, d, cap, slope):
    """No mask, and a row's LSE so low that the exponential of a score of 0 against it is infinite:
    the rows of zeros behind the last key must not count."""
    B, H, Hkv = 1, 4, 2
    q, k, v, do = _opposed(B, H, Hkv, T, d, 7 * T + d)
    sl = None if slope is None else torch.full((H,), slope)
    r = ref.attention(q, k, v, ref.visible_mask(B, T, False), d ** -0.5, cap, sl, do)
    assert float(r["lse"].max()) < -89.0
    ref.check(_run(q, k, v, do, causal=False, softcap=cap, slopes=sl), r, ALL)


@pytest.mark.parametrize("d", [64, 128])
def test_far_below_zero_in_the_dense_backward(d):
    for T in (1, 129, 300):
        q, k, v, do = _opposed(1, 2, 2, T, d, 5 * T + d)
        r = ref.attention(q, k, v, ref.visible_mask(1, T, False), d ** -0.5, do=do)
        t = [x.cuda() for x in (q, k, v, do)]
        o, lse = fa.fwd(*t[:3], causal=False)
        got = dict(zip(("dq", "dk", "dv"), fa.bwd(*t[:3], o, lse, t[3], causal=False)))
        ref.check(got, r, ("dq", "dk", "dv"), f"T {T}")


@pytest.mark.parametrize("d", [64, 128])
def test_distances_that_raise_scores(d):
    """A negative slope: keys behind the end would be the farthest and outweigh all others."""
    B, H, Hkv, T = 1, 2, 1, 130
    q, k, v, do = _tensors(B, H, Hkv, T, d, 15)
    sl = torch.tensor([-1.5, -0.25])
    r = ref.attention(q, k, v, ref.visible_mask(B, T, False), d ** -0.5, 0.0, sl, do)
    ref.check(_run(q, k, v, do, causal=False, slopes=sl), r, ALL)


# ------------------------------------------------------------------------ rows that see one key

@pytest.mark.parametrize("with_rest", [False, True])
@pytest.mark.parametrize("B,H,Hkv", [(1, 4, 2), (4, 80, 10)])      # one query tile a CTA, and two
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0, 50.0, 80.0])
def test_a_row_of_one_key_is_its_value(B, H, Hkv, d, cap, with_rest):
    """Documents of one token: the weight is 1, so o is v, to the last bit."""
    T = 260
    q, k, v, _ = _tensors(B, H, Hkv, T, d, 41, 4.0)
    ids = torch.arange(T, dtype=torch.int32).repeat(B, 1)
    seen = fa.visible(B, T, doc_ids=ids.cuda())
    rest = torch.full_like(q, math.nan).cuda() if with_rest else None
    o, _ = fa.fwd_mod(q.cuda(), k.cuda(), v.cuda(), visible=seen, softcap=cap, rest=rest)
    assert torch.equal(o.cpu(), v.repeat_interleave(H // Hkv, 1))
    # What is left of a value: the exponent is a score less its own rounding, 2⁻²⁴ of a score below
    # 64 in base 2, so the weight and with it the sum are within 2⁻¹⁸ of 1.
    assert rest is None or (rest.abs().float() <= 2.0 ** -18 * o.abs().float() + 1e-30).all()


@pytest.mark.parametrize("with_rest", [False, True])
@pytest.mark.parametrize("B,H", [(1, 4), (2, 160)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,sign", [(0.0, 1.0), (50.0, 1.0), (50.0, -1.0), (20.0, 1.0), (80.0, -1.0)])
def test_a_key_that_outweighs_all_others(B, H, d, cap, sign, with_rest):
    """Queries that are their own key, no mask: half a bf16 step of o, of which the outweighing key's
    rounding is no part; the others' rounding goes by their share (twice it, as in mod_reference.py),
    and 2⁻¹⁸ is the fp32 arithmetic's."""
    T = 256
    q, _, v, _ = _tensors(B, H, H, T, d, 45, 2.0)
    k = q if sign > 0 else -q
    scale = sign * 8.0 / d                                         # own scores around 32
    rest = torch.empty_like(q).cuda() if with_rest else None
    o, _ = fa.fwd_mod(q.cuda(), k.cuda(), v.cuda(), causal=False, softcap=cap, scale=scale, rest=rest)
    r = ref.attention(q, k, v, ref.visible_mask(B, T, False), scale, cap)
    own = (q.double() * k.double()).sum(-1) * scale
    own = cap * torch.tanh(own / cap) if cap else own
    others = (1.0 - torch.exp(own - r["lse"]))[..., None] * v.double().abs().amax(2, keepdim=True)
    assert float(others.max()) < 0.5
    bound = (ref.U + 2.0 ** -18) * r["o"].abs() + 2 * ref.U * others
    assert ((o.double().cpu() - r["o"]).abs() <= bound).all()


@pytest.mark.parametrize("n", [9, 40])                             # streaming kernel, tensor cores
@pytest.mark.parametrize("Tmax", [50, 3400])                       # a CTA an entry, and stretches
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0, 50.0, 80.0])
def test_a_token_of_one_key_is_its_value(n, Tmax, d, cap):
    """New tokens that see themselves alone."""
    B, H = 2, 3
    q, k, v = _tree_data(B, H, H, n, Tmax, d, 43, 4.0)
    o, _ = fa.fwd_tree(q.cuda(), k.cuda(), v.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"),
                       tree=torch.eye(n, dtype=torch.uint8).cuda(), softcap=cap)
    assert torch.equal(o.cpu(), v[:, :, :n])


# ----------------------------------------------------------------- padding in front and between

def _gaps(B, T):
    """Padding in front of, between and behind ragged documents, other places in each sequence."""
    rows = []
    for b in range(B):
        row, n = [-1] * (45 + 60 * b), b
        while len(row) < T:
            row += [n % 7] * (3, 90, 131, 40)[n % 4] + [-1] * (1, 17, 130)[n % 3]
            n += 1
        rows.append(row[:T - 20] + [-1] * 20)
    return torch.tensor(rows, dtype=torch.int32)


@pytest.mark.parametrize("with_rest", [False, True])
@pytest.mark.parametrize("B,H,Hkv", [(2, 4, 2), (4, 80, 10)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,cap,bias", [(True, 0.0, False), (False, 0.0, False), (True, 30.0, False),
                                             (False, 80.0, False), (True, 0.0, True), (True, 30.0, True)])
def test_padding_anywhere_may_hold_anything(B, H, Hkv, d, causal, cap, bias, with_rest):
    T = 500
    q, k, v, do = _tensors(B, H, Hkv, T, d, 51, 4.0 if cap else 1.0)
    ids = _gaps(B, T)
    seen = fa.visible(B, T, causal=causal, doc_ids=ids.cuda())
    sl = _slopes(H) if bias else None
    r = ref.attention(q, k, v, ref.visible_mask(B, T, causal, ids), d ** -0.5, cap, sl, do)
    pad = (ids < 0)[:, None, :, None]
    for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (do, -math.inf)):
        x.masked_fill_(pad, bad)
    got = _run(q, k, v, do, seen, softcap=cap, slopes=sl, with_rest=with_rest)
    ref.check(got, r, ALL)
    for n in ("o", "dq", "dk", "dv"):
        assert not got[n].masked_fill(~pad.cuda(), 0.0).any(), n


# ----------------------------------------------------------------------- values that are no numbers

@pytest.mark.parametrize("B,H,Hkv", [(1, 4, 2), (4, 80, 10)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (80.0, False), (0.0, True), (30.0, True)])
def test_a_query_that_is_no_number(B, H, Hkv, d, cap, bias):
    """Its row's o and LSE are none either, as in plain arithmetic; the other rows stay as they are."""
    T = 260
    q, k, v, _ = (x.cuda() for x in _tensors(B, H, Hkv, T, d, 61))
    sl = _slopes(H).cuda() if bias else None
    rows = torch.tensor([0, 77, 140, T - 1], device="cuda")
    o, lse = fa.fwd_mod(q, k, v, softcap=cap, slopes=sl)
    q[:, :, rows, 5] = math.nan
    o2, lse2 = fa.fwd_mod(q, k, v, softcap=cap, slopes=sl)
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[rows] = True
    assert torch.isnan(o2[:, :, hit].float()).all() and torch.isnan(lse2[:, :, hit]).all()
    assert torch.equal(o2[:, :, ~hit], o[:, :, ~hit]) and torch.equal(lse2[:, :, ~hit], lse[:, :, ~hit])


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("Tmax", [150, 3400])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0, 80.0])
def test_a_new_token_that_is_no_number(n, Tmax, d, cap):
    q, k, v = (x.cuda() for x in _tree_data(2, 4, 4, n, Tmax, d, 63))
    ctx = torch.tensor([100, Tmax - n], dtype=torch.int32, device="cuda")
    o, lse = fa.fwd_tree(q, k, v, ctx, softcap=cap)
    q[:, :, 2, 7] = math.nan
    o2, lse2 = fa.fwd_tree(q, k, v, ctx, softcap=cap)
    hit = torch.arange(n, device="cuda") == 2
    assert torch.isnan(o2[:, :, hit].float()).all() and torch.isnan(lse2[:, :, hit]).all()
    assert torch.equal(o2[:, :, ~hit], o[:, :, ~hit]) and torch.equal(lse2[:, :, ~hit], lse[:, :, ~hit])


# ------------------------------------------------------------------------------- far positions

@pytest.mark.parametrize("H", [2, 16])                            # streaming kernel, tensor cores
@pytest.mark.parametrize("d,ctx", [(64, (1 << 25) + 12345), (128, (1 << 24) + 77)])
def test_bias_behind_16_million_keys(H, d, ctx):
    """Positions past 2²⁴, which fp32 cannot tell apart: near keys keep their distances."""
    n, near = 5, 512
    Tmax = ctx + n + 3
    q, k, v = _tree_data(1, H, 1, n, near, d, 71)                 # the last rows of the context and the new ones
    kc, vc = (torch.zeros(1, 1, Tmax, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    first = ctx + n - near
    kc[:, :, first:ctx + n], vc[:, :, first:ctx + n] = k.cuda(), v.cuda()
    sl = torch.tensor([0.5 + 0.1 * h for h in range(H)])          # e^−0.5·507 of what lies before
    dep = torch.tensor([0, 1, 1, 2, 3], dtype=torch.int32)
    tree = torch.eye(n, dtype=torch.uint8)
    tree[3, 0] = tree[4, 0] = tree[4, 3] = 1
    at = ctx + dep.long()[None]
    ka = torch.arange(first, first + near)[None].clone()
    ka[0, near - n:] = at[0]
    ok = torch.ones(1, n, near, dtype=torch.bool)
    ok[0, :, near - n:] = tree.bool()
    r = ref.attention(q, k, v, ok, d ** -0.5, 0.0, sl, query_at=at, key_at=ka)
    o, lse = fa.fwd_tree(q.cuda(), kc, vc, torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                         tree=tree.cuda(), depths=dep.cuda(), slopes=sl.cuda())
    ref.check({"o": o, "lse": lse}, r, ("o", "lse"))


# ------------------------------------------------------------------ forms not reached elsewhere

@pytest.mark.parametrize("T,lengths,pad,prefix,std", [
    (300, (100, 1, 47), 30, "b", 9.0), (384, (300, 9), 140, None, 9.0), (290, (60, 200), 0, "t", 2.0),
])
@pytest.mark.parametrize("d", [64, 128])
def test_capped_inference_on_documents(T, d, lengths, pad, prefix, std):
    """Two query tiles a CTA, capped scores near and far, intervals with both ends, no rest."""
    B, H, Hkv = 4, 80, 10
    q, k, v, do = _tensors(B, H, Hkv, T, d, 29 * T + d, std)
    ids = _ids(B, T, lengths, pad)
    pre = None
    if prefix == "b":
        pre = torch.tensor([60 * b + 7 for b in range(B)], dtype=torch.int32)
    elif prefix == "t":
        pre = ((ids + 2) * 23 - 40).to(torch.int32)
    r = ref.attention(q, k, v, ref.visible_mask(B, T, True, ids, pre), d ** -0.5, 30.0, None, do)
    seen = fa.visible(B, T, doc_ids=ids.cuda(), prefix_len=None if pre is None else pre.cuda())
    ref.check(_run(q, k, v, do, seen, softcap=30.0, with_rest=False), r, ALL)


@pytest.mark.parametrize("room", [0, 3300])
@pytest.mark.parametrize("ctx,H,Hkv,n,Tmax,tree,cap,bias", [
    ([300, 77], 8, 2, 16, 320, True, 30.0, True),       # 64 rows
    ([129, 0, -1], 12, 3, 33, 200, True, 80.0, True),   # 132 rows: two row blocks
    ([500], 5, 5, 48, 560, True, 0.0, True),            # flags in whole 16-byte pieces
    ([63], 5, 5, 50, 130, False, 30.0, True),
    ([200, 31], 4, 1, 64, 270, True, 80.0, False),
])
def test_wide_rows_of_d128(ctx, H, Hkv, n, Tmax, tree, cap, bias, room):
    _check_tree(ctx, H, Hkv, n, Tmax + room, 128, tree, cap, bias, seed=5)


# ------------------------------------------------------------------------ the records of visible

def _records(seen, B, T):
    """(rows, fwd, pairs, bwd) of a Visible's buffer."""
    up = lambda x: (x + 255) // 256 * 256
    n_t = -(-T // 128)
    at, out = 0, []
    for count, width in ((B * n_t * 128, 2), (B * n_t, 4), (B * ((n_t + 1) // 2), 8), (B * n_t, 4)):
        n = count * width * 4
        out.append(seen.buffer[at:at + n].view(torch.int32).view(B, -1, width).cpu().long())
        at += up(n)
    return out


@pytest.mark.parametrize("T,lengths,pad,causal,prefix", [
    (1, (1,), 0, True, False), (129, (40, 50), 3, True, True), (1000, (128, 77), 300, False, False),
    (33000, (1000, 1, 2048), 129, True, True), (200000, (100, 60000, 17), 5000, True, True),
    (200000, (100, 60000, 17), 70000, False, False),
])
def test_walks_of_tiles(T, lengths, pad, causal, prefix):
    """Each query tile's K tiles and each key tile's query tiles, once each, the longest first, made
    from the rows' intervals (which test_mod.py checks); 1563 tiles a sequence at the longest."""
    B = 2
    ids = _ids(B, T, lengths, pad)
    pre = torch.tensor([5, 40000], dtype=torch.int32) if prefix else None
    seen = fa.visible(B, T, causal=causal, doc_ids=ids.cuda(), prefix_len=None if pre is None else pre.cuda())
    rows, fwd, pairs, bwd = _records(seen, B, T)
    n_t = -(-T // 128)
    for b in range(B):
        live = rows[b, :, 1] > rows[b, :, 0]
        padded = torch.tensor([bool((ids[b, 128 * t:128 * (t + 1)] < 0).any()) for t in range(n_t)])
        pad0 = int(padded.nonzero()[0]) if padded.any() else n_t      # the first tile with padding
        lo = torch.where(live, rows[b, :, 0], torch.full_like(rows[b, :, 0], T)).view(n_t, 128).amin(1)
        hi = torch.where(live, rows[b, :, 1], torch.zeros_like(rows[b, :, 1])).view(n_t, 128).amax(1)
        some = hi > lo
        zero = torch.zeros_like(lo)
        k0, k1 = torch.where(some, lo // 128, zero), torch.where(some, (hi + 127) // 128, zero)
        tile = torch.arange(n_t)
        assert torch.equal(fwd[b, :, 0].sort().values, tile)
        assert torch.equal(fwd[b, :, 1], k0[fwd[b, :, 0]]) and torch.equal(fwd[b, :, 2], k1[fwd[b, :, 0]])
        assert (fwd[b, :, 3] == pad0).all()
        n = fwd[b, :, 2] - fwd[b, :, 1]
        assert (n[1:] <= n[:-1]).all()
        # key tiles: the query tiles whose K tiles hold them
        meets = some[None] & (lo[None] < 128 * (tile[:, None] + 1)) & (hi[None] > 128 * tile[:, None])
        q0 = torch.where(meets, tile[None], torch.full_like(tile[None], n_t)).amin(1)
        q1 = torch.where(meets, tile[None] + 1, torch.zeros_like(tile[None])).amax(1)
        q0 = torch.where(q1 > 0, q0, zero)
        assert torch.equal(bwd[b, :, 0].sort().values, tile)
        assert torch.equal(bwd[b, :, 1], q0[bwd[b, :, 0]]) and torch.equal(bwd[b, :, 2], q1[bwd[b, :, 0]])
        assert torch.equal(bwd[b, :, 3], 2 * pad0 + padded.long()[bwd[b, :, 0]])
        n = bwd[b, :, 2] - bwd[b, :, 1]
        assert (n[1:] <= n[:-1]).all()
        # pairs
        n_p = (n_t + 1) // 2
        first = pairs[b, :, 0]
        assert torch.equal(first.sort().values, 2 * torch.arange(n_p)) and (pairs[b, :, 1] == pad0).all()
        k0, k1 = (torch.cat((x, torch.zeros(1, dtype=x.dtype))) for x in (k0, k1))
        for i, (a, z) in enumerate(((2, 3), (4, 5))):
            assert torch.equal(pairs[b, :, a], k0[first + i]) and torch.equal(pairs[b, :, z], k1[first + i])
        empty = [k1[first + i] == k0[first + i] for i in (0, 1)]
        big = torch.full_like(first, 1 << 30)
        start = torch.minimum(*(torch.where(e, big, k0[first + i]) for i, e in enumerate(empty)))
        stop = torch.maximum(*(torch.where(e, torch.zeros_like(big), k1[first + i]) for i, e in enumerate(empty)))
        n = (stop - start).clamp(min=0)
        assert (n[1:] <= n[:-1]).all()
