"""The windowed backward where its units go out in several groups of heads, the last a short one, with walks
of sinks in pieces: gradients bit for bit those of calls on few heads (one group), which the 64-bit reference
checks."""

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_mod import ALL, _tensors
from tests.test_window import window_mask


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d,cap", [
    (35, 35, 128, 0.0),     # 70 heads in groups of 22
    (35, 35, 64, 30.0),     # of 44
    (70, 35, 128, 0.0),     # pairs of heads on a key head, groups of 11
])
def test_groups_of_heads(H, Hkv, d, cap):
    B, T, window, sinks = 2, 2900, 100, 4
    q, k, v, do = (x.cuda() for x in _tensors(B, H, Hkv, T, d, 21, 4.0 if cap else 1.0))
    G = H // Hkv
    seen = fa.visible(B, T, window=window, sinks=sinks, device="cuda")
    rest = torch.empty_like(q)
    o, lse = fa.fwd_mod(q, k, v, visible=seen, softcap=cap, rest=rest)
    dq, dk, dv = fa.bwd_mod(q, k, v, o, lse, do, visible=seen, softcap=cap, rest=rest)
    one = fa.visible(1, T, window=window, sinks=sinks, device="cuda")
    for b, h in ((0, 0), (0, 21), (0, 22), (0, 34), (1, 8), (1, 9), (1, 34)):
        # (few heads are cut into parts where they share keys, with sums in another order: so by the same number)
        n = 20 if G > 1 else 1
        h = min(h, Hkv - n)
        ks, qs = slice(h, h + n), slice(h * G, (h + n) * G)
        take = lambda x, s: x[b:b + 1, s].contiguous()
        part = fa.bwd_mod(take(q, qs), take(k, ks), take(v, ks), take(o, qs), take(lse, qs), take(do, qs), visible=one,
                          softcap=cap, rest=take(rest, qs))
        assert torch.equal(part[1], take(dk, ks)) and torch.equal(part[2], take(dv, ks)), (b, h)
    # two key heads of either sequence, of the first and the last group, against the reference
    mask = window_mask(1, T, window, sinks)
    for b, h in ((0, 3), (1, Hkv - 1)):
        c = lambda x, s: x[b:b + 1, s].cpu()
        qs, ks = slice(h * G, (h + 1) * G), slice(h, h + 1)
        r = ref.attention(c(q, qs), c(k, ks), c(v, ks), mask, d ** -0.5, cap, None, c(do, qs))
        ref.check(dict(o=c(o, qs), lse=c(lse, qs), dq=c(dq, qs), dk=c(dk, ks), dv=c(dv, ks)), r, ALL)
