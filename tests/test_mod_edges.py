"""Modified scores and cached contexts at their edges, on the GPU: keys behind a length that is no
multiple of a tile. Bounds: those of mod_reference.py."""

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests import mod_reference as ref
from tests.test_mod import ALL, _run, _tensors

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
