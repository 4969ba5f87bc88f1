"""Gradients of head norms for rows at the end of fp32's range (norm_rope_bwd)."""

import math

import pytest
import torch

import exact_attention_23_gb300 as fa
from tests.test_norm import EPS, _backward, _near, _weights


def _rows(d, heads, T, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(1, heads, T, d, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_squares_pass_the_range(d, interleaved):
    """Finite rows whose Σ x² is no fp32 number: zeros forward, so n = 0, dx = 0 and nothing for dw, also
    where Σ h·w·x is none either; the rows beside them, of the same warp, are what they are without them."""
    x, up = _rows(d, 2, 9, d), _rows(d, 2, 9, 5)
    big = [1, 4, 7]
    for t, size in zip(big, (2.0 ** 64, 2.0 ** 120, 2.0 ** 127)):
        x[:, :, t] = (x[:, :, t].float().sign() + (x[:, :, t] == 0)) * size
    w, f = _weights(d, 1)[0], fa.rope_inv_freq(d)
    y, _ = fa.norm_rope(x, None, w, None, f, interleaved=interleaved)
    dx, _, dw, _ = fa.norm_rope_bwd(up, None, x, None, w, None, f, interleaved=interleaved)
    assert not y[:, :, big].any() and not dx[:, :, big].any()
    rest = [t for t in range(9) if t not in big]
    rows, sums = _backward(up[:, :, rest], x[:, :, rest], w, torch.tensor(rest)[None], f, interleaved, 1.0, EPS)
    _near(dx[:, :, rest], rows, "dx")
    _near(dw, sums, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_products_that_pass_the_range(d):
    """Σ x² is an fp32 number, Σ h·w·x is none, Σ h·w·n is one again."""
    x, up = _rows(d, 2, 5, d + 1), _rows(d, 2, 5, 6)
    x[:, :, 2] *= 2.0 ** 50
    up[:, :, 2] = up[:, :, 2].abs() * 2.0 ** 80
    x[:, :, 2] = x[:, :, 2].abs()
    w, f = _weights(d, 2)[0].abs(), fa.rope_inv_freq(16)
    pos = torch.zeros(5, dtype=torch.int32)                # (no turn: every product has the same sign)
    dx, _, dw, _ = fa.norm_rope_bwd(up, None, x, None, w, None, f, positions=pos.cuda())
    rows, sums = _backward(up, x, w, pos[None], f, False, 1.0, EPS)
    _near(dx, rows, "dx")
    _near(dw, sums, "dw")


@pytest.mark.gpu
def test_what_is_no_number_stays_in_its_row():
    x, up = _rows(64, 1, 6, 3), _rows(64, 1, 6, 4)
    x[0, 0, 1, 9], x[0, 0, 3, 40], up[0, 0, 4, 2] = math.nan, math.inf, math.nan
    w, f = _weights(64, 3)[0], fa.rope_inv_freq(64)
    dx, _, dw, _ = fa.norm_rope_bwd(up, None, x, None, w, None, f)
    assert all(dx[0, 0, t].isnan().all() for t in (1, 3, 4)) and dw.isnan().any()
    fine = [0, 2, 5]
    rows, _ = _backward(up[:, :, fine], x[:, :, fine], w, torch.tensor(fine)[None], f, False, 1.0, EPS)
    _near(dx[:, :, fine], rows, "dx")
