"""The rule by which a cache's entries go to a CTA each (fwd_tree without workspace) or are cut into
stretches: by the chunks that either leaves a CTA, on a GPU of 152 SMs."""

import pytest

import exact_attention_23_gb300 as fa


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,Tq,d,chunk,fit,least,join,most", [
    (8, 1, 1, 1, 64, 64, 456, 2, 7, 24), (8, 12, 12, 1, 64, 64, 456, 2, 7, 24),
    (38, 12, 12, 1, 64, 64, 456, 2, 7, 24), (39, 12, 12, 1, 64, 64, 456, 2, 7, 24),
    (8, 16, 4, 8, 64, 64, 456, 2, 7, 24), (2, 4, 4, 1, 128, 64, 304, 2, 5, 24),
    (8, 12, 12, 2, 128, 64, 304, 2, 5, 24), (8, 16, 4, 64, 64, 128, 152, 1, 5, 12),
    (2, 4, 1, 16, 128, 128, 152, 1, 4, 12), (4, 64, 16, 16, 128, 128, 152, 1, 4, 12),
])
def test_whole_entries(B, H, Hkv, Tq, d, chunk, fit, least, join, most):
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the sizes below are those of 152 SMs")
    R = H // Hkv * Tq
    entries = B * Hkv * (-(-R // 128) if R > 32 else 1)
    for chunks in range(1, 40):
        per = max(least, -(-entries * chunks // fit))              # chunks of a stretch
        whole = entries <= fit and chunks <= min(per + join, most)
        n = fa.fa_fwd_tree_workspace_size(B, H, Hkv, Tq, chunks * chunk, d)
        assert (n == 1) == whole, (chunks, n)
