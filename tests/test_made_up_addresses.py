"""No test may start a kernel on made-up addresses: refusals whose call a GPU would carry out are skipped there."""

import types

import pytest
import torch

from tests import conftest


def _items():
    out = []
    for name, path, kw in (("test_tree_refusals", "tests/test_window.py", dict(window=4000, ws=0)),
                           ("test_tree_refusals", "tests/test_window.py", dict(window=4000, ws_bytes=64)),
                           ("test_tree_refusals", "tests/test_window.py", dict(window=0)),
                           ("test_tree_refusals", "tests/test_tree.py", dict(ws=0)),
                           ("test_parity", "tests/test_window.py", dict(ws=0))):
        marks = []
        out.append(types.SimpleNamespace(originalname=name, nodeid=f"{path}::{name}[x]", keywords={}, marks=marks,
                                         callspec=types.SimpleNamespace(params={"kw": kw}), add_marker=marks.append))
    return out


@pytest.mark.parametrize("gpu,skipped", [(True, [True, True, False, False, False]), (False, [False] * 5)])
def test_refusals_that_are_valid_on_a_gpu_do_not_run_there(monkeypatch, gpu, skipped):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = _items()
    conftest.pytest_collection_modifyitems(None, items)
    assert [bool(i.marks) for i in items] == skipped
