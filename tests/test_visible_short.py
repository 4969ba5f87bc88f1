"""The visibility of up to 4096 tokens, which has a kernel of its own, row by row and record by record (shorter ones
have no walks in pieces; the parity tests run on them)."""

import pytest

from tests import test_window


@pytest.mark.gpu
@pytest.mark.parametrize("T,lengths,window,sinks", [
    (1025, (900,), 1, 1), (1500, (30, 1, 700), 33, 4), (2049, (2000, 3), 100, 130), (4095, (4000,), 64, 9),
    (4096, (3000, 1, 20), 300, 1024), (4096, (17,), 900, 4)])
def test_visible_rows_of_short_sequences(T, lengths, window, sinks):
    test_window.test_visible_rows(T, lengths, window, sinks)
