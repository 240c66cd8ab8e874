"""Sizes of the paged decode's workspace (CPU)."""
from __future__ import annotations

import pytest
import torch

from _util import ensure_built


@pytest.mark.parametrize("hq, hkv, d, most, win, dtype", [(64, 8, 128, 8192, 0, torch.bfloat16), (16, 1, 256, 640, 0, torch.float8_e4m3fn),
                                                         (32, 16, 256, 100000, 1024, torch.bfloat16), (1, 1, 128, 1, 0, torch.bfloat16)], ids=str)
def test_rows_beyond_256_take_the_same_partial_results(hq, hkv, d, most, win, dtype):
    """Partial results of 256 rows are held at a time, or of as many as 64 MiB take: more rows add what a call counts alone, 21
    bytes a row at most."""
    wa = ensure_built()
    size = lambda rows: wa.paged_decode_ws_bytes(rows, hq, hkv, d, 16, most, win, dtype)   # noqa: E731
    for rows in (257, 512, 4096, 65535):
        assert size(256) <= size(rows) <= max(size(256), 1 << 26) + 21 * rows + 1024
    assert size(128) < size(256)


def test_what_a_row_takes():
    """As the header says: (d + 5) floats a query head for each span that a row of the table's width, or of the window, may have."""
    wa = ensure_built()
    for hq, hkv, d, page, most, win, spans in [(32, 8, 128, 16, 1024, 0, 25), (32, 8, 128, 16, 8, 0, 1), (32, 4, 128, 64, 4096, 0, 275),
                                               (16, 1, 256, 16, 100000, 1000, 8)]:
        got = wa.paged_decode_ws_bytes(256, hq, hkv, d, page, most, win) - wa.paged_decode_ws_bytes(1, hq, hkv, d, page, most, win)
        assert abs(got - 255 * 4 * (d + 5) * hq * spans) <= 21 * 256 + 1024, (hq, hkv, d, page, most, win)
