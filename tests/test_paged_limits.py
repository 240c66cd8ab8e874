"""The size limits that the header states for the rotary and paged-cache calls, at both sides (CPU: the workspace's check comes last)."""
from __future__ import annotations

import ctypes

import pytest

import sliding_window_gqa_gb300 as wa
from _util import ensure_built
from test_paged_checks import FAKE, _append, _decode, _rot


@pytest.mark.parametrize("fits, cache, hq", [
    (True, dict(rows=65535), 16), (False, dict(rows=65536), 16),
    (True, dict(page_size=16, most=2 ** 27 - 257, table_row=2 ** 27), 16), (False, dict(page_size=16, most=2 ** 27 - 256, table_row=2 ** 27), 16),
    (True, dict(page_size=256, k_page=256 * 2048, v_page=256 * 2048, most=2 ** 23 - 17, table_row=2 ** 23), 16),
    (False, dict(page_size=256, k_page=256 * 2048, v_page=256 * 2048, most=2 ** 23 - 16, table_row=2 ** 23), 16),
], ids=str)
def test_rows_and_positions(fits, cache, hq):
    want = wa.WA_EWORKSPACE if fits else wa.WA_EINVAL
    assert _append(cache=cache, hq=hq, ws=None) == _decode(cache=cache, hq=hq, ws=None) == want


def test_heads_of_a_rotation():
    L = ensure_built().lib()
    for heads in (65536, 1 << 20):
        assert L.wa_rope(FAKE, FAKE, 1, heads, 128, ctypes.byref(_rot(dims=128)), 0, heads * 128, heads * 128, FAKE + (1 << 40), None) == wa.WA_EINVAL


def test_rows_times_heads():
    """16 heads a key head: rows * hq below 2^31."""
    for hkv, fits in ((2047, True), (2049, False)):
        c = dict(rows=65535, hkv=hkv, d=128, **{f"{s}_{n}": v for s in "kv" for n, v in (("head", 128), ("slot", hkv * 128), ("page", 16 * hkv * 128))})
        assert _decode(cache=c, hq=16 * hkv, q_row=16 * hkv * 128, out_row=16 * hkv * 128, ws=None) == (wa.WA_EWORKSPACE if fits else wa.WA_EINVAL)
        assert wa.paged_decode_ws_bytes(65535, 16 * hkv, hkv, 128, 16, 7) > 0 if fits else \
            wa.paged_decode_ws_bytes(65535, 16 * hkv, hkv, 128, 16, 7) == 0
