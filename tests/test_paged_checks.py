"""Refusals of the rotary and paged-cache calls: the C ABI's argument errors and the binding's (CPU, before any CUDA call)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sliding_window_gqa_gb300 as wa
from _util import ensure_built

FAKE, ODD = 1 << 20, (1 << 20) + 2     # never dereferenced: validation fails first


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE + (1 << 30), k_scale=None, v_scale=None, table=FAKE, pages=10, page_size=16, rows=3, most=7,
             hkv=8, d=256, type=0, table_row=7)
    a.update({s: v for n, v in (("page", 16 * 2048), ("slot", 2048), ("head", 256)) for s, v in ((f"k_{n}", v), (f"v_{n}", v))})
    a.update(kw)
    return wa._Pages(**a)


def _rot(**kw):
    return wa._Rotary(**dict(dict(inv_freq=FAKE, dims=256, layout=0, factor=1.0), **kw))


def _append(cache=None, rot=None, **kw):
    L = ensure_built().lib()
    a = dict(src=FAKE, pos=FAKE, row=None, n=3, hq=16, src_tok=32 * 256, q_tok=16 * 256, q=FAKE + (1 << 28), ws=FAKE, ws_bytes=256)
    a.update(kw)
    c = _cache(**(cache or {}))
    return L.wa_paged_append(a["src"], a["pos"], a["row"], a["n"], a["hq"], ctypes.byref(c), ctypes.byref(_rot(**(rot or {}))),
                             a["src_tok"], a["q_tok"], a["q"], a["ws"], a["ws_bytes"], None)


def _decode(cache=None, **kw):
    L = ensure_built().lib()
    a = dict(q=FAKE, pos=FAKE, hq=16, win=0, scale=1.0, q_row=16 * 256, out_row=16 * 256, out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    c = _cache(**(cache or {}))
    return L.wa_paged_decode(a["q"], a["pos"], a["hq"], ctypes.byref(c), a["win"], a["scale"], a["q_row"], a["out_row"], a["out"],
                             a["ws"], a["ws_bytes"], None)


CACHES = [dict(k=None), dict(v=None), dict(table=None), dict(k=ODD), dict(v=FAKE + 8), dict(table=ODD), dict(pages=0),
          dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=512), dict(rows=0), dict(rows=65536),
          dict(most=0), dict(most=1 << 27, table_row=1 << 27), dict(hkv=0), dict(hkv=3), dict(d=64), dict(d=192), dict(type=2), dict(type=-1),
          dict(k_scale=FAKE), dict(v_scale=FAKE), dict(table_row=6), dict(k_page=16 * 2048 - 8), dict(k_slot=0),
          dict(v_head=128), dict(v_slot=2044), dict(k_head=-256), dict(type=1, k_slot=2056), dict(k_page=1 << 45)]


@pytest.mark.parametrize("bad", CACHES, ids=str)
def test_caches_that_are_refused(bad):
    assert _append(cache=bad) == wa.WA_EINVAL
    assert _decode(cache=bad) == wa.WA_EINVAL


@pytest.mark.parametrize("bad", [
    dict(src=None), dict(pos=None), dict(q=None), dict(n=0), dict(n=-1), dict(n=4), dict(hq=12), dict(hq=136), dict(hq=0),
    dict(src=ODD), dict(q=ODD), dict(src_tok=32 * 256 + 4), dict(q_tok=100), dict(src_tok=31 * 256), dict(q_tok=15 * 256),
    dict(q=FAKE), dict(cache=dict(k=FAKE, v=FAKE)), dict(rot=dict(inv_freq=None)), dict(rot=dict(dims=8)),
    dict(rot=dict(dims=272)), dict(rot=dict(dims=-16)), dict(rot=dict(layout=2)), dict(rot=dict(factor=float("nan"))),
], ids=str)
def test_append_argument_errors(bad):
    assert _append(**bad) == wa.WA_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(pos=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(hq=12), dict(hq=136), dict(win=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q_row=15 * 256), dict(out_row=16 * 256 + 4), dict(out_row=0),
    dict(cache=dict(k_page=16 * 2048 + 8)),       # neither a multiple of 8 slots nor of a head
], ids=str)
def test_decode_argument_errors(bad):
    assert _decode(**bad) == wa.WA_EINVAL


def test_a_lone_head_may_have_any_head_stride():
    """(There is no other head to be apart from.  The checks before the workspace pass, without a division by it.)"""
    for stride in (0, -256, 256, 1 << 50):
        c = dict(hkv=1, **{f"{s}_{n}": v for s in "kv" for n, v in (("head", stride), ("slot", 256), ("page", 16 * 256 + 256))})
        assert _decode(cache=c, hq=2, ws=None) == wa.WA_EWORKSPACE
        assert _append(cache=c, hq=2, ws=None) == wa.WA_EWORKSPACE
        c["k_page"] += 8                  # a multiple of neither
        assert _decode(cache=c, hq=2, ws=None) == wa.WA_EINVAL


def test_workspace_errors():
    L = ensure_built().lib()
    assert _append(ws=None) == _append(ws_bytes=255) == _append(ws=FAKE + 128) == wa.WA_EWORKSPACE
    need = L.wa_paged_decode_ws_bytes(ctypes.byref(_cache()), 16, 0)
    assert need > 256
    assert _decode(ws=None) == _decode(ws_bytes=need - 1) == _decode(ws=FAKE + 128) == wa.WA_EWORKSPACE


def test_ws_bytes_of_invalid_sizes():
    assert wa.paged_decode_ws_bytes(3, 16, 8, 256, 16, 7) > 0
    for size in [(0, 16, 8, 256, 16, 7), (3, 17, 8, 256, 16, 7), (3, 16, 8, 192, 16, 7), (3, 16, 8, 256, 17, 7), (3, 16, 8, 256, 16, 0),
                 (3, 16, 8, 256, 16, 7, -1), (3, 16, 8, 256, 16, 2 ** 31), (3, 16, 8, 256, 16, 7, 0, torch.float16)]:
        assert wa.paged_decode_ws_bytes(*size) == 0


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(pos=None), dict(out=None), dict(rot=dict(inv_freq=None)), dict(rot=dict(dims=24)), dict(n=0), dict(heads=0),
    dict(d=64), dict(inverse=2), dict(x=ODD), dict(out=ODD), dict(x_tok=4 * 128 - 8), dict(out_tok=4 * 128 + 4), dict(x_tok=1024, out=FAKE),
], ids=str)
def test_rope_argument_errors(bad):
    L = ensure_built().lib()
    a = dict(x=FAKE, pos=FAKE, n=5, heads=4, d=128, inverse=0, x_tok=512, out_tok=512, out=FAKE + (1 << 28), rot={})
    a.update(bad)
    rot = _rot(**dict(dict(dims=128), **a["rot"]))
    assert L.wa_rope(a["x"], a["pos"], a["n"], a["heads"], a["d"], ctypes.byref(rot), a["inverse"], a["x_tok"], a["out_tok"],
                     a["out"], None) == wa.WA_EINVAL


# ---- the binding, by tensors that claim to be on the GPU

class Cuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA one: every check passes or fails before a pointer is used."""

    @property
    def is_cuda(self):
        return True


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape).to(dtype).as_subclass(Cuda)


def _good():
    return dict(src=_t(3, 12 * 128), pos=_t(3, dtype=torch.int32), q_out=_t(3, 8, 128), k_pages=_t(5, 16, 2, 128),
                v_pages=_t(5, 16, 2, 128), table=_t(3, 4, dtype=torch.int32))


@pytest.mark.parametrize("bad, error", [
    (dict(src=_t(3, 12 * 128, dtype=torch.float16)), TypeError), (dict(src=_t(3, 12 * 128 - 8)), ValueError),
    (dict(src=_t(12 * 128, 3).T), ValueError), (dict(q_out=_t(4, 8, 128)), ValueError), (dict(q_out=_t(3, 8, 256)), ValueError),
    (dict(q_out=_t(3, 8 * 128)), ValueError), (dict(pos=_t(3, dtype=torch.int64)), TypeError), (dict(pos=_t(4, dtype=torch.int32)), ValueError),
    (dict(k_pages=_t(5, 16, 2, 128, dtype=torch.float16)), TypeError), (dict(v_pages=_t(5, 16, 2, 128, dtype=torch.float8_e4m3fn)), ValueError),
    (dict(v_pages=_t(4, 16, 2, 128)), ValueError), (dict(k_pages=_t(5, 16, 256)), ValueError),
    (dict(table=_t(3, 4, dtype=torch.int64)), TypeError), (dict(table=_t(4, 3, dtype=torch.int32).T), ValueError),
    (dict(table=_t(2, 4, dtype=torch.int32)), ValueError), (dict(row=_t(2, dtype=torch.int32)), ValueError),
    (dict(inv_freq=_t(60, dtype=torch.float32)), ValueError), (dict(inv_freq=_t(72, dtype=torch.float32)), ValueError),
    (dict(inv_freq=_t(64)), TypeError), (dict(inv_freq=_t(0, dtype=torch.float32)), ValueError), (dict(layout="pairs"), ValueError),
    (dict(inv_freq=_t(64, dtype=torch.float32), factor=float("nan")), ValueError), (dict(factor="1"), TypeError),
    (dict(k_scale=_t(2, dtype=torch.float32)), ValueError), (dict(src=_t(1, 12 * 128).expand(3, -1)), ValueError),
], ids=lambda x: next(iter(x)) if isinstance(x, dict) else x.__name__)
def test_append_refuses_tensors_that_disagree(bad, error):
    with pytest.raises(error):
        wa.paged_append(**dict(_good(), **bad))


@pytest.mark.parametrize("bad, error", [
    (dict(q=_t(3, 8, 128, dtype=torch.float32)), TypeError), (dict(q=_t(4, 8, 128)), ValueError), (dict(q=_t(3, 8, 256)), ValueError),
    (dict(q=_t(3, 128, 8).transpose(1, 2)), ValueError), (dict(pos=_t(4, dtype=torch.int32)), ValueError), (dict(out=_t(3, 4, 128)), ValueError),
    (dict(out=_t(1, 8, 128).expand(3, -1, -1)), ValueError), (dict(win=1.5), ValueError), (dict(win=2 ** 31), ValueError), (dict(win="1"), TypeError),
    (dict(scale="1"), TypeError), (dict(k_pages=_t(5, 16, 128, 2).transpose(2, 3)), ValueError), (dict(v_scale=_t(2, dtype=torch.float32)), ValueError),
], ids=lambda x: next(iter(x)) if isinstance(x, dict) else x.__name__)
def test_decode_refuses_tensors_that_disagree(bad, error):
    g = _good()
    with pytest.raises(error):
        wa.paged_decode(**dict(dict(q=_t(3, 8, 128), k_pages=g["k_pages"], v_pages=g["v_pages"], table=g["table"], pos=g["pos"]), **bad))


def test_scales_of_8_bit_pages_are_checked():
    g = _good()
    pages = _t(5, 16, 2, 128, dtype=torch.float8_e4m3fn)
    for bad, error in ((_t(3, dtype=torch.float32), ValueError), (_t(2, dtype=torch.float64), TypeError)):
        with pytest.raises(error):
            wa.paged_decode(_t(3, 8, 128), pages, pages, g["table"], g["pos"], k_scale=bad)


def test_tensors_on_the_cpu_are_refused():
    g = {n: t.as_subclass(torch.Tensor) for n, t in _good().items()}
    with pytest.raises(TypeError):
        wa.paged_append(**g)
    with pytest.raises(TypeError):
        wa.paged_decode(torch.zeros(3, 8, 128, dtype=torch.bfloat16), g["k_pages"], g["v_pages"], g["table"], g["pos"])
    with pytest.raises(TypeError):
        wa.rope(torch.zeros(3, 8, 128, dtype=torch.bfloat16), g["pos"], torch.zeros(64))


@pytest.mark.parametrize("bad, error", [
    (dict(x=_t(5, 4 * 128)), ValueError), (dict(x=_t(5, 4, 128, dtype=torch.float32)), TypeError), (dict(pos=_t(4, dtype=torch.int32)), ValueError),
    (dict(inv_freq=None), TypeError), (dict(inv_freq=_t(65, dtype=torch.float32)), ValueError), (dict(layout=None), ValueError),
    (dict(out=_t(5, 3, 128)), ValueError), (dict(x=_t(1, 4, 128).expand(5, -1, -1)), ValueError), (dict(factor=float("inf")), ValueError),
], ids=lambda x: next(iter(x)) if isinstance(x, dict) else x.__name__)
def test_rope_refuses_tensors_that_disagree(bad, error):
    a = dict(x=_t(5, 4, 128), pos=_t(5, dtype=torch.int32), inv_freq=_t(64, dtype=torch.float32))
    with pytest.raises(error):
        wa.rope(**dict(a, **bad))
