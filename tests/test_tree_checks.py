"""Refusals of the calls for drafted tokens: the C ABI's argument errors and the binding's (CPU, before any CUDA call)."""
from __future__ import annotations

import ctypes
import warnings

import numpy as np
import pytest
import torch

import sliding_window_gqa_gb300 as wa
from _util import ensure_built

FAKE = ctypes.c_void_p(1 << 20)    # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _decode(**kw):
    L = ensure_built().lib()
    a = dict(q=FAKE, k=FAKE, v=FAKE, kt=FAKE, vt=FAKE, pos=FAKE, parent=FAKE, n=None, rows=3, nodes=8, hq=16, hkv=8,
             d=256, win=1024, ring=1536, scale=1.0, st=None, out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    st = None if a["st"] is None else ctypes.byref(wa._TreeStrides(**a["st"]))
    return L.wa_tree_decode(a["q"], a["k"], a["v"], a["kt"], a["vt"], a["pos"], a["parent"], a["n"], a["rows"],
                            a["nodes"], a["hq"], a["hkv"], a["d"], a["win"], a["ring"], a["scale"], st, a["out"],
                            a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(kt=None), dict(pos=None), dict(parent=None), dict(out=None), dict(rows=0), dict(rows=65536),
    dict(nodes=0), dict(nodes=129), dict(hq=12), dict(hq=136), dict(d=192), dict(d=64), dict(win=-1), dict(win=1537),
    dict(ring=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=ODD), dict(kt=ODD), dict(out=ODD),
    dict(st=dict(q_tok=100)), dict(st=dict(q_tok=16 * 256 + 4)), dict(st=dict(k_row=8)), dict(st=dict(v_tok=-2048)),
    dict(st=dict(out_row=-8)), dict(rows=60000, nodes=128, hq=512, hkv=512, d=128),
], ids=str)
def test_tree_decode_argument_errors(bad):
    assert _decode(**bad) == wa.WA_EINVAL


def test_tree_decode_workspace_errors():
    need = ensure_built().lib().wa_tree_decode_ws_bytes(3, 8, 16, 8, 256, 1024, 1536)
    assert need > 0
    assert _decode(ws=None) == wa.WA_EWORKSPACE
    assert _decode(ws_bytes=need - 1) == wa.WA_EWORKSPACE
    assert _decode(ws=ctypes.c_void_p((1 << 20) + 128)) == wa.WA_EWORKSPACE


@pytest.mark.parametrize("size", [(0, 8, 16, 8, 256, 0, 64), (1, 0, 16, 8, 256, 0, 64), (1, 129, 16, 8, 256, 0, 64),
                                  (1, 8, 17, 8, 256, 0, 64), (1, 8, 16, 8, 192, 0, 64), (1, 8, 16, 8, 256, 65, 64),
                                  (1, 8, 16, 8, 256, 0, 0)])
def test_tree_decode_ws_bytes_of_invalid_sizes(size):
    assert ensure_built().lib().wa_tree_decode_ws_bytes(*size) == 0


def _verify(**kw):
    L = ensure_built().lib()
    a = dict(target=FAKE, draft=FAKE, parent=FAKE, tokens=FAKE, n=None, u=FAKE, rows=3, nodes=8, vocab=1000, st=None,
             path=FAKE, length=FAKE, token=FAKE, ws=FAKE, ws_bytes=256)
    a.update(kw)
    st = None if a["st"] is None else ctypes.byref(wa._VerifyStrides(**a["st"]))
    return L.wa_tree_verify(a["target"], a["draft"], a["parent"], a["tokens"], a["n"], a["u"], a["rows"], a["nodes"],
                            a["vocab"], st, a["path"], a["length"], a["token"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(target=None), dict(parent=None), dict(tokens=None), dict(u=None), dict(path=None), dict(length=None),
    dict(token=None), dict(rows=0), dict(rows=65536), dict(nodes=0), dict(nodes=129), dict(vocab=0),
    dict(vocab=(1 << 24) + 1), dict(target=ODD), dict(draft=ODD), dict(st=dict(t_node=999)), dict(st=dict(t_row=8)),
    dict(st=dict(d_node=-1000)),
], ids=str)
def test_tree_verify_argument_errors(bad):
    assert _verify(**bad) == wa.WA_EINVAL


def test_tree_verify_workspace_errors():
    assert _verify(ws=None) == wa.WA_EWORKSPACE
    assert _verify(ws_bytes=255) == wa.WA_EWORKSPACE
    assert _verify(ws=ctypes.c_void_p((1 << 20) + 8)) == wa.WA_EWORKSPACE


def _commit(**kw):
    L = ensure_built().lib()
    a = dict(layers=2, ptr=1 << 20, ring=64, rows=3, nodes=8, hkv=8, d=256, st=None, path=FAKE, most=8, length=FAKE,
             pos=FAKE, ws=FAKE, ws_bytes=256, lists=True)
    a.update(kw)
    st = None if a["st"] is None else ctypes.byref(wa._TreeStrides(**a["st"]))
    arr = (ctypes.c_void_p * 64)(*[a["ptr"]] * 64) if a["lists"] else None
    return L.wa_tree_commit(a["layers"], arr, arr, arr, arr, (ctypes.c_int32 * 64)(*[a["ring"]] * 64), a["rows"],
                            a["nodes"], a["hkv"], a["d"], st, a["path"], a["most"], a["length"], a["pos"], a["ws"],
                            a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(layers=0), dict(layers=65), dict(ptr=0), dict(ptr=(1 << 20) + 8), dict(ring=0), dict(rows=0), dict(nodes=0),
    dict(nodes=129), dict(hkv=0), dict(d=64), dict(path=None), dict(most=0), dict(most=129), dict(length=None),
    dict(pos=None), dict(lists=False), dict(st=dict(k_tok=8)), dict(st=dict(v_tok=8 * 256 + 4)),
], ids=str)
def test_tree_commit_argument_errors(bad):
    assert _commit(**bad) == wa.WA_EINVAL


def test_tree_commit_workspace_errors():
    assert _commit(ws=None) == wa.WA_EWORKSPACE
    assert _commit(ws_bytes=128) == wa.WA_EWORKSPACE


@pytest.mark.parametrize("kt,vt,kr,vr,ok", [
    ([1, 2], [3, 4], [5, 6], [7, 8], True),
    ([1, 2], [3, 4], [5, 5], [7, 8], False),          # two layers' nodes into one ring
    ([1, 2], [3, 4], [5, 6], [7, 6], False),          # keys and values into one ring
    ([1, 2], [3, 1], [5, 6], [7, 5], True),           # one layer's values are another's keys
    ([1, 1], [3, 3], [5, 5], [7, 7], True),           # a cache that layers share
    ([1, 2], [1, 2], [5, 6], [5, 6], True),           # keys that are the values
    ([1, 1], [3, 3], [5, 5], [7, 8], True),
])
def test_tree_commit_of_one_ring_twice(kt, vt, kr, vr, ok):
    L = ensure_built().lib()
    arr = lambda xs: (ctypes.c_void_p * 2)(*[x << 20 for x in xs])     # noqa: E731

    def call(rings, st=None):
        # without a workspace, which is looked at last: nothing is launched
        return L.wa_tree_commit(2, arr(kt), arr(vt), arr(kr), arr(vr), (ctypes.c_int32 * 2)(*rings), 3, 8, 8, 256,
                                None if st is None else ctypes.byref(st), FAKE, 8, FAKE, FAKE, None, 0, None)

    assert call([64, 64]) == (wa.WA_EWORKSPACE if ok else wa.WA_EINVAL)
    if ok and len({*kr, *vr}) < 4 and kr[0] == kr[1]:
        assert call([64, 65]) == wa.WA_EINVAL          # one ring of two lengths
    if ok and kr == vr:                                # one tree read two ways
        assert call([64, 64], wa._TreeStrides(k_tok=2048, v_tok=4096)) == wa.WA_EINVAL


def test_status_names():
    L = ensure_built().lib()
    assert b"tree" in L.wa_strerror(wa.WA_STATUS_BAD_TREE)
    assert b"mass" in L.wa_strerror(wa.WA_STATUS_NO_MASS)


# ---- the binding: tensors that disagree never reach the library

def _shapes(**kw):
    a = dict(q=bf16(3, 8, 16, 256), k_ring=bf16(3, 64, 8, 256), v_ring=bf16(3, 64, 8, 256), k_tree=bf16(3, 8, 8, 256),
             v_tree=bf16(3, 8, 8, 256), out=None)
    a.update(kw)
    return wa._tree_shapes(**a)


def test_tree_shapes_accept_a_consistent_call():
    assert _shapes() == (3, 8, 16, 8, 256, 64)
    assert _shapes(out=bf16(3, 8, 16, 256)) == (3, 8, 16, 8, 256, 64)


@pytest.mark.parametrize("bad", [
    dict(q=bf16(8, 16, 256)), dict(k_ring=bf16(2, 64, 8, 256)), dict(k_ring=bf16(3, 64, 8, 128)),
    dict(v_ring=bf16(3, 63, 8, 256)), dict(k_tree=bf16(3, 7, 8, 256)), dict(v_tree=bf16(3, 8, 4, 256)),
    dict(out=bf16(3, 8, 8, 256)), dict(out=torch.zeros(3, 8, 16, 256)),
    dict(k_ring=bf16(64, 3, 8, 256).transpose(0, 1)),
], ids=range(9))
def test_tree_shapes_refuse_disagreeing_tensors(bad):
    with pytest.raises(ValueError):
        _shapes(**bad)


def test_node_strides():
    assert wa._node_strides("q", bf16(3, 8, 16, 256), 256) == (8 * 4096, 4096)
    assert wa._node_strides("q", bf16(8, 3, 16, 256).transpose(0, 1), 256) == (4096, 3 * 4096)
    fused = bf16(3, 8, 24 * 128)
    assert wa._node_strides("v", fused[:, :, 20 * 128:].unflatten(2, (4, 128)), 128) == (8 * 24 * 128, 24 * 128)
    assert wa._node_strides("q", bf16(1, 1, 4, 128), 128) == (512, 512)
    for t in (bf16(1, 8, 4, 128).expand(3, 8, 4, 128), bf16(3, 1, 4, 128).expand(3, 8, 4, 128),
              bf16(3, 8, 4, 256)[..., ::2], bf16(3, 8, 8, 128)[:, :, ::2]):
        with pytest.raises(ValueError):
            wa._node_strides("q", t, 128)


def test_calls_refuse_host_tensors_and_types():
    q, ring, tr = bf16(1, 2, 4, 128), bf16(1, 8, 4, 128), bf16(1, 2, 4, 128)
    i = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        wa.tree_decode(q, ring, ring, tr, tr, i[:, 0], i, 0)
    with pytest.raises(TypeError):
        wa.tree_verify(torch.zeros(1, 2, 9), i, i, torch.zeros(1, 2))
    with pytest.raises(TypeError):
        wa.tree_commit(tr, tr, ring, ring, i, i[:, 0], i[:, 0])


def _spans(p, win, hq):
    """Spans that a row at position p is cut into, from the documented rule: its own key count, window and hq."""
    lo = max(0, p + 2 - win) if win else 0
    tiles = -(-max(p - lo + 1, 0) // 128) + 1
    want = win * hq // 64 if win else (p + 1) * hq // 128
    length = 256 if win else 512
    while length < 2048 and 2 * length <= want:
        length *= 2
    return -(-tiles // (length // 128 + 1))


@pytest.mark.parametrize("win", [0, 1, 2, 300, 512, 513, 1000, 1024, 2049, 9000])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 8), (12, 4), (16, 1), (64, 4)])
def test_the_workspace_holds_every_rows_spans(win, hq, hkv):
    """The workspace's size counts the most spans any position can have, whatever the ring."""
    L = ensure_built().lib()
    for ring in (win, win + 7, win + 5000) if win else (1, 511, 512, 513, 4095, 4096, 20000, 60001):
        lanes = (hq // hkv + 31) // 32 * 32
        held = (L.wa_tree_decode_ws_bytes(1, 1, hq, hkv, 128, win, ring) - 256) // (hkv * lanes * (128 + 5) * 4)
        at = range(-1, 30000, 13) if win else [*range(-1, ring, 29), ring - 1]
        most = max(_spans(p, win, hq) for p in at)
        assert most <= held <= most + 1, (ring, most, held)


def test_windows_of_any_numeric_type():
    for win in (64, 64.0, np.int64(64), np.float32(64.0), torch.tensor(64)):
        assert wa._window(win) == 64 and type(wa._window(win)) is int
    for win in (None, "64", [64]):
        with pytest.raises(TypeError, match="win"):
            wa._window(win)
    for win in (64.5, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="win"):
            wa._window(win)


def test_numbers_past_32_bits():
    """What ctypes would take modulo 2^32 is refused (or no valid size, for a workspace) instead."""
    for win in (2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 32 + 64, 2 ** 70, 2.0 ** 40):
        with pytest.raises(ValueError, match="win"):
            wa._window(win)
    for sizes in ((2 ** 32 + 1, 8), (1, 2 ** 31), (-2 ** 32 + 1,)):
        with pytest.raises(ValueError):
            wa._check_sizes(sizes)
    wa._check_sizes((1, 2 ** 31 - 1))
    good = (1, 8, 16, 8, 256, 64, 64)
    assert wa.tree_decode_ws_bytes(*good) > 0
    for i in range(7):
        assert wa.tree_decode_ws_bytes(*good[:i], good[i] + 2 ** 32, *good[i + 1:]) == 0


# ---- the extension module is a shorter way to the same calls, not a condition for any

def test_the_extension_module_is_built_and_used():
    ensure_built()
    assert wa._short_way() is not None and wa._short_way().built_for == wa._BIND_FOR


@pytest.fixture
def not_loaded(monkeypatch):
    ensure_built()
    monkeypatch.setattr(wa, "_lib", None)
    monkeypatch.setattr(wa, "_bind", False)
    return monkeypatch


@pytest.mark.parametrize("what", ["missing", "no module", "built for another"])
def test_without_the_extension_module(not_loaded, tmp_path, what):
    if what == "built for another":
        not_loaded.setattr(wa, "_BIND_FOR", "PyTorch 1.0, Python 2.7")
    else:
        path = tmp_path / "wa_bind.so"
        if what == "no module":
            path.write_bytes(b"nothing")
        not_loaded.setattr(wa, "_BIND_PATH", str(path))
    assert wa.lib().wa_version() > 0              # the library, and with it every other call, does without
    assert wa.decode_ws_bytes(1, 16, 256, 1024, 1536) > 0
    q, ring, tr, i = bf16(1, 2, 4, 128), bf16(1, 8, 4, 128), bf16(1, 2, 4, 128), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="wa_bind.so"), pytest.raises(TypeError, match="CUDA"):
        wa.tree_decode(q, ring, ring, tr, tr, i[:, 0], i, 0)
    with warnings.catch_warnings():
        warnings.simplefilter("error")            # said once
        with pytest.raises(TypeError, match="CUDA"):
            wa.tree_verify(torch.zeros(1, 2, 9), i, i, torch.zeros(1, 2))
        with pytest.raises(TypeError, match="CUDA"):
            wa.tree_commit(tr, tr, ring, ring, i, i[:, 0], i[:, 0])


def test_a_missing_library_is_named(not_loaded, tmp_path):
    not_loaded.setattr(wa, "_LIB_PATH", str(tmp_path / "libwa.so"))
    with pytest.raises(RuntimeError, match="libwa.so is missing"):
        wa.lib()


def test_the_build_goes_on_without_the_extension_module(monkeypatch, tmp_path, capsys):
    """A compiler that refuses wa_bind.cpp: libwa.so is built, an older wa_bind.so is taken away, and it is said."""
    from sliding_window_gqa_gb300 import build
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libwa.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "wa_bind.so"))
    monkeypatch.setattr(build, "SOURCES", ["wa_tree_commit.cu"])

    def refuse(*a):
        raise RuntimeError("g++ on wa_bind.cpp failed")

    monkeypatch.setattr(build, "_compile_bind", refuse)
    (tmp_path / "wa_bind.so").write_bytes(b"old")
    assert build.build() == str(tmp_path / "libwa.so")
    assert (tmp_path / "libwa.so").exists() and not (tmp_path / "wa_bind.so").exists()
    assert "wa_bind.so was not built" in capsys.readouterr().err
