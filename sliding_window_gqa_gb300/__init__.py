"""Sliding-window grouped-query attention for one GB300 (sm_103a).

A thin ctypes binding of ``libwa.so`` (the C ABI declared in ``include/wa.h``):
it checks dtypes and devices, turns tensors into pointers and strides, and
calls the library on the current CUDA stream.  Every step of the attention
runs in the library's CUDA kernels; there is no Python or CPU fallback, and
calling an entry point without the built library raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import re
import sys
import warnings

import torch

__all__ = [
    "WAError", "lib", "lib_path", "decode", "decode_static", "prompt", "prompt_sparse", "prep_append", "status",
    "tree_decode", "tree_verify", "tree_commit", "decode_ws_bytes", "prompt_ws_bytes", "tree_decode_ws_bytes",
    "rope", "rope_frequencies", "paged_append", "paged_decode", "paged_decode_ws_bytes",
    "WA_OK", "WA_EINVAL", "WA_EWORKSPACE", "WA_ECUDA", "WA_EDEVICE",
    "WA_STATUS_BAD_POS", "WA_STATUS_BAD_HI", "WA_STATUS_TIMEOUT",
    "WA_STATUS_BAD_TREE", "WA_STATUS_NO_MASS", "WA_STATUS_BAD_PAGE", "WA_TREE_MAX_NODES", "WA_COMMIT_MAX_LAYERS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libwa.so")
_BIND_PATH = os.path.join(_HERE, "_build", "wa_bind.so")
_BIND_FOR = f"PyTorch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"   # as build.py has it
_HEADER = os.path.join(os.path.dirname(_HERE), "include", "wa.h")


def _header_constants() -> dict:
    consts = {}
    with open(_HEADER) as f:
        for line in f:
            m = re.match(r"#define\s+(WA_\w+)\s+\(?(-?\d+)\)?", line)
            if m:
                consts[m.group(1)] = int(m.group(2))
    return consts


_C = _header_constants()
WA_OK = _C["WA_OK"]
WA_EINVAL = _C["WA_EINVAL"]
WA_EWORKSPACE = _C["WA_EWORKSPACE"]
WA_ECUDA = _C["WA_ECUDA"]
WA_EDEVICE = _C["WA_EDEVICE"]
WA_STATUS_BAD_POS = _C["WA_STATUS_BAD_POS"]
WA_STATUS_BAD_HI = _C["WA_STATUS_BAD_HI"]
WA_STATUS_TIMEOUT = _C["WA_STATUS_TIMEOUT"]
WA_STATUS_BAD_TREE = _C["WA_STATUS_BAD_TREE"]
WA_STATUS_NO_MASS = _C["WA_STATUS_NO_MASS"]
WA_STATUS_BAD_PAGE = _C["WA_STATUS_BAD_PAGE"]
WA_TREE_MAX_NODES = _C["WA_TREE_MAX_NODES"]
WA_COMMIT_MAX_LAYERS = _C["WA_COMMIT_MAX_LAYERS"]


class WAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().wa_strerror(code).decode()} ({code})")


class _Strides(ctypes.Structure):
    _fields_ = [("q", ctypes.c_int64), ("k", ctypes.c_int64), ("v", ctypes.c_int64), ("out", ctypes.c_int64)]


class _PrepLayout(ctypes.Structure):
    _fields_ = [("src_tok", ctypes.c_int64), ("q_tok", ctypes.c_int64), ("ring_row", ctypes.c_int64),
                ("slot", ctypes.c_int64)]


class _TreeStrides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("q_row", "q_tok", "k_row", "k_tok", "v_row", "v_tok", "out_row", "out_tok")]


class _VerifyStrides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("t_row", "t_node", "d_row", "d_node")]


class _Rotary(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("dims", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("factor", ctypes.c_float)]


class _Pages(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale", "table")] \
        + [(f, ctypes.c_int64) for f in ("k_page", "k_slot", "k_head", "v_page", "v_slot", "v_head", "table_row")] \
        + [(f, ctypes.c_int32) for f in ("pages", "page_size", "rows", "most", "hkv", "d", "type")]


_lib = None
_bind = False     # the short way to the drafted-token and paged-cache calls (csrc/wa_bind.cpp); None: there is none, False: not looked for
_P = ctypes.c_void_p
_I = ctypes.c_int32


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(_LIB_PATH)
        L.wa_decode_ws_bytes.argtypes = [_I, _I, _I, _I, _I]
        L.wa_decode_ws_bytes.restype = ctypes.c_size_t
        L.wa_decode.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
        L.wa_decode.restype = ctypes.c_int
        L.wa_decode_static.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P]
        L.wa_decode_static.restype = ctypes.c_int
        L.wa_prompt_ws_bytes.argtypes = [_I, _I]
        L.wa_prompt_ws_bytes.restype = ctypes.c_size_t
        L.wa_prompt.argtypes = [_P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _I, ctypes.c_float, _I,
                                ctypes.POINTER(_Strides), _P, _P, ctypes.c_size_t, _P]
        L.wa_prompt.restype = ctypes.c_int
        L.wa_prompt_sparse.argtypes = [_P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P, _I,
                                       ctypes.POINTER(_Strides), _P, _P, ctypes.c_size_t, _P]
        L.wa_prompt_sparse.restype = ctypes.c_int
        L.wa_prep_append.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _I, ctypes.POINTER(_PrepLayout),
                                     _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.wa_prep_append.restype = ctypes.c_int
        L.wa_tree_decode_ws_bytes.argtypes = [_I] * 7
        L.wa_tree_decode_ws_bytes.restype = ctypes.c_size_t
        L.wa_tree_decode.argtypes = [_P] * 8 + [_I] * 7 + [ctypes.c_float, ctypes.POINTER(_TreeStrides), _P, _P,
                                                          ctypes.c_size_t, _P]
        L.wa_tree_decode.restype = ctypes.c_int
        L.wa_tree_verify.argtypes = [_P] * 6 + [_I] * 3 + [ctypes.POINTER(_VerifyStrides), _P, _P, _P, _P,
                                                          ctypes.c_size_t, _P]
        L.wa_tree_verify.restype = ctypes.c_int
        L.wa_tree_commit.argtypes = [_I, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(_TreeStrides), _P, _I, _P,
                                     _P, _P, ctypes.c_size_t, _P]
        L.wa_tree_commit.restype = ctypes.c_int
        L.wa_rope.argtypes = [_P, _P, _I, _I, _I, ctypes.POINTER(_Rotary), _I, ctypes.c_int64, ctypes.c_int64, _P, _P]
        L.wa_rope.restype = ctypes.c_int
        L.wa_paged_append.argtypes = [_P, _P, _P, _I, _I, ctypes.POINTER(_Pages), ctypes.POINTER(_Rotary),
                                      ctypes.c_int64, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P]
        L.wa_paged_append.restype = ctypes.c_int
        L.wa_paged_decode_ws_bytes.argtypes = [ctypes.POINTER(_Pages), _I, _I]
        L.wa_paged_decode_ws_bytes.restype = ctypes.c_size_t
        L.wa_paged_decode.argtypes = [_P, _P, _I, ctypes.POINTER(_Pages), _I, ctypes.c_float, ctypes.c_int64,
                                      ctypes.c_int64, _P, _P, ctypes.c_size_t, _P]
        L.wa_paged_decode.restype = ctypes.c_int
        L.wa_status.argtypes = [_P, _P]
        L.wa_status.restype = ctypes.c_int
        L.wa_strerror.argtypes = [ctypes.c_int]
        L.wa_strerror.restype = ctypes.c_char_p
        L.wa_version.argtypes = []
        L.wa_version.restype = ctypes.c_int
        _lib = L
    return _lib


def _short_way():
    """The extension module, or None where it is missing or was built for another PyTorch or Python: every call goes
    through ctypes then, with the same results and some microseconds more on the host, which is warned of once."""
    global _bind
    if _bind is False:
        lib()
        try:
            spec = importlib.util.spec_from_file_location("wa_bind", _BIND_PATH)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            built_for = getattr(module, "built_for", "something else")
            if built_for != _BIND_FOR:
                raise ImportError(f"built for {built_for}, this is {_BIND_FOR}")
            _bind = module
        except (ImportError, OSError) as e:
            _bind = None
            warnings.warn(f"{_BIND_PATH} cannot be used ({e}): the drafted-token and paged-cache calls take some microseconds longer",
                          RuntimeWarning, stacklevel=3)
    return _bind


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check_bf16(name: str, t: torch.Tensor) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a bf16 CUDA tensor")


def decode_ws_bytes(rows: int, hq: int, d: int, win: int, ring: int) -> int:
    return int(lib().wa_decode_ws_bytes(rows, hq, d, win, ring))


def prompt_ws_bytes(n: int, hq: int) -> int:
    return int(lib().wa_prompt_ws_bytes(n, hq))


def _workspace(nbytes: int, device, ws):
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous CUDA tensor on the inputs' device")
    return ws


def _ws_bytes(ws) -> int:
    return int(ws.numel() * ws.element_size())


def _same_device(device, **ts) -> None:
    for name, t in ts.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other inputs on {device}")


# Shape agreement between the tensors of one call.  The C ABI receives bare pointers and
# trusts these extents, so a mismatch here would become an out-of-bounds access there.

def _decode_shapes(q, k_ring, v_ring, pos, out):
    """(rows, hq, hkv, d, ring) of a decode call; ValueError if the tensors disagree."""
    if q.dim() != 3 or k_ring.dim() != 4:
        raise ValueError("q must be [rows, hq, d] and k_ring [rows, ring, hkv, d]")
    rows, hq, d = q.shape
    if k_ring.shape[0] != rows or k_ring.shape[3] != d:
        raise ValueError(f"k_ring {tuple(k_ring.shape)} does not match q {tuple(q.shape)}")
    if tuple(v_ring.shape) != tuple(k_ring.shape):
        raise ValueError(f"v_ring {tuple(v_ring.shape)} must have k_ring's shape {tuple(k_ring.shape)}")
    if pos.dim() != 1 or pos.numel() != rows or not pos.is_contiguous():
        raise ValueError(f"pos must be a contiguous vector of {rows} positions")
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != tuple(q.shape)
                            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous bf16 tensor of q's shape {tuple(q.shape)}")
    return rows, hq, k_ring.shape[2], d, k_ring.shape[1]


def _prompt_shapes(q, k, v, hi, out):
    """(n, hq, hkv, d, ring) of a prompt call; ValueError if the tensors disagree."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [n, hq, d] and k, v [ring, hkv, d]")
    n, hq, d = q.shape
    ring, hkv, dk = k.shape
    if dk != d:
        raise ValueError(f"k's head dim {dk} differs from q's {d}")
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"v {tuple(v.shape)} must have k's shape {tuple(k.shape)}")
    if hi is not None and (hi.dtype != torch.int32 or hi.dim() != 1 or hi.numel() != n or not hi.is_contiguous()):
        raise TypeError("hi must be None or a contiguous int32 tensor of n elements")
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != (n, hq, d)):
        raise ValueError(f"out must be a bf16 tensor of shape {(n, hq, d)}")
    return n, hq, hkv, d, ring


def _prep_shapes(src, pos, q_out, k_ring, v_ring):
    """(n, hq, hkv, d) of a preparation call; ValueError if the tensors disagree."""
    if src.dim() != 2 or q_out.dim() != 3 or k_ring.dim() not in (3, 4):
        raise ValueError("src must be [n, row], q_out [n, hq, d], k_ring [ring, hkv, d] or [n, ring, hkv, d]")
    n = src.shape[0]
    d = k_ring.shape[-1]
    hq, hkv = q_out.shape[1], k_ring.shape[-2]
    if q_out.shape[0] != n or q_out.shape[2] != d:
        raise ValueError(f"q_out {tuple(q_out.shape)} does not match {n} tokens of head dim {d}")
    if src.shape[1] < (hq + 2 * hkv) * d:
        raise ValueError(f"src rows hold {src.shape[1]} values, fewer than (hq + 2 hkv) d = {(hq + 2 * hkv) * d}")
    if k_ring.dim() == 4 and k_ring.shape[0] != n:
        raise ValueError(f"per-token rings: k_ring has {k_ring.shape[0]} rings for {n} tokens")
    if v_ring is not None and tuple(v_ring.shape) != tuple(k_ring.shape):
        raise ValueError(f"v_ring {tuple(v_ring.shape)} must have k_ring's shape {tuple(k_ring.shape)}")
    if pos.dim() != 1 or pos.numel() != n or not pos.is_contiguous():
        raise ValueError(f"pos must be a contiguous vector of {n} positions")
    return n, hq, hkv, d


def decode(q, k_ring, v_ring, pos, win: int, scale: float = 1.0, out=None, ws=None, stream=None):
    """Decode attention: q [rows,hq,d], k_ring/v_ring [rows,ring,hkv,d] (bf16, dense), pos int32 [rows].

    Returns out [rows,hq,d] bf16.  ``ws`` may be a reused uint8 CUDA buffer of
    at least decode_ws_bytes(...) bytes; the call is asynchronous on ``stream``."""
    for n_, t in (("q", q), ("k_ring", k_ring), ("v_ring", v_ring)):
        _check_bf16(n_, t)
        if not t.is_contiguous():
            raise ValueError(f"{n_} must be contiguous")
    if pos.dtype != torch.int32 or not pos.is_cuda:
        raise TypeError("pos must be an int32 CUDA tensor")
    rows, hq, hkv, d, ring = _decode_shapes(q, k_ring, v_ring, pos, out)
    _same_device(q.device, k_ring=k_ring, v_ring=v_ring, pos=pos, out=out)
    if out is None:
        out = torch.empty_like(q)
    nbytes = decode_ws_bytes(rows, hq, d, win, ring)
    ws = _workspace(nbytes, q.device, ws)
    rc = lib().wa_decode(q.data_ptr(), k_ring.data_ptr(), v_ring.data_ptr(), pos.data_ptr(), rows, hq, hkv, d,
                         win, ring, float(scale), out.data_ptr(), ws.data_ptr(), _ws_bytes(ws),
                         _stream_handle(stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_decode")
    return out


def decode_static(q, k_ring, v_ring, pos, win: int, scale: float = 1.0, out=None, stream=None):
    """decode() without a workspace: the library's fixed device scratch (WA_STATIC_WS_BYTES a
    device) holds the partials, for callers that cannot allocate device memory.  Calls that
    may overlap on the GPU share that scratch and must be ordered by the caller; the status
    bits of the last call are status(None)."""
    for n_, t in (("q", q), ("k_ring", k_ring), ("v_ring", v_ring)):
        _check_bf16(n_, t)
        if not t.is_contiguous():
            raise ValueError(f"{n_} must be contiguous")
    if pos.dtype != torch.int32 or not pos.is_cuda:
        raise TypeError("pos must be an int32 CUDA tensor")
    rows, hq, hkv, d, ring = _decode_shapes(q, k_ring, v_ring, pos, out)
    _same_device(q.device, k_ring=k_ring, v_ring=v_ring, pos=pos, out=out)
    if out is None:
        out = torch.empty_like(q)
    rc = lib().wa_decode_static(q.data_ptr(), k_ring.data_ptr(), v_ring.data_ptr(), pos.data_ptr(), rows, hq, hkv,
                                d, win, ring, float(scale), out.data_ptr(), _stream_handle(stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_decode_static")
    return out


def _token_stride(name: str, t: torch.Tensor, d: int) -> int:
    if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != d:
        raise ValueError(f"{name} must be [tokens, heads, d] with head stride d and unit dim stride")
    return int(t.stride(0))


def prompt(q, k, v, p0: int, hi=None, win: int = 0, scale: float = 1.0, p32=False,
           out=None, ws=None, stream=None):
    """Prompt attention for rows p0 .. p0+n-1: q [n,hq,d], k/v [ring,hkv,d] (bf16, token-strided).

    ``hi`` is None (each row's last key is its own position) or an int32 CUDA
    tensor [n].  ``p32``: False / 0 (one bf16 P), True / 1 (two parts) or 2 (three
    parts).  Returns out [n,hq,d] bf16."""
    for n_, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n_, t)
    n, hq, hkv, d, ring = _prompt_shapes(q, k, v, hi, out)
    _same_device(q.device, k=k, v=v, hi=hi, out=out)
    if out is None:
        out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=q.device)
    st = _Strides(_token_stride("q", q, d), _token_stride("k", k, d), _token_stride("v", v, d),
                  _token_stride("out", out, d))
    ws = _workspace(prompt_ws_bytes(n, hq), q.device, ws)
    rc = lib().wa_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), int(p0), n,
                         None if hi is None else hi.data_ptr(), hq, hkv, d, int(win), ring, float(scale),
                         int(p32), ctypes.byref(st), out.data_ptr(), ws.data_ptr(), _ws_bytes(ws),
                         _stream_handle(stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_prompt")
    return out


def prompt_sparse(q, k, v, p0: int, sel, hi=None, win: int = 0, scale: float = 1.0, p32=False,
                  out=None, ws=None, stream=None):
    """Block-sparse prompt: as prompt(), with sel an int32 CUDA tensor [n, hkv, nsel] of selected
    64-key blocks (-1 = unused).  Returns out [n,hq,d] bf16."""
    for n_, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(n_, t)
    n, hq, hkv, d, ring = _prompt_shapes(q, k, v, hi, out)
    if sel.dtype != torch.int32 or not sel.is_cuda or not sel.is_contiguous() or sel.dim() != 3 or \
            sel.shape[0] != n or sel.shape[1] != hkv:
        raise TypeError("sel must be a contiguous int32 CUDA tensor [n, hkv, nsel]")
    _same_device(q.device, k=k, v=v, hi=hi, sel=sel, out=out)
    if out is None:
        out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=q.device)
    st = _Strides(_token_stride("q", q, d), _token_stride("k", k, d), _token_stride("v", v, d),
                  _token_stride("out", out, d))
    ws = _workspace(prompt_ws_bytes(n, hq), q.device, ws)
    rc = lib().wa_prompt_sparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), int(p0), n,
                                None if hi is None else hi.data_ptr(), hq, hkv, d, int(win), ring, float(scale),
                                int(p32), sel.data_ptr(), sel.shape[2], ctypes.byref(st), out.data_ptr(),
                                ws.data_ptr(), _ws_bytes(ws), _stream_handle(stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_prompt_sparse")
    return out


_PREP_MODES = {"rmsnorm": _C["WA_PREP_RMSNORM"], "l2_rope": _C["WA_PREP_L2_ROPE"]}


def _ring_layout(name: str, t: torch.Tensor, d: int):
    """(ring, ring_row, slot) of a [ring, hkv, d] shared ring or [tokens, ring, hkv, d] per-token rings."""
    if t.stride(-1) != 1 or t.stride(-2) != d:
        raise ValueError(f"{name} must have head stride d and unit dim stride")
    if t.dim() == 3:
        return t.shape[0], 0, int(t.stride(0))
    if t.dim() == 4:
        return t.shape[1], int(t.stride(0)), int(t.stride(1))
    raise ValueError(f"{name} must be [ring, hkv, d] or [tokens, ring, hkv, d]")


def prep_append(src, pos, q_out, k_ring, v_ring=None, mode: str = "rmsnorm", q_scale=None, inv_freq=None,
                ws=None, stream=None):
    """q/k preparation and KV append.

    src [n, >= (hq + 2 hkv) d] bf16 projection rows (unit inner stride), pos int32 [n],
    q_out [n, hq, d] (token-strided), k_ring / v_ring [ring, hkv, d] (one shared ring) or
    [n, ring, hkv, d] (one ring per token).  v_ring None leaves v where it is.  mode "rmsnorm"
    or "l2_rope" (then inv_freq fp32 [d/2], q_scale fp32 [d] or None).  Returns the workspace,
    whose status wa_status / status() reads."""
    _check_bf16("src", src)
    _check_bf16("q_out", q_out)
    _check_bf16("k_ring", k_ring)
    if v_ring is not None:
        _check_bf16("v_ring", v_ring)
    if pos.dtype != torch.int32 or not pos.is_cuda:
        raise TypeError("pos must be an int32 CUDA tensor")
    if src.dim() != 2 or src.stride(1) != 1:
        raise ValueError("src must be [n, row] with unit inner stride")
    n, hq, hkv, d = _prep_shapes(src, pos, q_out, k_ring, v_ring)
    _same_device(src.device, pos=pos, q_out=q_out, k_ring=k_ring, v_ring=v_ring, q_scale=q_scale, inv_freq=inv_freq)
    ring, ring_row, slot = _ring_layout("k_ring", k_ring, d)
    if v_ring is not None and _ring_layout("v_ring", v_ring, d) != (ring, ring_row, slot):
        raise ValueError("v_ring must have k_ring's layout")
    for n_, t, cnt in (("q_scale", q_scale, d), ("inv_freq", inv_freq, d // 2)):
        if t is not None and (t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != cnt):
            raise TypeError(f"{n_} must be a contiguous fp32 CUDA tensor of {cnt} elements")
    lay = _PrepLayout(int(src.stride(0)), _token_stride("q_out", q_out, d), ring_row, slot)
    ws = _workspace(256, src.device, ws)
    rc = lib().wa_prep_append(src.data_ptr(), pos.data_ptr(), n, hq, hkv, d, _PREP_MODES[mode],
                              None if q_scale is None else q_scale.data_ptr(),
                              None if inv_freq is None else inv_freq.data_ptr(), ring, ctypes.byref(lay),
                              q_out.data_ptr(), k_ring.data_ptr(), None if v_ring is None else v_ring.data_ptr(),
                              ws.data_ptr(), _ws_bytes(ws), _stream_handle(stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_prep_append")
    return ws


# Drafted tokens.  These calls run on their inputs' device, whichever is current, and on `stream` or
# that device's current stream; what they allocate is that stream's.  A drafted step makes one
# call a layer, of a few microseconds on the GPU for a single sequence, so the ordinary call (contiguous
# tensors on the current device and stream) is checked and made by the extension module; it returns None
# for any other one, which goes through the checks here.

def _empty(shape, dtype, device, stream, handed_back=True):
    """Memory for a call on ``stream``, from that stream's own: what was freed on the current stream may yet be written
    by what is queued there.  The caller uses what is handed back on the current stream, so it is kept for that one too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if handed_back and stream != torch.cuda.current_stream():
        t.record_stream(torch.cuda.current_stream())
    return t


def _workspace_on(stream, nbytes: int, device, ws, handed_back=False):
    if ws is None:
        return _empty(max(nbytes, 256), torch.uint8, device, stream, handed_back)
    return _workspace(0, device, ws)


def _stream_on(index: int, stream) -> int:
    return int((torch.cuda.current_stream(index) if stream is None else stream).cuda_stream)


def _result(got, what: str):
    """What the extension module returned: tensors, or a code that is raised."""
    if isinstance(got, int):
        raise WAError(got, what)
    return got


def _check_i32(name: str, t, shape) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda:
        raise TypeError(f"{name} must be an int32 CUDA tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and of shape {tuple(shape)}")


def _number(name: str, x):
    if not hasattr(x, "__index__") and not hasattr(x, "__float__"):
        raise TypeError(f"{name} must be a number, not {type(x).__name__}")
    return x


def _fit_32_bits(*sizes) -> bool:
    """Whether the library can be told these numbers: ctypes would take larger ones modulo 2^32."""
    return all(-2 ** 31 <= x < 2 ** 31 for x in sizes)


def _check_sizes(sizes) -> None:
    if not _fit_32_bits(*sizes):
        raise ValueError(f"sizes {tuple(sizes)} must be below 2^31")


def _window(win) -> int:
    """A window of any numeric type as an int."""
    try:
        w = int(_number("win", win))
    except (ValueError, OverflowError):      # not a finite number
        w = None
    if w is None or w != win:
        raise ValueError(f"win must be a whole number of keys, not {win}")
    if not _fit_32_bits(w):
        raise ValueError(f"win {w} must be below 2^31")
    return w


def _tree_shapes(q, k_ring, v_ring, k_tree, v_tree, out):
    """(rows, nodes, hq, hkv, d, ring) of a tree decode call; ValueError if the tensors disagree."""
    if q.dim() != 4 or k_ring.dim() != 4:
        raise ValueError("q must be [rows, nodes, hq, d] and k_ring [rows, ring, hkv, d]")
    rows, nodes, hq, d = q.shape
    _, ring, hkv, _ = k_ring.shape
    if k_ring.shape[0] != rows or k_ring.shape[3] != d:
        raise ValueError(f"k_ring {tuple(k_ring.shape)} does not match q {tuple(q.shape)}")
    if v_ring.shape != k_ring.shape:
        raise ValueError(f"v_ring {tuple(v_ring.shape)} must have k_ring's shape {tuple(k_ring.shape)}")
    if not k_ring.is_contiguous() or not v_ring.is_contiguous():
        raise ValueError("k_ring and v_ring must be contiguous")
    for name, t in (("k_tree", k_tree), ("v_tree", v_tree)):
        if t.shape != (rows, nodes, hkv, d):
            raise ValueError(f"{name} must have shape {(rows, nodes, hkv, d)}")
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != q.shape):
        raise ValueError(f"out must be a bf16 tensor of q's shape {tuple(q.shape)}")
    return rows, nodes, hq, hkv, d, ring


def _node_strides(name: str, t: torch.Tensor, d: int):
    """(row, node) strides in elements of a [rows, nodes, heads, d] tensor."""
    row, tok, head, one = t.stride()
    rows, nodes, heads, _ = t.shape
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name} must be [rows, nodes, heads, d] with head stride d and unit dim stride")
    # a dimension of one element may carry any stride
    tok = tok if nodes > 1 else heads * d
    row = row if rows > 1 else tok * nodes
    if tok < heads * d or row < heads * d:      # an expanded tensor: the library reads stride 0 as dense
        raise ValueError(f"{name}'s rows and nodes must not share memory")
    return row, tok


def _tree_check(q, k_ring, v_ring, k_tree, v_tree, pos, parent, n, out):
    """((rows, nodes, hq, hkv, d, ring), strides) of a tree decode call; raises where its tensors disagree."""
    for n_, t in (("q", q), ("k_ring", k_ring), ("v_ring", v_ring), ("k_tree", k_tree), ("v_tree", v_tree)):
        _check_bf16(n_, t)
    sizes = rows, nodes, hq, hkv, d, ring = _tree_shapes(q, k_ring, v_ring, k_tree, v_tree, out)
    _check_sizes(sizes)
    _check_i32("pos", pos, (rows,))
    _check_i32("parent", parent, (rows, nodes))
    if n is not None:
        _check_i32("n", n, (rows,))
    _same_device(q.device, k_ring=k_ring, v_ring=v_ring, k_tree=k_tree, v_tree=v_tree, pos=pos, parent=parent, n=n,
                 out=out)
    dense = (0, 0)      # as the library takes them
    return sizes, _TreeStrides(*_node_strides("q", q, d), *_node_strides("k_tree", k_tree, d),
                               *_node_strides("v_tree", v_tree, d),
                               *(dense if out is None else _node_strides("out", out, d)))


def tree_decode_ws_bytes(rows: int, nodes: int, hq: int, hkv: int, d: int, win: int, ring: int) -> int:
    sizes = rows, nodes, hq, hkv, d, win, ring
    return int(lib().wa_tree_decode_ws_bytes(*sizes)) if _fit_32_bits(*sizes) else 0


def tree_decode(q, k_ring, v_ring, k_tree, v_tree, pos, parent, win: int, n=None, scale: float = 1.0,
                out=None, ws=None, stream=None):
    """Decode for a tree of drafted tokens a row.

    q [rows, nodes, hq, d] and k_tree / v_tree [rows, nodes, hkv, d] hold the nodes (bf16, row- and
    node-strided), k_ring / v_ring [rows, ring, hkv, d] (dense) the cache up to position pos (int32
    [rows], -1 = empty).  parent int32 [rows, nodes]: the node before each (below its own index), -1
    for one that follows the cache; n int32 [rows] or None: nodes in use.  A node sees the cache, its
    ancestors and itself, as far as the window reaches back.  Returns out [rows, nodes, hq, d] bf16,
    whose nodes past n are not written.  ``ws``: a reused uint8 CUDA buffer of tree_decode_ws_bytes(...)."""
    bind = _short_way() if stream is None else None
    if bind is not None:
        got = bind.tree_decode(q, k_ring, v_ring, k_tree, v_tree, pos, parent, win, n, scale, out, ws)
        if got is not None:
            return _result(got, "wa_tree_decode")
    (rows, nodes, hq, hkv, d, ring), st = _tree_check(q, k_ring, v_ring, k_tree, v_tree, pos, parent, n, out)
    win, scale = _window(win), float(_number("scale", scale))
    dev = q.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return tree_decode(q, k_ring, v_ring, k_tree, v_tree, pos, parent, win, n, scale, out, ws, stream)
    if out is None:
        out = _empty((rows, nodes, hq, d), torch.bfloat16, dev, stream)
    ws = _workspace_on(stream, tree_decode_ws_bytes(rows, nodes, hq, hkv, d, win, ring), dev, ws)
    rc = lib().wa_tree_decode(
        q.data_ptr(), k_ring.data_ptr(), v_ring.data_ptr(), k_tree.data_ptr(), v_tree.data_ptr(), pos.data_ptr(),
        parent.data_ptr(), None if n is None else n.data_ptr(), rows, nodes, hq, hkv, d, win, ring, scale,
        ctypes.byref(st), out.data_ptr(), ws.data_ptr(), _ws_bytes(ws), _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_tree_decode")
    return out


def _prob_strides(name: str, t: torch.Tensor, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be an fp32 CUDA tensor")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be [rows, nodes, vocab], the same for target and draft")
    rows, nodes, vocab = t.shape
    if vocab > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride over the vocabulary")
    node = t.stride(1) if nodes > 1 else vocab
    row = t.stride(0) if rows > 1 else node * nodes
    if node < vocab or row < vocab:      # an expanded tensor: the library reads stride 0 as dense
        raise ValueError(f"{name}'s rows and nodes must not share memory")
    return row, node


def _verify_check(target, parent, tokens, u, draft, n, path, length, token):
    """Strides of a verification call; raises where its tensors disagree."""
    t_st = _prob_strides("target", target, None)
    rows, nodes, vocab = target.shape
    _check_sizes(target.shape)
    d_st = (0, 0) if draft is None else _prob_strides("draft", draft, target.shape)
    _check_i32("parent", parent, (rows, nodes))
    _check_i32("tokens", tokens, (rows, nodes))
    if not isinstance(u, torch.Tensor) or u.dtype != torch.float32 or not u.is_cuda:
        raise TypeError("u must be an fp32 CUDA tensor")
    if u.shape != (rows, nodes) or not u.is_contiguous():
        raise ValueError(f"u must be contiguous and of shape {(rows, nodes)}")
    for n_, t, shape in (("n", n, (rows,)), ("path", path, (rows, nodes)), ("length", length, (rows,)),
                         ("token", token, (rows,))):
        if t is not None:
            _check_i32(n_, t, shape)
    _same_device(target.device, draft=draft, parent=parent, tokens=tokens, u=u, n=n, path=path, length=length,
                 token=token)
    return _VerifyStrides(*t_st, *d_st)


def tree_verify(target, parent, tokens, u, draft=None, n=None, path=None, length=None, token=None, ws=None,
                stream=None):
    """Which drafted tokens the target keeps, and the token after them: speculative sampling over a tree.

    target fp32 [rows, nodes, vocab]: the target's probabilities after each node; draft: those that the
    node's children were drawn from, or None where they were not drawn.  parent, tokens int32
    [rows, nodes]; node 0 is the last sampled token.  u fp32 [rows, nodes] in [0, 1): u[:, c] tests node
    c, u[:, 0] samples the last token.  n int32 [rows] or None: nodes in use.  Returns (path int32
    [rows, nodes], length int32 [rows], token int32 [rows]): the kept nodes in order, then -1; how many;
    the token sampled after them (-1: no nodes, or a distribution without mass)."""
    bind = _short_way() if stream is None and path is None and length is None and token is None else None
    if bind is not None:
        got = bind.tree_verify(target, parent, tokens, u, draft, n, ws)
        if got is not None:
            return _result(got, "wa_tree_verify")
    st = _verify_check(target, parent, tokens, u, draft, n, path, length, token)
    rows, nodes, vocab = target.shape
    dev = target.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return tree_verify(target, parent, tokens, u, draft, n, path, length, token, ws, stream)
    path, length, token = [_empty(shape, torch.int32, dev, stream) if t is None else t
                           for t, shape in ((path, (rows, nodes)), (length, (rows,)), (token, (rows,)))]
    ws = _workspace_on(stream, 256, dev, ws)
    rc = lib().wa_tree_verify(
        target.data_ptr(), None if draft is None else draft.data_ptr(), parent.data_ptr(), tokens.data_ptr(),
        None if n is None else n.data_ptr(), u.data_ptr(), rows, nodes, vocab, ctypes.byref(st), path.data_ptr(),
        length.data_ptr(), token.data_ptr(), ws.data_ptr(), _ws_bytes(ws), _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_tree_verify")
    return path, length, token


def _commit_layers(kt, vt, kr, vr):
    """(rows, nodes, hkv, d, k strides, v strides) of the layers' tensors; raises where they disagree."""
    L = len(kt)
    if not (0 < L <= WA_COMMIT_MAX_LAYERS) or not len(vt) == len(kr) == len(vr) == L:
        raise ValueError(f"between 1 and {WA_COMMIT_MAX_LAYERS} layers, the same number of each tensor")
    for name, ts in (("k_tree", kt), ("v_tree", vt), ("k_ring", kr), ("v_ring", vr)):
        for t in ts:
            _check_bf16(name, t)
            if t.dim() != 4:
                raise ValueError(f"{name} must be [rows, nodes or ring, hkv, d]")
    shape = kt[0].shape
    rows, nodes, hkv, d = shape
    _check_sizes((*shape, *[t.shape[1] for t in kr]))
    k_st, v_st = _node_strides("k_tree", kt[0], d), _node_strides("v_tree", vt[0], d)
    for l in range(L):
        if kt[l].shape != shape or vt[l].shape != shape:
            raise ValueError(f"k_tree and v_tree must have one shape, {tuple(shape)}")
        if l and (_node_strides("k_tree", kt[l], d) != k_st or _node_strides("v_tree", vt[l], d) != v_st):
            raise ValueError("the layers' trees must have the same strides")
        want = (rows, kr[l].shape[1], hkv, d)
        if kr[l].shape != want or vr[l].shape != want or not kr[l].is_contiguous() or not vr[l].is_contiguous():
            raise ValueError(f"k_ring and v_ring must be contiguous [rows, ring, hkv, d] = {want}")
        _same_device(kt[0].device, k_tree=kt[l], v_tree=vt[l], k_ring=kr[l], v_ring=vr[l])
    return rows, nodes, hkv, d, k_st, v_st


def tree_commit(k_tree, v_tree, k_ring, v_ring, path, length, pos, ws=None, stream=None):
    """The kept nodes' keys and values into the rings: node path[r, j], j < length[r], goes to slot
    (pos[r] + 1 + j) mod ring.

    k_tree / v_tree [rows, nodes, hkv, d] and k_ring / v_ring [rows, ring, hkv, d] (bf16), or lists of
    them, one a layer (at most WA_COMMIT_MAX_LAYERS; rings may differ in length, trees share their
    strides).  path int32 [rows, most], length and pos int32 [rows], as tree_verify returned and
    tree_decode took them; afterwards the row's last position is pos + length.  Returns the
    workspace, whose status status() reads."""
    bind = _short_way() if stream is None else None
    if bind is not None:
        got = bind.tree_commit(k_tree, v_tree, k_ring, v_ring, path, length, pos, ws)
        if got is not None:
            return _result(got, "wa_tree_commit")
    kt, vt, kr, vr = ([x] if isinstance(x, torch.Tensor) else list(x) for x in (k_tree, v_tree, k_ring, v_ring))
    rows, nodes, hkv, d, k_st, v_st = _commit_layers(kt, vt, kr, vr)
    if not isinstance(path, torch.Tensor) or path.dim() != 2:
        raise ValueError("path must be [rows, most]")
    most = path.shape[1]
    _check_sizes(path.shape)
    _check_i32("path", path, (rows, most))
    _check_i32("length", length, (rows,))
    _check_i32("pos", pos, (rows,))
    dev = kt[0].device
    _same_device(dev, path=path, length=length, pos=pos)
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return tree_commit(kt, vt, kr, vr, path, length, pos, ws, stream)
    ws = _workspace_on(stream, 256, dev, ws, handed_back=True)
    L = len(kt)
    ptrs = [(_P * L)(*[t.data_ptr() for t in ts]) for ts in (kt, vt, kr, vr)]
    rc = lib().wa_tree_commit(
        L, *ptrs, (_I * L)(*[t.shape[1] for t in kr]), rows, nodes, hkv, d,
        ctypes.byref(_TreeStrides(0, 0, *k_st, *v_st, 0, 0)), path.data_ptr(), most, length.data_ptr(), pos.data_ptr(),
        ws.data_ptr(), _ws_bytes(ws), _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_tree_commit")
    return ws


# Rotary positions and a cache in pages.  As the drafted-token calls, these run on their inputs' device and on `stream`
# or that device's current stream.

_ROTARY_LAYOUTS = {"half": _C["WA_ROTARY_HALF"], "interleaved": _C["WA_ROTARY_INTERLEAVED"]}
_PAGE_TYPES = {torch.bfloat16: _C["WA_PAGE_BF16"], torch.float8_e4m3fn: _C["WA_PAGE_E4M3"]}


def rope_frequencies(dims: int, base: float = 10000.0, scaling=None, device=None):
    """(inv_freq fp32 [dims / 2], factor) for rope() and paged_append(): base ** (-2 j / dims), and 1.0.

    ``scaling`` stretches them for positions beyond the ``original`` length of training; s = its "factor":
      {"kind": "linear", "factor"}: every frequency divided by s;
      {"kind": "base", "factor"}: base times s ** (dims / (dims - 2)), which leaves the fastest pair as it is and
          divides the slowest by s;
      {"kind": "wavelength", "factor", "original", "low": 1, "high": 4}: pairs with fewer than `low` turns over the
          original length divided by s, those with more than `high` as they are, in between a blend linear in the turns;
      {"kind": "ramp", "factor", "original", "slow": 1, "fast": 32, "attention": None}: the pairs between the one of
          `fast` turns over the original length and the one of `slow` blended linearly in the pair's index, and both
          sides of the scores grow by `attention` (None: 0.1 ln s + 1), which is the factor returned.
    Worked out in float64 and rounded once.  A scaling that brings a pair's frequency to 16 or more is refused."""
    dims = int(dims)
    if dims <= 0 or dims % 2:
        raise ValueError(f"dims must be even and positive, not {dims}")
    if not (math.isfinite(base) and base > 1.0):
        raise ValueError(f"base must be a number above 1, not {base}")
    if scaling is not None and not isinstance(scaling, dict):
        raise TypeError('scaling must be None or a dict with a "kind"')
    opt = dict(scaling or {"kind": None})
    kind, factor = opt.pop("kind", None), 1.0
    inv = [base ** (-2.0 * j / dims) for j in range(dims // 2)]

    def take(name, *default):
        if name not in opt and not default:
            raise ValueError(f'scaling "{kind}" needs "{name}"')
        x = opt.pop(name, *default)
        if x is not None and not (math.isfinite(x) and x > 0):
            raise ValueError(f'"{name}" must be a positive number, not {x}')
        return x

    if kind is not None:
        s = take("factor")
    if kind == "linear":
        inv = [w / s for w in inv]
    elif kind == "base":
        if dims < 4:
            raise ValueError('scaling "base" needs at least 4 dims')
        stretched = base * s ** (dims / (dims - 2))
        inv = [stretched ** (-2.0 * j / dims) for j in range(dims // 2)]
    elif kind == "wavelength":
        original, lo, hi = take("original"), take("low", 1.0), take("high", 4.0)
        if lo >= hi:
            raise ValueError('"low" must be below "high"')
        keep = [min(1.0, max(0.0, (original * w / (2 * math.pi) - lo) / (hi - lo))) for w in inv]
        inv = [w * (k + (1 - k) / s) for w, k in zip(inv, keep)]
    elif kind == "ramp":
        original, slow, fast, attention = take("original"), take("slow", 1.0), take("fast", 32.0), take("attention", None)
        if slow >= fast:
            raise ValueError('"slow" must be below "fast"')

        def pair(turns):      # the index of the pair with so many turns over the original length
            return dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        first, last = max(0, math.floor(pair(fast))), min(dims - 1, math.ceil(pair(slow)))
        cut = [min(1.0, max(0.0, (j - first) / max(last - first, 1e-3))) for j in range(dims // 2)]
        inv = [w * (1 - c + c / s) for w, c in zip(inv, cut)]
        factor = (0.1 * math.log(s) + 1.0 if s > 1 else 1.0) if attention is None else attention
    elif kind is not None:
        raise ValueError(f'scaling kind must be "linear", "base", "wavelength" or "ramp", not {kind!r}')
    if opt:
        raise ValueError(f"scaling has entries that {kind!r} does not take: {sorted(opt)}")
    inv_freq = torch.tensor(inv, dtype=torch.float64).float()
    if not (inv_freq < 16.0).all():
        raise ValueError(f"a pair's frequency of {max(inv)} is not below 16, which is all that the rotation takes")
    return inv_freq.to(device=device), float(factor)


def _rotary(inv_freq, layout, factor, d: int):
    """The library's description of a rotation (None: none); raises where it is not one of head dim d."""
    if layout not in _ROTARY_LAYOUTS:
        raise ValueError(f'layout must be "half" or "interleaved", not {layout!r}')
    factor = float(_number("factor", factor))
    if inv_freq is None:
        return None
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float32 or not inv_freq.is_cuda:
        raise TypeError("inv_freq must be an fp32 CUDA tensor")
    dims = 2 * inv_freq.numel()
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or dims == 0 or dims % 16 or dims > d:
        raise ValueError(f"inv_freq must be a contiguous vector of a multiple of 8 frequencies, at most {d // 2}")
    if not math.isfinite(factor):
        raise ValueError(f"factor must be finite, not {factor}")
    return _Rotary(inv_freq.data_ptr(), dims, _ROTARY_LAYOUTS[layout], factor)


def _token_rows(name: str, t: torch.Tensor):
    """(token stride, heads, d) of a bf16 [tokens, heads, d] tensor whose tokens do not share memory."""
    _check_bf16(name, t)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, d]")
    n, heads, d = t.shape
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name} must be [tokens, heads, d] with head stride d and unit dim stride")
    tok = int(t.stride(0)) if n > 1 else heads * d
    if tok < heads * d:
        raise ValueError(f"{name}'s tokens must not share memory")
    return tok, heads, d


def rope(x, pos, inv_freq, layout: str = "half", factor: float = 1.0, inverse: bool = False, out=None, stream=None):
    """Rotary positions: x [n, heads, d] bf16 (token-strided), pos int32 [n], inv_freq fp32 [dims / 2] on the GPU.

    Pair (j, j + dims / 2) ("half") or (2 j, 2 j + 1) ("interleaved") of the first dims dims turns by pos * inv_freq[j]
    and grows by ``factor``; the other dims stay.  A frequency of 16 or more in size gives NaN to its
    pair.  ``inverse`` turns back: the gradient of x, given that of the result.  The call itself records nothing for autograd, so
    an output has no history whatever x requires.  Angles are within 2^-25.9 of a turn at every position.  ``out`` may be x
    itself.  Returns out, [n, heads, d] bf16."""
    bind = _short_way() if stream is None else None
    if bind is not None:
        got = bind.rope(x, pos, inv_freq, layout, factor, inverse, out)
        if got is not None:
            return _result(got, "wa_rope")
    x_tok, heads, d = _token_rows("x", x)
    n = x.shape[0]
    _check_sizes(x.shape)
    _check_i32("pos", pos, (n,))
    if inv_freq is None:
        raise TypeError("inv_freq must be an fp32 CUDA tensor")
    rot = _rotary(inv_freq, layout, factor, d)
    if out is not None:
        out_tok = _token_rows("out", out)[0]
        if out.shape != x.shape:
            raise ValueError(f"out must have x's shape {tuple(x.shape)}")
    _same_device(x.device, pos=pos, inv_freq=inv_freq, out=out)
    dev = x.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return rope(x, pos, inv_freq, layout, factor, inverse, out, stream)
    if out is None:
        out, out_tok = _empty((n, heads, d), torch.bfloat16, dev, stream), heads * d
    rc = lib().wa_rope(x.data_ptr(), pos.data_ptr(), n, heads, d, ctypes.byref(rot), int(bool(inverse)), x_tok, out_tok,
                       out.data_ptr(), _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_rope")
    return out


def _pages(k_pages, v_pages, table, k_scale, v_scale):
    """The library's description of a paged cache; raises where its tensors disagree."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor) or t.dtype not in _PAGE_TYPES or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 or float8_e4m3fn CUDA tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [pages, page, hkv, d]")
        if t.stride(3) != 1:
            raise ValueError(f"{name} must have unit dim stride")
    if v_pages.dtype != k_pages.dtype or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have one type and one shape")
    pages, page, hkv, d = k_pages.shape
    if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or not table.is_cuda:
        raise TypeError("table must be an int32 CUDA tensor")
    if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [rows, most] with unit inner stride")
    rows, most = table.shape
    _check_sizes((*k_pages.shape, rows, most))
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None:
            continue
        if k_pages.dtype == torch.bfloat16:
            raise ValueError(f"{name} belongs to pages of 8 bits")
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError(f"{name} must be an fp32 CUDA tensor")
        if t.shape != (hkv,) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and of shape {(hkv,)}")
    _same_device(k_pages.device, v_pages=v_pages, table=table, k_scale=k_scale, v_scale=v_scale)

    def strides(t):       # a dimension of one element may carry any stride
        slot, head = t.stride(1), t.stride(2)
        head = head if hkv > 1 else d
        return (t.stride(0) if pages > 1 else max(slot * page, head * hkv)), slot, head

    def at(t):
        return None if t is None else t.data_ptr()

    return _Pages(k_pages.data_ptr(), v_pages.data_ptr(), at(k_scale), at(v_scale), table.data_ptr(), *strides(k_pages),
                  *strides(v_pages), table.stride(0) if rows > 1 else most, pages, page, rows, most, hkv, d,
                  _PAGE_TYPES[k_pages.dtype])


def paged_append(src, pos, q_out, k_pages, v_pages, table, row=None, inv_freq=None, layout: str = "half",
                 factor: float = 1.0, k_scale=None, v_scale=None, ws=None, stream=None):
    """Append to a paged cache, with the rotation on the way.

    src [n, (hq + 2 hkv) d] bf16 (token-strided): the tokens' query, key and value heads.  The query heads are rotated
    into q_out [n, hq, d] (which may be their place in src), the key heads rotated and the value heads as they are into
    position pos[t] (int32 [n]; -1: a token to leave out) of sequence row[t] (int32 [n], None: sequence t): slot
    pos mod page of page table[row, pos / page] of k_pages / v_pages [pages, page, hkv, d], bf16 or float8_e4m3fn
    (a value is stored as x / scale of its head, k_scale / v_scale fp32 [hkv]).  inv_freq (below 16 in size, or NaN), layout,
    factor as in rope(); None: no rotation.  Returns the workspace, whose status status() reads."""
    bind = _short_way() if stream is None else None
    if bind is not None:
        got = bind.paged_append(src, pos, q_out, k_pages, v_pages, table, row, inv_freq, layout, factor, k_scale, v_scale, ws)
        if got is not None:
            return _result(got, "wa_paged_append")
    _check_bf16("src", src)
    if src.dim() != 2 or (src.shape[1] > 1 and src.stride(1) != 1):
        raise ValueError("src must be [n, row] with unit inner stride")
    cache = _pages(k_pages, v_pages, table, k_scale, v_scale)
    q_tok, hq, d = _token_rows("q_out", q_out)
    n, width = src.shape
    _check_sizes((n, hq))
    if q_out.shape[0] != n or d != cache.d:
        raise ValueError(f"q_out {tuple(q_out.shape)} does not match {n} tokens of head dim {cache.d}")
    if width < (hq + 2 * cache.hkv) * d:
        raise ValueError(f"src rows hold {width} values, fewer than (hq + 2 hkv) d = {(hq + 2 * cache.hkv) * d}")
    src_tok = int(src.stride(0)) if n > 1 else width
    if src_tok < width:
        raise ValueError("src's tokens must not share memory")
    src_tok, q_tok = (src_tok, q_tok) if n > 1 else ((hq + 2 * cache.hkv) * d,) * 2
    _check_i32("pos", pos, (n,))
    if row is not None:
        _check_i32("row", row, (n,))
    elif n > cache.rows:
        raise ValueError(f"{n} tokens of {cache.rows} sequences need `row`")
    rot = _rotary(inv_freq, layout, factor, d)
    _same_device(src.device, pos=pos, q_out=q_out, k_pages=k_pages, row=row, inv_freq=inv_freq)
    dev = src.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return paged_append(src, pos, q_out, k_pages, v_pages, table, row, inv_freq, layout, factor, k_scale, v_scale, ws,
                                stream)
    ws = _workspace_on(stream, 256, dev, ws, handed_back=True)
    rc = lib().wa_paged_append(
        src.data_ptr(), pos.data_ptr(), None if row is None else row.data_ptr(), n, hq, ctypes.byref(cache),
        None if rot is None else ctypes.byref(rot), src_tok, q_tok, q_out.data_ptr(), ws.data_ptr(), _ws_bytes(ws),
        _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_paged_append")
    return ws


def paged_decode_ws_bytes(rows: int, hq: int, hkv: int, d: int, page: int, most: int, win: int = 0,
                          dtype=torch.bfloat16) -> int:
    """Workspace bytes of paged_decode for these sizes (most: the table's columns); 0 for invalid ones.

    They grow with ``most``, whatever the rows hold, and with up to 256 rows: 64/8 heads of 128 and a table for 131,072
    positions take 4.7 MB a row.  Pass the columns that the batch's longest sequence needs (``table[:, :columns]``) to keep
    them small; no row's output depends on it."""
    if not _fit_32_bits(rows, hq, hkv, d, page, most, win) or dtype not in _PAGE_TYPES:
        return 0
    sizes = _Pages(pages=1, page_size=page, rows=rows, most=most, hkv=hkv, d=d, type=_PAGE_TYPES[dtype])
    return int(lib().wa_paged_decode_ws_bytes(ctypes.byref(sizes), hq, win))


def paged_decode(q, k_pages, v_pages, table, pos, win: int = 0, scale: float = 1.0, k_scale=None, v_scale=None, out=None,
                 ws=None, stream=None):
    """Decode over a paged cache, one new token a sequence.

    q [rows, hq, d] bf16 (row-strided); k_pages / v_pages [pages, page, hkv, d], bf16 or float8_e4m3fn with k_scale /
    v_scale fp32 [hkv], in any layout of unit dim stride (heads of positions as a transposed view, keys and values in
    one tensor); table int32 [rows, most]: the page of each `page` positions of a sequence, only those with a visible
    key are read; pos int32 [rows]: the last key's position, -1 for an empty sequence, whose output is zeros.
    Sequence r sees the last ``win`` keys (0: all).  Returns out [rows, hq, d] bf16.  ``ws``: a reused uint8 CUDA buffer
    of paged_decode_ws_bytes(...)."""
    bind = _short_way() if stream is None else None
    if bind is not None:
        got = bind.paged_decode(q, k_pages, v_pages, table, pos, win, scale, k_scale, v_scale, out, ws)
        if got is not None:
            return _result(got, "wa_paged_decode")
    q_row, hq, d = _token_rows("q", q)
    cache = _pages(k_pages, v_pages, table, k_scale, v_scale)
    _check_sizes(q.shape)
    if q.shape[0] != cache.rows or d != cache.d:
        raise ValueError(f"q {tuple(q.shape)} does not match {cache.rows} sequences of head dim {cache.d}")
    _check_i32("pos", pos, (cache.rows,))
    if out is not None:
        out_row = _token_rows("out", out)[0]
        if out.shape != q.shape:
            raise ValueError(f"out must have q's shape {tuple(q.shape)}")
    win, scale = _window(win), float(_number("scale", scale))
    _same_device(q.device, k_pages=k_pages, pos=pos, out=out)
    dev = q.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return paged_decode(q, k_pages, v_pages, table, pos, win, scale, k_scale, v_scale, out, ws, stream)
    if out is None:
        out, out_row = _empty(q.shape, torch.bfloat16, dev, stream), hq * d
    ws = _workspace_on(stream, int(lib().wa_paged_decode_ws_bytes(ctypes.byref(cache), hq, win)), dev, ws)
    rc = lib().wa_paged_decode(q.data_ptr(), pos.data_ptr(), hq, ctypes.byref(cache), win, scale, q_row, out_row,
                               out.data_ptr(), ws.data_ptr(), _ws_bytes(ws), _stream_on(dev.index, stream))
    if rc != WA_OK:
        raise WAError(rc, "wa_paged_decode")
    return out


def status(ws, stream=None) -> int:
    """WA_STATUS_* bits of the last call on ``ws`` (waits for the stream); ``ws`` None reads those
    of the last decode_static call on the current device."""
    rc = lib().wa_status(None if ws is None else ws.data_ptr(), _stream_handle(stream))
    if rc < 0:
        raise WAError(rc, "wa_status")
    return rc
