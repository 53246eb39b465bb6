"""Thin ctypes binding over include/mqd.h: what a decoder layer does between its matrix products and its cache, and what picks
the tokens at its end.  Argument marshalling only.

Every ``mqd_*`` function has the name of the C entry point it calls and takes torch CUDA tensors; sizes, strides and dtypes are
read off them.  ``rope_plan`` makes the description that the rotations take, ``alloc_*`` the memory a user owns.  As in ``binding``, there is
no Python or CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

from . import binding
from .binding import _check
from .kv import _bad, _bytes, _dtype, _i32, _on, _rows, _ws

HEADER = os.path.join(os.path.dirname(binding.HEADER), "mqd.h")
SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3, "index": 4}


class RopePlan(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float)]


_L = None


def header_functions():
    """The C entry points include/mqd.h declares."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mqd_\w+)\s*\(", text)))


def lib():
    """The loaded libmq.so with this header's argument types (raises if it was not built)."""
    global _L
    if _L is None:
        L = binding.lib()
        P, I64, I32, SZ, F, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float, ctypes.c_double
        types = {
            "mqd_add_quantize_q8": [I32, P, I64, P, I64, P, I64, I64, I64, P, F, ctypes.c_uint, P, P],
            "mqd_dequantize_q8": [P, I64, I64, ctypes.c_uint, I32, P, I64, P],
            "mqd_rope_turns": [I32, D, I32, D, D, D, D, P, P],
            "mqd_rope": [ctypes.POINTER(RopePlan), I32, P, I64, I64, P, I64, I64, I64, I32, I32, P, P],
            "mqd_beam_workspace_bytes": [I64, I32, I64, I32],
            "mqd_beam_select": [I32, P, I64, I64, I32, I64, P, I32, I32, P, P, P, P, P, P, P, SZ, P],
        }
        for name, args in types.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = SZ if name.endswith("_bytes") else ctypes.c_int
        _L = L
    return _L


_float32 = _int32 = None


def _types():
    """What of torch the calls compare with, resolved on the first one."""
    global _float32, _int32
    import torch
    _float32, _int32 = torch.float32, torch.int32


def _mat(name, t, shape):
    """(pointer, row stride) of a CUDA tensor of this shape [rows, columns] with contiguous rows."""
    if t.shape != shape or not t.is_cuda:
        _bad(f"{name} is not a CUDA tensor of {list(shape)}, but {tuple(t.shape)} on {t.device}")
    a, b = t.stride()
    if b != 1 and shape[1] > 1:
        _bad(f"{name}: rows are not contiguous (strides {t.stride()})")
    return t.data_ptr(), a if shape[0] > 1 else shape[1]


def _two(name, t):
    if len(t.shape) != 2:
        _bad(f"{name} has shape {tuple(t.shape)}, two dimensions wanted")
    return t.shape


def _f32(name, t, shape):
    if _float32 is None:
        _types()
    if t.dtype is not _float32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(f"{name} is not a contiguous float32 CUDA tensor of {list(shape)}")
    return t.data_ptr()


def _ints(name, t, shape):
    if t.dtype is not _int32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(f"{name} is not a contiguous int32 CUDA tensor of {list(shape)}")
    return t.data_ptr()


_plane_bytes = functools.lru_cache(maxsize=256)(binding.mq_q8_plane_bytes)


def _bad_plane(M, K):
    _bad(f"the plane is not contiguous CUDA memory of {_plane_bytes(M, K)} bytes")


# ------------------------------------------------------------------ residual, RMSNorm, Q8 plane ---

def mqd_add_quantize_q8(x, res, h, rms_w, eps: float, sections: int, plane, stream=None):
    """h = x + res ([M, K], one dtype; x None: no addition, h is not used) and the Q8 plane of RMSNorm(h) rms_w."""
    shape, dtype = res.shape, res.dtype
    M, K = _two("res", res)
    if x is None:
        a = b = (None, 0)
    else:
        if x.dtype is not dtype or h.dtype is not dtype:
            _bad(f"x is {x.dtype}, res is {dtype}, h is {h.dtype}")
        a, b = _mat("x", x, shape), _mat("h", h, shape)
    if isinstance(plane, int):
        at = plane
    else:
        at = plane.data_ptr()
        if plane.nbytes < _plane_bytes(M, K) or not plane.is_cuda or not plane.is_contiguous():
            _bad_plane(M, K)
    return _check((_L or lib()).mqd_add_quantize_q8(_dtype(dtype), *a, *_mat("res", res, shape), *b, M, K, _f32("rms_w", rms_w, (K,)), eps, sections, at,
                                                    _on(stream, res)))


def mqd_dequantize_q8(plane, sections: int, y, stream=None):
    """The values of the plane of a y.shape activation into y (any of the three dtypes); sections: what the plane holds."""
    M, K = _two("y", y)
    out = _mat("y", y, y.shape)
    if isinstance(plane, int):
        at = plane
    else:
        at = plane.data_ptr()
        if plane.nbytes < _plane_bytes(M, K) or not plane.is_cuda or not plane.is_contiguous():
            _bad_plane(M, K)
    return _check((_L or lib()).mqd_dequantize_q8(at, M, K, sections, _dtype(y.dtype), *out, _on(stream, y)))


# ----------------------------------------------------------------------------- rotary positions ---

def mqd_rope_turns(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 0.0, low: float = 1.0,
                   high: float = 4.0, factors=None) -> list[int]:
    """The turns per position of every pair, as 64-bit fractions of a turn (include/mqd.h has the formulas)."""
    if scaling not in SCALINGS:
        _bad(f"scaling {scaling!r} is none of {', '.join(SCALINGS)}")
    n = max(rot_dim // 2, 1)
    if factors is not None and len(factors) != n:
        _bad(f"{len(factors)} factors, {n} wanted")
    out = (ctypes.c_uint64 * n)()
    _check(lib().mqd_rope_turns(rot_dim, base, SCALINGS[scaling], factor, original, low, high,
                                None if factors is None else (ctypes.c_double * n)(*factors), out))
    return list(out)


def rope_plan(rot_dim: int, base: float = 10000.0, interleaved: bool = False, amplitude: float = 1.0, device="cuda", **scaling) -> RopePlan:
    """The description of a rotation (``scaling`` as in mqd_rope_turns), with its table on the device."""
    import torch
    table = torch.tensor([t - (1 << 64) if t >> 63 else t for t in mqd_rope_turns(rot_dim, base, **scaling)], dtype=torch.int64, device=device)
    if not table.is_cuda:
        _bad(f"the table of a rotation is read by kernels: device {device} is not a CUDA device")
    p = RopePlan(table.data_ptr(), rot_dim, interleaved, amplitude)
    p.tensors = (table,)
    return p


def mqd_rope(plan, x, out, pos, stream=None):
    """out = x [tokens, heads, head_dim] with the first rot_dim values of every head turned by pos (int32 [tokens]); out may be x."""
    if x.dim() != 3 or out.dtype is not x.dtype:
        _bad(f"x {tuple(x.shape)} of {x.dtype} into {out.dtype}: [tokens, heads, head_dim] of one dtype wanted")
    n, heads, dim = x.shape
    return _check((_L or lib()).mqd_rope(plan, _dtype(x.dtype), *_rows("x", x, n, heads, dim), *_rows("out", out, n, heads, dim), n, heads, dim,
                                         _i32("pos", pos, n), _on(stream, x)))


# -------------------------------------------------------------------------------- beam search ---

def mqd_beam_workspace_bytes(n_groups: int, n_beams: int, vocab: int, n_cand: int) -> int:
    return lib().mqd_beam_workspace_bytes(n_groups, n_beams, vocab, n_cand)


def alloc_beam_workspace(n_groups: int, n_beams: int, vocab: int, n_cand: int):
    return _bytes(mqd_beam_workspace_bytes(n_groups, n_beams, vocab, n_cand))


def _triple(name, t, rows, n):
    """(score f32, row int32, token int32) of [rows, n] each"""
    score, row, token = t
    shape = rows, n
    return _f32(name, score, shape), _ints(name, row, shape), _ints(name, token, shape)


def mqd_beam_select(logits, scores, cand, next, stop: int, workspace, stream=None):
    """The best continuations of logits [n_groups * n_beams, vocab] by scores (f32 [n_groups, n_beams]): cand = (score f32, row int32, token
    int32) of [n_groups, n_cand] each; next (or None) the same of [n_groups, n_beams], without the token `stop` (-1: none)."""
    if len(scores.shape) != 2:
        _bad(f"scores has shape {tuple(scores.shape)}, [n_groups, n_beams] wanted")
    G, B = scores.shape
    V, n = logits.shape[-1], cand[0].shape[-1]
    own = _f32("scores", scores, scores.shape)
    p, stride = _mat("logits", logits, (G * B, V))
    return _check((_L or lib()).mqd_beam_select(_dtype(logits.dtype), p, stride, G, B, V, own, n, stop, *_triple("cand", cand, G, n),
                                                *((None,) * 3 if next is None else _triple("next", next, G, B)), *_ws(workspace), _on(stream, logits)))
