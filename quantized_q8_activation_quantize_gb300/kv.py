"""Thin ctypes binding over the paged 8-bit KV cache of libmq.so (include/mqkv.h).  Argument marshalling only.

Every ``mqkv_*`` function has the name of the C entry point it calls and takes torch CUDA tensors; shapes, strides and
dtypes are read off them.  ``cache`` and ``sequences`` make the two descriptions that the calls take (they hold on to the
tensors they describe), ``alloc_*`` the memory a user owns.  As in ``binding``, there is no Python or CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import binding
from .binding import MQ_ERR_ARG, MQError, _check, _stream

HEADER = os.path.join(os.path.dirname(binding.HEADER), "mqkv.h")
MQKV_ERR_STATE = -7
binding.STATUS_NAMES.setdefault(MQKV_ERR_STATE, "MQKV_ERR_STATE")
BLOCK = 32                                   # tokens that share one scale per head and half


class Layout(ctypes.Structure):
    _fields_ = [("off_v", ctypes.c_size_t), ("off_scales", ctypes.c_size_t), ("layer_bytes", ctypes.c_size_t),
                ("page_bytes", ctypes.c_size_t)]


class Cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_layers", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


class Sequences(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_L = None


def header_functions():
    """The C entry points include/mqkv.h declares."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mqkv_\w+)\s*\(", text)))


def lib():
    """The loaded libmq.so with this header's argument types (raises if it was not built)."""
    global _L
    if _L is None:
        L = binding.lib()
        P, I64, I32, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        C, S = ctypes.POINTER(Cache), ctypes.POINTER(Sequences)
        rows = [P, I64, I64]
        types = {
            "mqkv_page_layout": [I32, I32, I32, I32, ctypes.POINTER(Layout)],
            "mqkv_append": [C, S, I32, I32, *rows, *rows, P, I64, P],
            "mqkv_read": [C, S, I32, I32, *rows, *rows, P, P, I64, P],
            "mqkv_attention": [C, S, I32, I32, *rows, *rows, I32, P, I64, I64, I64, I32, I64, F, P, SZ, P],
            "mqkv_attention_workspace_bytes": [C, S, I32, I32, I64, I64, I64],
            "mqkv_pages_workspace_bytes": [C, S],
            "mqkv_extend": [C, S, P, P, SZ, P],
            "mqkv_release": [C, S, P, I32, P],
            "mqkv_fork": [C, S, P, P, I32, P, SZ, P],
            "mqkv_compact": [C, S, P, SZ, P],
            "mqkv_copy_pages": [C, P, P, I32, P],
            "mqkv_device_status": [P],
        }
        for name, args in types.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = SZ if name.endswith("_bytes") else ctypes.c_int
        _L = L
    return _L


_DTYPES = {}
_int32 = _raw_stream = None


def _torch():
    """What of torch the calls need, resolved on the first one (the package imports without torch)."""
    global _int32, _raw_stream
    import torch
    _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    _int32 = torch.int32
    # the current stream's handle without making a Stream object of it (3 us a call); the public way where there is none
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(stream, t):
    """The handle of a stream, None: the current one of the tensor's device."""
    if stream is None:
        if _raw_stream is None:
            _torch()
        return _raw_stream(t.get_device())
    return _stream(stream)


def _dtype(t) -> int:
    if not _DTYPES:
        _torch()
    d = _DTYPES.get(t)
    if d is None:
        raise MQError(MQ_ERR_ARG, f"dtype {t} is none of float32, float16, bfloat16")
    return d


def _bad(message):
    raise MQError(MQ_ERR_ARG, message)


def _rows(name, t, n, heads, dim):
    """(pointer, token stride, head stride) of a [n, heads, dim] CUDA tensor."""
    if t.shape != (n, heads, dim):
        _bad(f"{name} has shape {tuple(t.shape)}, [{n}, {heads}, {dim}] wanted")
    if not t.is_cuda:
        _bad(f"{name} is not a CUDA tensor")
    a, b, c = t.stride()
    if c != 1 and n:
        _bad(f"{name}: head_dim is not contiguous (strides {t.stride()})")
    return t.data_ptr(), a, b


def _i32(name, t, n=None):
    if t is None:
        return None
    if _int32 is None:
        _torch()
    if t.dtype is not _int32 or not t.is_contiguous() or not t.is_cuda or (n is not None and t.numel() != n):
        _bad(f"{name} is not a contiguous int32 CUDA tensor{'' if n is None else f' of {n}'}")
    return t.data_ptr()


def _ws(t):
    """(pointer, bytes) of a workspace: contiguous CUDA memory of any type."""
    if not t.is_cuda or not t.is_contiguous():
        _bad("the workspace is not a contiguous CUDA tensor")
    return t.data_ptr(), t.numel() * t.element_size()


# ----------------------------------------------------------------------- descriptions, memory ---

def mqkv_page_layout(n_layers: int, n_kv_heads: int, head_dim: int, page_tokens: int) -> dict:
    out = Layout()
    _check(lib().mqkv_page_layout(n_layers, n_kv_heads, head_dim, page_tokens, ctypes.byref(out)))
    return {f: getattr(out, f) for f, _ in Layout._fields_}


def alloc_pool(n_pages: int, n_layers: int, n_kv_heads: int, head_dim: int, page_tokens: int, device="cuda"):
    """(pool uint8 [n_pages, page_bytes], refs int32 [n_pages] of zeros)."""
    import torch
    size = mqkv_page_layout(n_layers, n_kv_heads, head_dim, page_tokens)["page_bytes"]
    return (torch.empty((n_pages, size), dtype=torch.uint8, device=device),
            torch.zeros(n_pages, dtype=torch.int32, device=device))


def cache(pool, refs, n_layers: int, n_kv_heads: int, head_dim: int, page_tokens: int) -> Cache:
    """The description of a pool (uint8 [n_pages, page_bytes], contiguous); refs int32 [n_pages] or None."""
    import torch
    size = mqkv_page_layout(n_layers, n_kv_heads, head_dim, page_tokens)["page_bytes"]
    if pool.dtype is not torch.uint8 or pool.dim() != 2 or pool.shape[1] != size or not pool.is_contiguous() or not pool.is_cuda:
        _bad(f"pool is not a contiguous uint8 CUDA tensor of [n_pages, {size}]")
    c = Cache(pool.data_ptr(), _i32("refs", refs, pool.shape[0]), pool.shape[0], n_layers, n_kv_heads, head_dim, page_tokens)
    c.tensors = (pool, refs)
    return c


def sequences(page_table, kv_len) -> Sequences:
    """The description of a page table (int32 [n_seqs, max_pages]) and its lengths (int32 [n_seqs])."""
    if page_table.dim() != 2:
        _bad(f"page_table has shape {tuple(page_table.shape)}, [n_seqs, max_pages] wanted")
    s = Sequences(_i32("page_table", page_table), _i32("kv_len", kv_len, page_table.shape[0]), *page_table.shape)
    s.tensors = (page_table, kv_len)
    return s


def _bytes(n):
    import torch
    if n == 0:
        raise MQError(MQ_ERR_ARG, binding.last_error() or "invalid sizes")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def mqkv_attention_workspace_bytes(cache, seqs, dtype, n_q_heads: int, n_tokens: int, max_q: int, max_kv: int) -> int:
    return lib().mqkv_attention_workspace_bytes(cache, seqs, _dtype(dtype), n_q_heads, n_tokens, max_q, max_kv)


def alloc_attention_workspace(cache, seqs, n_q_heads: int, n_tokens: int, max_q: int, max_kv: int, dtype):
    return _bytes(mqkv_attention_workspace_bytes(cache, seqs, dtype, n_q_heads, n_tokens, max_q, max_kv))


def mqkv_pages_workspace_bytes(cache, seqs) -> int:
    return lib().mqkv_pages_workspace_bytes(cache, seqs)


def alloc_pages_workspace(cache, seqs):
    return _bytes(mqkv_pages_workspace_bytes(cache, seqs))


# --------------------------------------------------------------------------------- entry points ---

def mqkv_append(cache, seqs, layer: int, k, v, cu=None, stream=None):
    """k, v [tokens, n_kv_heads, head_dim] are the last tokens of their sequences (cu int32 [n_seqs + 1], or as many
    for each)."""
    n, H, D = len(k), cache.n_kv_heads, cache.head_dim
    dtype = k.dtype
    if v.dtype is not dtype:
        _bad(f"k is {dtype}, v is {v.dtype}")
    return _check((_L or lib()).mqkv_append(cache, seqs, layer, _dtype(dtype), *_rows("k", k, n, H, D), *_rows("v", v, n, H, D),
                                            _i32("cu", cu, seqs.n_seqs + 1), n, _on(stream, k)))


def mqkv_read(cache, seqs, layer: int, k, v, cu=None, start=None, stream=None):
    """Into k, v [tokens, n_kv_heads, head_dim] (either may be None) the cached values from position start (int32
    [n_seqs]) of each sequence on, or the last ones."""
    t = k if k is not None else v
    if t is None:
        _bad("both outputs are None")
    n, H, D = len(t), cache.n_kv_heads, cache.head_dim
    if k is not None and v is not None and v.dtype is not k.dtype:
        _bad(f"k is {k.dtype}, v is {v.dtype}")
    none = (None, 0, 0)
    return _check((_L or lib()).mqkv_read(cache, seqs, layer, _dtype(t.dtype), *(none if k is None else _rows("k", k, n, H, D)),
                                          *(none if v is None else _rows("v", v, n, H, D)), _i32("cu", cu, seqs.n_seqs + 1),
                                          _i32("start", start, seqs.n_seqs), n, _on(stream, t)))


def mqkv_attention(cache, seqs, layer: int, q, out, cu, max_q: int, max_kv: int, workspace, causal: bool = True,
                   window: int = 0, scale: float | None = None, stream=None):
    """out = softmax(scale q K^T + mask) V for q, out [tokens, n_q_heads, head_dim]; scale None: 1 / sqrt(head_dim)."""
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        _bad(f"q has shape {tuple(shape)}, [tokens, heads, head_dim] wanted")
    n, heads, D = shape[0], shape[1], cache.head_dim
    if out.dtype is not dtype:
        _bad(f"q is {dtype}, out is {out.dtype}")
    return _check((_L or lib()).mqkv_attention(cache, seqs, layer, _dtype(dtype), *_rows("q", q, n, heads, D),
                                               *_rows("out", out, n, heads, D), heads, _i32("cu", cu, seqs.n_seqs + 1), n, max_q,
                                               max_kv, causal, window, D ** -0.5 if scale is None else scale,
                                               *_ws(workspace), _on(stream, q)))


def mqkv_extend(cache, seqs, add, workspace, stream=None):
    """kv_len += add (int32 [n_seqs]; None: 1), with pages for the new tokens."""
    return _check((_L or lib()).mqkv_extend(cache, seqs, _i32("add", add, seqs.n_seqs), *_ws(workspace), _on(stream, workspace)))


def mqkv_release(cache, seqs, ids, stream=None):
    return _check((_L or lib()).mqkv_release(cache, seqs, _i32("ids", ids), ids.numel(), _on(stream, ids)))


def mqkv_fork(cache, seqs, parent, child, workspace, stream=None):
    n = parent.numel()
    return _check((_L or lib()).mqkv_fork(cache, seqs, _i32("parent", parent), _i32("child", child, n), n, *_ws(workspace),
                                          _on(stream, workspace)))


def mqkv_compact(cache, seqs, workspace, stream=None):
    return _check((_L or lib()).mqkv_compact(cache, seqs, *_ws(workspace), _on(stream, workspace)))


def mqkv_copy_pages(cache, src, dst, stream=None):
    return _check((_L or lib()).mqkv_copy_pages(cache, _i32("src", src), _i32("dst", dst, src.numel()), src.numel(), _on(stream, src)))


def mqkv_device_status(stream=None):
    return _check(lib().mqkv_device_status(_stream(stream)))
