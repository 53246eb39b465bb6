"""Host-side tests of the KV cache's C ABI: what include/mqkv.h declares is exported and bound, the page layout, and the
refusals that need no GPU."""
import ctypes
import subprocess

import numpy as np
import pytest

from quantized_q8_activation_quantize_gb300 import binding as B
from quantized_q8_activation_quantize_gb300 import build as mqbuild
from quantized_q8_activation_quantize_gb300 import kv
from tests import kv_util as U


@pytest.fixture(scope="session")
def L():
    mqbuild.build()
    return kv.lib()


def test_header_library_and_binding_agree(L):
    names = set(kv.header_functions())
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    assert {ln.split()[-1] for ln in out.splitlines() if ln.split() and ln.split()[-1].startswith("mqkv_")} == names
    for name in names:
        assert callable(getattr(kv, name)), name


@pytest.mark.parametrize("layers,heads,dim,page", [(1, 1, 64, 32), (28, 4, 128, 64), (2, 3, 64, 256), (5, 8, 128, 128)])
def test_page_layout(L, layers, heads, dim, page):
    lay = kv.mqkv_page_layout(layers, heads, dim, page)
    m = U.Model(1, layers, heads, dim, page)
    assert lay == {"off_v": heads * page * dim, "off_scales": m.off_s, "layer_bytes": m.slab, "page_bytes": layers * m.slab}
    assert lay["layer_bytes"] % 256 == 0 and lay["layer_bytes"] - lay["off_scales"] >= 8 * heads * page // 32


@pytest.mark.parametrize("args", [(0, 4, 128, 64), (1, 0, 128, 64), (1, 4, 96, 64), (1, 4, 256, 64), (1, 4, 128, 16), (1, 4, 128, 96),
                                  (1, 4, 128, 512), (5000, 4, 128, 64), (1, 1000, 128, 64), (-1, 4, 128, 64)])
def test_page_layout_refusals(L, args):
    with pytest.raises(B.MQError) as e:
        kv.mqkv_page_layout(*args)
    assert e.value.status == B.MQ_ERR_SHAPE


POOL, REFS, TABLE, LEN = 1 << 32, 1 << 20, 2 << 20, 3 << 20
K, V, Q, OUT, CU, WS = 1 << 24, 2 << 24, 3 << 24, 4 << 24, 5 << 20, 1 << 28


def cache(**kw):
    f = dict(pool=POOL, refs=REFS, n_pages=10, n_layers=2, n_kv_heads=4, head_dim=128, page_tokens=64)
    return kv.Cache(**{**f, **kw})


def seqs(**kw):
    return kv.Sequences(**{**dict(page_table=TABLE, kv_len=LEN, n_seqs=3, max_pages=5), **kw})


BAD_CACHES = [(dict(pool=None), B.MQ_ERR_ARG), (dict(pool=POOL + 128), B.MQ_ERR_ALIGN), (dict(n_pages=0), B.MQ_ERR_SHAPE),
              (dict(n_pages=1 << 31), B.MQ_ERR_SHAPE), (dict(head_dim=96), B.MQ_ERR_SHAPE), (dict(page_tokens=48), B.MQ_ERR_SHAPE),
              (dict(n_layers=0), B.MQ_ERR_SHAPE), (dict(refs=REFS + 2), B.MQ_ERR_ALIGN)]
BAD_SEQS = [(dict(page_table=None), B.MQ_ERR_ARG), (dict(kv_len=None), B.MQ_ERR_ARG), (dict(n_seqs=-1), B.MQ_ERR_ARG), (dict(n_seqs=1 << 24), B.MQ_ERR_SHAPE),
            (dict(max_pages=0), B.MQ_ERR_SHAPE), (dict(max_pages=-2), B.MQ_ERR_ARG), (dict(page_table=TABLE + 1), B.MQ_ERR_ALIGN)]


def calls(L):
    """every entry point that takes a cache and sequences, as f(cache, sequences)"""
    return {
        "append": lambda c, s: L.mqkv_append(c, s, 0, 0, K, 512, 128, V, 512, 128, CU, 7, None),
        "read": lambda c, s: L.mqkv_read(c, s, 0, 0, K, 512, 128, V, 512, 128, CU, None, 7, None),
        "attention": lambda c, s: L.mqkv_attention(c, s, 0, 0, Q, 1024, 128, OUT, 1024, 128, 8, CU, 7, 4, 100, 1, 0, 0.1, WS, 1 << 24, None),
        "extend": lambda c, s: L.mqkv_extend(c, s, None, WS, 1 << 20, None),
        "release": lambda c, s: L.mqkv_release(c, s, CU, 2, None),
        "fork": lambda c, s: L.mqkv_fork(c, s, CU, CU, 1, WS, 1 << 20, None),
        "compact": lambda c, s: L.mqkv_compact(c, s, WS, 1 << 20, None),
    }


@pytest.mark.parametrize("name", ["append", "read", "attention", "extend", "release", "fork", "compact"])
def test_descriptions_are_checked(L, name):
    f = calls(L)[name]
    for kw, status in BAD_CACHES:
        assert f(cache(**kw), seqs()) == status, kw
        assert B.last_error()
    for kw, status in BAD_SEQS:
        assert f(cache(), seqs(**kw)) == status, kw
    assert f(None, seqs()) == B.MQ_ERR_ARG and f(cache(), None) == B.MQ_ERR_ARG
    if name in ("extend", "release", "fork", "compact"):
        assert f(cache(refs=None), seqs()) == B.MQ_ERR_ARG


def test_append_and_read_refusals(L):
    ok = [cache(), seqs(), 0, 0, K, 512, 128, V, 512, 128, CU, 7, None]

    def rc(f, **at):
        a = list(ok) if f is L.mqkv_append else ok[:11] + [None] + ok[11:]
        for i, x in at.items():
            a[int(i[1:])] = x
        return f(*a)
    for f in (L.mqkv_append, L.mqkv_read):
        assert rc(f, _2=2) == B.MQ_ERR_ARG and rc(f, _2=-1) == B.MQ_ERR_ARG              # layer
        assert rc(f, _3=3) == B.MQ_ERR_ARG and rc(f, _3=-1) == B.MQ_ERR_ARG              # dtype
        assert rc(f, _4=K + 8) == B.MQ_ERR_ALIGN and rc(f, _7=V + 4) == B.MQ_ERR_ALIGN   # 4 elements
        assert rc(f, _3=1, _4=K + 4) == B.MQ_ERR_ALIGN
        assert rc(f, _5=510) == B.MQ_ERR_ALIGN and rc(f, _9=130) == B.MQ_ERR_ALIGN       # strides
        assert rc(f, _5=-512) == B.MQ_ERR_ARG
        assert rc(f, _10=CU + 2) == B.MQ_ERR_ALIGN
        assert rc(f, _4=POOL + 256) == B.MQ_ERR_ARG and "overlap" in B.last_error()
        assert rc(f, _10=None) == B.MQ_ERR_ARG                                         # 7 tokens, 3 sequences, no cu
    assert rc(L.mqkv_append, _4=None) == B.MQ_ERR_ARG and rc(L.mqkv_append, _7=None) == B.MQ_ERR_ARG
    assert rc(L.mqkv_append, _11=-1) == B.MQ_ERR_SHAPE and rc(L.mqkv_append, _11=0) == B.MQ_OK
    assert rc(L.mqkv_read, _4=None, _7=None) == B.MQ_ERR_ARG
    assert rc(L.mqkv_read, _5=256) == B.MQ_ERR_ARG and "overlap" in B.last_error()      # rows of the output overlap
    assert rc(L.mqkv_read, _11=LEN + 1) == B.MQ_ERR_ALIGN and rc(L.mqkv_read, _12=0) == B.MQ_OK
    assert L.mqkv_append(cache(), seqs(n_seqs=0), 0, 0, K, 512, 128, V, 512, 128, CU, 7, None) == B.MQ_ERR_ARG


def test_attention_refusals(L):
    need = L.mqkv_attention_workspace_bytes(cache(), seqs(), 0, 8, 7, 4, 100)
    assert need > 0
    ok = [cache(), seqs(), 0, 0, Q, 1024, 128, OUT, 1024, 128, 8, CU, 7, 4, 100, 1, 0, 0.1, WS, need, None]

    def rc(**at):
        a = list(ok)
        for i, x in at.items():
            a[int(i[1:])] = x
        return L.mqkv_attention(*a)
    assert rc(_2=2) == B.MQ_ERR_ARG and rc(_3=5) == B.MQ_ERR_ARG
    assert rc(_4=None) == B.MQ_ERR_ARG and rc(_7=None) == B.MQ_ERR_ARG
    assert rc(_4=Q + 4) == B.MQ_ERR_ALIGN and rc(_5=1022) == B.MQ_ERR_ALIGN
    assert rc(_10=6) == B.MQ_ERR_SHAPE and rc(_10=0) == B.MQ_ERR_SHAPE                  # not a multiple of the KV heads
    assert rc(_8=512) == B.MQ_ERR_ARG                                                  # rows of out overlap
    assert rc(_12=0) == B.MQ_OK and rc(_13=0) == B.MQ_ERR_ARG and rc(_13=-1) == B.MQ_ERR_SHAPE and rc(_14=-1) == B.MQ_ERR_SHAPE
    assert rc(_11=None, _12=9, _13=2) == B.MQ_ERR_ARG                                  # three rows each, max_q 2
    assert rc(_16=-1) == B.MQ_ERR_ARG
    assert rc(_17=float("nan")) == B.MQ_ERR_ARG and rc(_17=float("inf")) == B.MQ_ERR_ARG
    assert rc(_18=None) == B.MQ_ERR_ARG and rc(_18=WS + 16) == B.MQ_ERR_ALIGN
    assert rc(_19=need - 1) == B.MQ_ERR_ARG and "workspace" in B.last_error()
    assert rc(_7=Q + 4096) == B.MQ_ERR_ARG and rc(_7=POOL) == B.MQ_ERR_ARG and rc(_18=POOL + 256) == B.MQ_ERR_ARG
    for bad in [(cache(head_dim=80), seqs(), 0, 8, 7, 4, 100), (cache(), seqs(), 9, 8, 7, 4, 100), (cache(), seqs(), 0, 7, 7, 4, 100),
                (cache(), seqs(), 0, 8, -1, 4, 100)]:
        assert L.mqkv_attention_workspace_bytes(*bad) == 0


def test_pages_refusals(L):
    c, s = cache(), seqs()
    need = L.mqkv_pages_workspace_bytes(c, s)
    assert need > 0 and L.mqkv_pages_workspace_bytes(cache(n_pages=0), s) == 0
    for f in (lambda ws, n: L.mqkv_extend(c, s, None, ws, n, None), lambda ws, n: L.mqkv_fork(c, s, CU, CU, 1, ws, n, None),
              lambda ws, n: L.mqkv_compact(c, s, ws, n, None)):
        assert f(None, need) == B.MQ_ERR_ARG and f(WS + 64, need) == B.MQ_ERR_ALIGN and f(WS, need - 1) == B.MQ_ERR_ARG
    assert L.mqkv_extend(c, s, CU + 2, WS, need, None) == B.MQ_ERR_ALIGN
    assert L.mqkv_release(c, s, None, 1, None) == B.MQ_ERR_ARG and L.mqkv_release(c, s, CU, 4, None) == B.MQ_ERR_ARG
    assert L.mqkv_release(c, s, CU, -1, None) == B.MQ_ERR_ARG and L.mqkv_release(c, s, CU, 0, None) == B.MQ_OK
    assert L.mqkv_fork(c, s, CU, None, 1, WS, need, None) == B.MQ_ERR_ARG and L.mqkv_fork(c, s, CU, CU, 0, WS, need, None) == B.MQ_OK
    assert L.mqkv_copy_pages(c, CU, None, 1, None) == B.MQ_ERR_ARG and L.mqkv_copy_pages(c, CU, CU, -1, None) == B.MQ_ERR_ARG
    assert L.mqkv_copy_pages(c, CU + 1, CU, 1, None) == B.MQ_ERR_ALIGN and L.mqkv_copy_pages(c, CU, CU, 0, None) == B.MQ_OK
    for f in (lambda s0: L.mqkv_extend(c, s0, None, WS, need, None), lambda s0: L.mqkv_compact(c, s0, WS, need, None)):
        assert f(seqs(n_seqs=0)) == B.MQ_OK


def test_valid_calls_without_a_device_fail_loudly(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for name, f in calls(L).items():
        assert f(cache(), seqs()) in (B.MQ_ERR_CUDA, B.MQ_ERR_DEVICE), name
        assert B.last_error()


def test_binding_refuses_wrong_tensors(L):
    import torch
    with pytest.raises(B.MQError):
        kv.cache(torch.zeros((2, 100), dtype=torch.uint8), None, 1, 1, 64, 32)
    with pytest.raises(B.MQError):
        kv.sequences(torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    c, s = cache(), seqs()
    with pytest.raises(B.MQError):
        kv.mqkv_append(c, s, 0, torch.zeros((7, 4, 128)), torch.zeros((7, 4, 128), dtype=torch.float16))
    with pytest.raises(B.MQError):
        kv.mqkv_append(c, s, 0, torch.zeros((7, 4, 64)), torch.zeros((7, 4, 64)))
    with pytest.raises(B.MQError):
        kv.mqkv_append(c, s, 0, torch.zeros((7, 4, 128), dtype=torch.float64), torch.zeros((7, 4, 128), dtype=torch.float64))


def test_binding_refuses_a_workspace_that_is_not_the_device_s(L, monkeypatch):
    import torch

    class OnDevice:                                          # a tensor of a device, as far as the binding looks
        is_cuda, dtype = True, torch.int32

        def __init__(self, shape, stride, size=4, contiguous=True):
            self.shape, self.size, self.contiguous, self.strides = shape, size, contiguous, stride

        numel = lambda self: int(np.prod(self.shape))        # noqa: E731
        element_size = lambda self: self.size                # noqa: E731
        is_contiguous = lambda self: self.contiguous         # noqa: E731
        data_ptr = lambda self: WS                           # noqa: E731
        get_device = lambda self: 0                          # noqa: E731
        stride = lambda self: self.strides                   # noqa: E731
    c, s = cache(), seqs()
    monkeypatch.setattr(kv, "_on", lambda stream, t: None)
    ids = OnDevice((1,), (1,))
    q, out = OnDevice((3, 8, 128), (1024, 128, 1)), OnDevice((3, 8, 128), (1024, 128, 1))
    q.dtype = out.dtype = torch.float32
    calls = [lambda ws: kv.mqkv_extend(c, s, None, ws), lambda ws: kv.mqkv_fork(c, s, ids, ids, ws), lambda ws: kv.mqkv_compact(c, s, ws),
             lambda ws: kv.mqkv_attention(c, s, 0, q, out, None, 1, 9, ws)]
    for f in calls:
        for ws in (torch.empty(1 << 20, dtype=torch.uint8), OnDevice((1 << 20, 2), (4, 1), contiguous=False)):
            with pytest.raises(B.MQError, match="workspace is not a contiguous CUDA tensor"):
                f(ws)
    # its size counts in bytes
    need = L.mqkv_pages_workspace_bytes(c, s)
    assert kv._ws(OnDevice((need // 4,), (1,))) == (WS, need)
    with pytest.raises(B.MQError, match="bytes, .* needed"):
        kv.mqkv_extend(c, s, None, OnDevice((need // 4 - 1,), (1,)))


# ------------------------------------------------------------- the model itself is pinned ---

def test_model_append_closed_forms():
    m = U.Model(3, 1, 1, 64, 32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :4] = [127, 0.5, -0.5, 2.5]
    m.append(0, 0, [2, 1], 2, x)
    assert m.scales[2, 0, 0, 0, 0] == 1 and list(m.codes[2, 0, 0, 0, 0, :4]) == [127, 1, -1, 3]
    y = np.zeros((1, 1, 64), np.float32)
    y[0, 0, 0] = 254                                        # the scale doubles: old codes halve, half away from zero
    m.append(0, 0, [2, 1], 3, y)
    assert m.scales[2, 0, 0, 0, 0] == 2 and list(m.codes[2, 0, 0, 0, 0, :4]) == [64, 1, -1, 2] and m.codes[2, 0, 0, 0, 2, 0] == 127
    z = np.full((1, 1, 64), np.nan, np.float32)
    z[0, 0, 0], z[0, 0, 1] = np.inf, -np.inf                 # what cannot be a scale: the ends of the block's range
    m.append(0, 0, [2, 1], 4, z)
    assert m.scales[2, 0, 0, 0, 0] == 2 and list(m.codes[2, 0, 0, 0, 3, :3]) == [127, -127, 0]
    full = np.ones((33, 1, 64), np.float32)
    m.append(0, 1, [2, 1], 33, full)                         # over a page's end
    assert (m.codes[2, 0, 1] == 127).all() and m.codes[1, 0, 1, 0, 0, 0] == 127 and m.scales[1, 0, 1, 0, 0] == np.float32(1) * np.float32(1 / 127)


def test_model_attention_closed_forms():
    k, v = np.zeros((5, 1, 64)), np.arange(5.0)[:, None, None] * np.ones((5, 1, 64))
    q = np.ones((2, 3, 64))
    out, _, _ = U.attention(q, k, v, 5)
    assert np.allclose(out[0], 1.5) and np.allclose(out[1], 2.0)                          # means of 0..3 and 0..4
    out, _, _ = U.attention(q, k, v, 5, window=2)
    assert np.allclose(out[0], 2.5) and np.allclose(out[1], 3.5)
    out, _, _ = U.attention(np.ones((7, 1, 64)), k, v, 5)
    assert (out[:2] == 0).all() and (out[2] == 0).all() and np.allclose(out[3], 0.5)      # two rows before the first token
    out, _, _ = U.attention(q, np.zeros((0, 1, 64)), np.zeros((0, 1, 64)), 0, causal=False)
    assert (out == 0).all()
