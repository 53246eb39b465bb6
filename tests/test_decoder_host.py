"""Host-side tests of include/mqd.h and of the calls that it adds to the cache: what is declared is exported and bound, the turns of a
rotation, and the refusals that need no GPU."""
import ctypes
import math
import subprocess

import numpy as np
import pytest

from quantized_q8_activation_quantize_gb300 import binding as B
from quantized_q8_activation_quantize_gb300 import build as mqbuild
from quantized_q8_activation_quantize_gb300 import decoder as dec
from quantized_q8_activation_quantize_gb300 import kv
from tests.test_kv_host import BAD_CACHES, BAD_SEQS, CU, K, POOL, Q, V, WS, cache, seqs

ARG, SHAPE, ALIGN, OK = B.MQ_ERR_ARG, B.MQ_ERR_SHAPE, B.MQ_ERR_ALIGN, B.MQ_OK


@pytest.fixture(scope="session")
def L():
    mqbuild.build()
    kv.lib()
    return dec.lib()


def test_header_library_and_binding_agree(L):
    names = set(dec.header_functions())
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True).stdout
    assert {ln.split()[-1] for ln in out.splitlines() if ln.split() and ln.split()[-1].startswith("mqd_")} == names
    for name in names:
        assert callable(getattr(dec, name)), name


def caller(f, ok):
    def rc(**at):
        a = list(ok)
        for i, x in at.items():
            a[int(i[1:])] = x
        return f(*a)
    return rc


X, R, H, W, PL = 1 << 28, 2 << 28, 3 << 28, 4 << 28, 5 << 28


def test_add_quantize_refusals(L):
    rc = caller(L.mqd_add_quantize_q8, [0, X, 512, R, 512, H, 512, 4, 512, W, 1e-6, 7, PL, None])
    assert rc(_0=3) == ARG and rc(_0=-1) == ARG
    assert rc(_7=-1) == ARG and rc(_7=1 << 31) == SHAPE and rc(_7=0) == OK
    assert rc(_8=300) == SHAPE and rc(_8=0) == SHAPE and rc(_8=1 << 31) == SHAPE
    assert rc(_3=None) == ARG and rc(_5=None) == ARG and rc(_9=None) == ARG and rc(_12=None) == ARG
    assert rc(_1=X + 8) == ALIGN and rc(_3=R + 4) == ALIGN and rc(_5=H + 8) == ALIGN and rc(_9=W + 4) == ALIGN and rc(_12=PL + 128) == ALIGN
    assert rc(_2=516) == ALIGN and rc(_2=504) == ARG and rc(_4=0) == ARG and rc(_6=-512) == ARG        # strides
    assert rc(_10=float("nan")) == ARG and rc(_10=-1.0) == ARG and rc(_11=0) == ARG and rc(_11=8) == ARG
    for at in (dict(_12=X + 256), dict(_12=R), dict(_12=H + 512), dict(_12=W), dict(_5=W), dict(_5=X + 1024), dict(_5=R + 1024), dict(_5=R, _6=520)):
        assert rc(**at) == ARG and "overlap" in B.last_error(), at


def test_dequantize_refusals(L):
    rc = caller(L.mqd_dequantize_q8, [PL, 4, 512, 7, 0, H, 512, None])
    assert rc(_3=0) == ARG and rc(_3=4) == ARG and rc(_3=8) == ARG and rc(_4=3) == ARG
    assert rc(_1=-1) == ARG and rc(_1=0) == OK and rc(_2=100) == SHAPE and rc(_1=1 << 31) == SHAPE and rc(_1=(1 << 31) - 1, _2=1 << 20) == SHAPE
    assert rc(_0=None) == ARG and rc(_5=None) == ARG and rc(_0=PL + 16) == ALIGN and rc(_5=H + 4) == ALIGN and rc(_6=516) == ALIGN and rc(_6=256) == ARG
    assert rc(_5=PL + 1024) == ARG and "overlap" in B.last_error()


def frequencies(rot, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0, factors=None):
    """radians per position, pair by pair"""
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling in ("turns", "index"):
            if scaling == "turns":
                w = (original * f / (2 * math.pi) - low) / (high - low)
            else:
                def g(n):
                    return rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
                i0, i1 = max(math.floor(g(high)), 0), min(math.ceil(g(low)), rot - 1)
                w = 1 - (i - i0) / max(i1 - i0, 0.001)
            w = min(max(w, 0.0), 1.0)
            f *= w + (1 - w) / factor
        out.append(f / (factors[i] if factors else 1.0))
    return out


@pytest.mark.parametrize("kw", [{}, {"scaling": "linear", "factor": 4.0}, {"scaling": "base", "factor": 8.0},
                                {"scaling": "turns", "factor": 8.0, "original": 8192.0}, {"scaling": "turns", "factor": 2.0, "original": 100.0, "low": 0.5, "high": 30.0},
                                {"scaling": "index", "factor": 4.0, "original": 4096.0, "low": 1.0, "high": 32.0},
                                {"scaling": "index", "factor": 4.0, "original": 7.0, "low": 1.0, "high": 32.0}])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (8, 1e6), (1024, 10000.0), (96, 10000.0)])
def test_turns(L, rot, base, kw):
    got = dec.mqd_rope_turns(rot, base, **kw)
    want = frequencies(rot, base, **kw)
    # pow, log and the divisions are good to a few steps of a double; in the exponent a step counts ln(base) times
    for g, f in zip(got, want):
        assert abs(g - 2.0 ** 64 * f / (2 * math.pi)) <= 2.0 ** 64 * f * 1e-14 + 1
    factors = [1 + 0.25 * i for i in range(rot // 2)]
    for g, f in zip(dec.mqd_rope_turns(rot, base, factors=factors, **kw), frequencies(rot, base, factors=factors, **kw)):
        assert abs(g - 2.0 ** 64 * f / (2 * math.pi)) <= 2.0 ** 64 * f * 1e-14 + 1


def test_turns_refusals(L):
    out = (ctypes.c_uint64 * 512)()
    rc = caller(L.mqd_rope_turns, [128, 1e4, 0, 1.0, 0.0, 1.0, 4.0, None, out])
    assert rc() == OK and rc(_8=None) == ARG
    for rot in (0, 4, 12, 20, 1032, -8):
        assert rc(_0=rot) == SHAPE
    assert rc(_1=1.0) == ARG and rc(_1=float("nan")) == ARG and rc(_1=float("inf")) == ARG and rc(_2=5) == ARG and rc(_2=-1) == ARG
    assert rc(_3=0.5) == ARG and rc(_3=float("inf")) == ARG
    for kind in (3, 4):
        assert rc(_2=kind) == ARG and rc(_2=kind, _4=4096.0) == OK                       # original
        assert rc(_2=kind, _4=4096.0, _5=4.0) == ARG and rc(_2=kind, _4=4096.0, _5=0.0) == ARG and rc(_2=kind, _4=4096.0, _6=float("inf")) == ARG
    assert rc(_7=(ctypes.c_double * 64)(*[1.0] * 63, 0.0)) == ARG and rc(_7=(ctypes.c_double * 64)(0.1, *[1.0] * 63)) == ARG
    with pytest.raises(B.MQError):
        dec.mqd_rope_turns(128, scaling="stretch")
    with pytest.raises(B.MQError):
        dec.mqd_rope_turns(128, factors=[1.0])


def test_a_stretched_base_stays_a_number(L):
    out = (ctypes.c_uint64 * 4)()
    rc = caller(L.mqd_rope_turns, [8, 1e300, 2, 1e7, 0.0, 1.0, 4.0, None, out])
    assert rc(_3=1e10) == ARG and "range of a double" in B.last_error()                   # (all pairs but the first would stand still)
    assert rc(_3=1e5) == OK


TURNS, POS = 6 << 20, 7 << 20


def plan(**kw):
    return ctypes.byref(dec.RopePlan(**{**dict(turns=TURNS, rot_dim=64, interleaved=0, amplitude=1.0), **kw}))


BAD_PLANS = [(dict(turns=None), ARG), (dict(turns=TURNS + 4), ALIGN), (dict(rot_dim=0), SHAPE), (dict(rot_dim=12), SHAPE), (dict(rot_dim=136), SHAPE),
             (dict(amplitude=float("nan")), ARG), (dict(amplitude=float("inf")), ARG)]


def test_rope_refusals(L):
    rc = caller(L.mqd_rope, [plan(), 0, X, 1024, 128, H, 1024, 128, 7, 8, 128, POS, None])
    for kw, status in BAD_PLANS:
        assert rc(_0=plan(**kw)) == status, kw
    assert rc(_0=None) == ARG and rc(_1=3) == ARG
    assert rc(_8=-1) == ARG and rc(_8=1 << 31) == SHAPE and rc(_8=0) == OK and rc(_9=0) == OK and rc(_9=-1) == ARG and rc(_9=65537) == SHAPE
    assert rc(_10=100) == SHAPE and rc(_10=1032) == SHAPE and rc(_10=56) == SHAPE
    assert rc(_11=None) == ARG and rc(_11=POS + 2) == ALIGN
    assert rc(_2=None) == ARG and rc(_5=None) == ARG and rc(_2=X + 8) == ALIGN and rc(_1=1, _5=H + 4) == ALIGN and rc(_3=1022) == ALIGN and rc(_7=130) == ALIGN
    assert rc(_4=-128) == ARG and rc(_6=512) == ARG                                       # heads of out overlap
    assert rc(_5=X + 16) == ARG and rc(_5=X, _6=2048) == ARG and rc(_5=POS - 64) == ARG and rc(_5=TURNS) == ARG


def _has_device():
    import torch
    return torch.cuda.is_available()


def test_append_rope_refusals(L):
    QO = 8 << 24
    ok = [cache(), seqs(), 0, 0, plan(), POS, Q, 1024, 128, QO, 1024, 128, 8, K, 512, 128, V, 512, 128, CU, 7, None]
    rc = caller(kv.lib().mqkv_append_rope, ok)
    for kw, status in BAD_CACHES:
        assert rc(_0=cache(**kw)) == status, kw
    for kw, status in BAD_SEQS:
        assert rc(_1=seqs(**kw)) == status, kw
    for kw, status in BAD_PLANS:
        assert rc(_4=plan(**kw)) == status, kw
    assert rc(_4=plan(rot_dim=128), _0=cache(head_dim=64)) == SHAPE
    assert rc(_2=2) == ARG and rc(_3=4) == ARG and rc(_5=POS + 1) == ALIGN and rc(_12=-1) == SHAPE and rc(_20=0) == OK and rc(_19=None) == ARG
    assert rc(_6=None) == ARG and rc(_9=None) == ARG and rc(_13=None) == ARG and rc(_16=None) == ARG
    assert rc(_9=QO + 4) == ALIGN and rc(_10=512) == ARG and rc(_9=POOL) == ARG and rc(_6=POOL + 1024) == ARG and rc(_13=POOL) == ARG
    assert rc(_9=Q + 1024) == ARG and rc(_9=K) == ARG and "overlap" in B.last_error() and rc(_9=POS) == ARG and rc(_9=CU) == ARG and rc(_9=TURNS) == ARG
    # q turned in place in one buffer with k and v: refused where the heads meet, fine where they do not (the call then misses its device)
    one = dict(_6=Q, _7=2048, _9=Q, _10=2048, _14=2048, _17=2048)
    assert rc(**one, _13=Q + 4 * 896, _16=Q + 4 * 1536) == ARG and rc(**one, _13=Q + 4 * 1024, _16=Q + 4 * 1600) == ARG
    if not _has_device():
        assert rc(**one, _13=Q + 4 * 1024, _16=Q + 4 * 1536) in (B.MQ_ERR_CUDA, B.MQ_ERR_DEVICE)


def test_beam_refusals(L):
    need = L.mqd_beam_workspace_bytes(3, 4, 1000, 8)
    assert need > 0 and L.mqd_beam_workspace_bytes(0, 4, 1000, 8) == 256
    for bad in ((-1, 4, 1000, 8), (3, 0, 1000, 8), (3, 65, 1000, 8), (3, 4, -1, 8), (3, 4, 1 << 31, 8), (3, 4, 1000, 0), (3, 4, 1000, 65), (1 << 23, 4, 1000, 8)):
        assert L.mqd_beam_workspace_bytes(*bad) == 0, bad
    sc, c, n = 1 << 20, [(2 + i) << 20 for i in range(3)], [(6 + i) << 20 for i in range(3)]
    rc = caller(L.mqd_beam_select, [0, X, 1000, 3, 4, 1000, sc, 8, 2, *c, *n, WS, need, None])
    assert rc(_0=3) == ARG and rc(_2=999) == ARG and rc(_3=-1) == ARG and rc(_3=0) == OK and rc(_4=65) == SHAPE and rc(_5=0) == SHAPE and rc(_7=65) == SHAPE
    assert rc(_8=-2) == ARG and rc(_1=None) == ARG and rc(_6=None) == ARG and rc(_10=None) == ARG
    assert rc(_12=None) == ARG and "all given or none" in B.last_error()
    assert rc(_1=X + 2) == ALIGN and rc(_9=c[0] + 2) == ALIGN and rc(_15=WS + 16) == ALIGN and rc(_15=None) == ARG and rc(_16=need - 1) == ARG
    assert rc(_9=X) == ARG and rc(_10=c[0] + 32) == ARG and rc(_13=c[2]) == ARG and rc(_15=X - 256) == ARG and rc(_13=sc) == ARG and rc(_9=sc) == ARG
    assert "overlaps" in B.last_error()


def test_reorder_refusals(L):
    need = kv.lib().mqkv_pages_workspace_bytes(cache(), seqs())
    rc = caller(kv.lib().mqkv_reorder, [cache(), seqs(), CU, WS, need, None])
    for kw, status in BAD_CACHES:
        assert rc(_0=cache(**kw)) == status, kw
    for kw, status in BAD_SEQS:
        assert rc(_1=seqs(**kw)) == status, kw
    assert rc(_0=None) == ARG and rc(_1=None) == ARG and rc(_0=cache(refs=None)) == ARG and rc(_1=seqs(n_seqs=0)) == OK
    assert rc(_1=seqs(n_seqs=4097)) == SHAPE and rc(_2=None) == ARG and rc(_2=CU + 2) == ALIGN
    assert rc(_3=None) == ARG and rc(_3=WS + 8) == ALIGN and rc(_4=need - 1) == ARG and "workspace" in B.last_error()


def test_binding_refusals(L):
    import torch
    t = torch.zeros((4, 512))
    with pytest.raises(B.MQError, match="not a CUDA"):
        dec.mqd_add_quantize_q8(t, t, t, t[0], 1e-6, 7, t)
    with pytest.raises(B.MQError, match="not a CUDA"):
        dec.mqd_dequantize_q8(t, 7, t)
    with pytest.raises(B.MQError, match="head_dim"):
        dec.mqd_rope(dec.RopePlan(), t, t, t)
    with pytest.raises(B.MQError, match="n_groups"):
        dec.mqd_beam_select(t, t[0], (t, t, t), None, -1, t)


def test_a_plan_lies_on_the_device(L):
    with pytest.raises(B.MQError, match="not a CUDA"):
        dec.rope_plan(64, device="cpu")


def cos_sin_model(pos, F):
    """rope_cos_sin of csrc/mqd_rope.cuh in numpy float32 (fused multiply-adds through f64 products)"""
    f = np.float32

    def fma(a, b, c):
        return (a.astype(np.float64) * b.astype(np.float64) + c).astype(f)
    phase = ((pos.astype(np.int64).astype(np.uint64) * F) >> np.uint64(32)).astype(np.uint32)
    quarter = (phase + np.uint32(0x20000000)) >> np.uint32(30)
    t = (phase - (quarter << np.uint32(30))).astype(np.int32).astype(f) * f(1.5707963267948966 * 2.0 ** -30)
    z = t * t
    s = np.full_like(t, 2.75573192e-6)
    for c in (-1.98412698e-4, 8.33333333e-3, -1.66666667e-1):
        s = fma(s, z, f(c))
    s = fma(s * z, t, t)
    c = np.full_like(t, -2.75573192e-7)
    for k in (2.48015873e-5, -1.38888889e-3, 4.16666667e-2, -0.5, 1.0):
        c = fma(c, z, f(k))
    x, y = np.where(quarter & 1, s, c), np.where(quarter & 1, c, s)
    return np.where((quarter + 1) & 2, -x, x), np.where(quarter & 2, -y, y)


def test_cos_and_sin_over_every_quarter():
    r = np.random.default_rng(1)
    pos = np.concatenate([np.arange(-70, 70), r.integers(-2 ** 31, 2 ** 31, 200_000), [2 ** 31 - 1, -2 ** 31]]).astype(np.int32)
    F = r.integers(0, 2 ** 64, len(pos), dtype=np.uint64)
    F[:140] = np.uint64(2 ** 61)                              # eighths of a turn, exactly on the border between quarters
    with np.errstate(over="ignore"):
        c, s = cos_sin_model(pos, F)
        phase = pos.astype(np.int64).astype(np.uint64) * F
    angle = 2 * np.pi * (phase.astype(np.float64) / 2.0 ** 64)
    # the rest in f32 (2^-24 of at most pi / 4, twice: its conversion, the product), the phase cut to 2^-32 of a turn, the last steps of the series
    # (2^-24 each, cos near 1: half of it) and what the series leave out (3e-9)
    tol = 2 * 2.0 ** -24 * np.pi / 4 + 2 * np.pi * 2.0 ** -32 + 2.0 ** -24 + 3e-9
    assert np.abs(c - np.cos(angle)).max() < tol and np.abs(s - np.sin(angle)).max() < tol
