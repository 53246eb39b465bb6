"""The join of attention's partials follows no record that leads outside its call (csrc/mq_kv_join.h, compiled for the host)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from quantized_q8_activation_quantize_gb300 import build

SOURCE = """
#include "mq_kv_join.h"
extern "C" int holds(const void *w, int first, int workers, int rows, int H, int group, long long n) {
    return mq::at_join_holds(*static_cast<const mq::AtJoin *>(w), first, workers, rows, H, group, n);
}
"""
RECORD = np.dtype([("nrow", "i4"), ("last", "i4"), ("h", "i4"), ("r0", "i4"), ("tok", "i8")])


@pytest.fixture(scope="module")
def holds(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    src, lib = os.path.join(d, "j.cpp"), os.path.join(d, "j.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    f = ctypes.CDLL(lib).holds
    f.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 5 + [ctypes.c_longlong]
    return lambda w, *a: bool(f(np.array(w, RECORD).ctypes.data, *a))


def test_records_of_this_call_hold(holds):
    # 20 workers, 16 rows a pass, 4 KV heads of 7 query heads, 30 tokens
    assert holds((16, 9, 3, 0, 0), 8, 20, 16, 4, 7, 30)
    assert holds((1, 19, 0, 13, 28), 0, 20, 16, 4, 7, 30)            # the last row of the last token
    assert not holds((0, 9, 3, 0, 0), 8, 20, 16, 4, 7, 30)           # none


@pytest.mark.parametrize("record", [(17, 9, 0, 0, 0), (-1, 9, 0, 0, 0), (1, 8, 0, 0, 0), (1, 20, 0, 0, 0), (1, 9, 4, 0, 0), (1, 9, -1, 0, 0),
                                    (1, 9, 0, -7, 3), (1, 9, 0, 0, 30), (1, 9, 0, 0, -1), (1, 9, 0, 14, 28), (2, 9, 0, 13, 28),
                                    (1, 9, 0, 2 ** 31 - 1, 0), (16, 9, 0, 2 ** 31 - 8, 0), (1, 9, 0, 0, 2 ** 63 - 1)])
def test_records_that_lead_outside_do_not(holds, record):
    assert not holds(record, 8, 20, 16, 4, 7, 30)


def test_whatever_the_workspace_holds(holds):
    r = np.random.default_rng(0)
    some = 0
    for _ in range(200000):
        w = np.array((r.choice([0, 1, 5, 16, 400]), r.integers(-3, 40), r.integers(-2, 9), r.integers(-3, 300), r.integers(-3, 60)), RECORD)
        first, workers, rows, H, group, n = int(r.integers(0, 20)), 20, 16, int(r.integers(1, 8)), int(r.integers(1, 9)), int(r.integers(1, 50))
        if holds(w, first, workers, rows, H, group, n):
            some += 1
            i = np.arange(int(w["nrow"]))
            token, head = w["tok"] + (w["r0"] + i) // group, w["h"] * group + (w["r0"] + i) % group
            assert len(i) <= rows and token.min() >= 0 and token.max() < n and head.min() >= 0 and head.max() < H * group
            assert first < w["last"] < workers
    assert some > 100                                               # (records that hold are among them)
