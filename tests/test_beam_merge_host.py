"""What beam search's join compares and how it merges lists (csrc/mqd_beam_merge.h, compiled for the host): a list's keys are not quite in the order of its
logits, and the merge names every slot all the same."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

from quantized_q8_activation_quantize_gb300 import build

SOURCE = """
#include "mqd_beam_merge.h"
#include <vector>
extern "C" {
void logarithm(float s, float rest, float *h, float *l) { mq::pair_log(s, rest, *h, *l); }
void keys(float cum, const float *x, int n, float lh, float ll, uint64_t *out) {
    for (int i = 0; i < n; ++i) out[i] = mq::score_key(cum, x[i], lh, ll);
}
void mergeable(uint64_t *key, int n) {           // a list's keys as the join loads them
    for (int i = 1; i < n; ++i) key[i] = key[i] < key[i - 1] ? key[i] : key[i - 1];
}
// left lists of k keys; the best k and where they came from (list * k + entry).  Returns how many reads met a slot that no round had written.
int merge(const uint64_t *lists, int left, int k, uint64_t *best, int *from) {
    std::vector<uint64_t> key(lists, lists + left * k), key2(left * k);
    std::vector<int> place(left * k), place2(left * k);
    for (int i = 0; i < left * k; ++i) place[i] = i;
    int stale = 0;
    for (int s = 1, runs = left; s < left; s *= 2, runs = (runs + 1) / 2) {
        std::fill(place2.begin(), place2.end(), -1);
        std::fill(key2.begin(), key2.end(), 0);
        for (int i = 0; i < runs * k; ++i) {
            const int a = i / k, j = i % k, to = mq::merge_slot(key.data(), runs, s, k, a, j);
            if (to < -1 || to >= left * k) return -1;
            if (to >= 0) key2[to] = key[a * s * k + j], place2[to] = place[a * s * k + j];
        }
        key.swap(key2), place.swap(place2);
        for (int a = 0; a < (runs + 1) / 2; ++a)
            for (int j = 0; j < k; ++j) stale += place[a * 2 * s * k + j] < 0;
    }
    for (int j = 0; j < k; ++j) best[j] = key[j], from[j] = place[j];
    return stale;
}
}
"""
F = np.float32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("merge")
    src, so = os.path.join(d, "m.cpp"), os.path.join(d, "m.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", so], check=True)
    L = ctypes.CDLL(so)
    f, p = ctypes.c_float, ctypes.c_void_p
    L.logarithm.argtypes, L.keys.argtypes, L.mergeable.argtypes = [f, f, p, p], [f, p, ctypes.c_int, f, f, p], [p, ctypes.c_int]
    L.merge.argtypes = [p, ctypes.c_int, ctypes.c_int, p, p]
    return L


def logarithm(lib, s, rest=0.0):
    h, l = ctypes.c_float(), ctypes.c_float()
    lib.logarithm(s, rest, ctypes.byref(h), ctypes.byref(l))
    return F(h.value), F(l.value)


def keys(lib, cum, x, lh, ll):
    x, out = np.ascontiguousarray(x, F), np.zeros(len(x), np.uint64)
    lib.keys(cum, x.ctypes.data, len(x), lh, ll, out.ctypes.data)
    return out


def loaded(lib, k):
    k = k.copy()
    lib.mergeable(k.ctypes.data, len(k))
    return k


def merge(lib, lists, k):
    a = np.zeros((len(lists), k), np.uint64)
    for row, l in zip(a, lists):
        row[:min(k, len(l))] = l[:k]
    best, place = np.zeros(k, np.uint64), np.zeros(k, np.int32)
    stale = lib.merge(a.ctypes.data, len(lists), k, best.ctypes.data, place.ctypes.data)
    return stale, best, place


def falling(start, n):
    """n neighbouring f32 numbers from start down"""
    x = [F(start)]
    for _ in range(n - 1):
        x.append(np.nextafter(x[-1], F(-1)))
    return np.array(x, F)


def row_log(lib, x):
    """the logarithm of a row all of whose exponentials relative to its largest value are 1, as the join has it: largest value + ln n as a pair"""
    h, l = logarithm(lib, len(x))
    a = F(x[0] + h)
    bv = F(a - x[0])
    rest = F(F(x[0] - F(a - bv)) + F(h - bv))
    return a, F(rest + l)


def test_logarithms(lib):
    r = np.random.default_rng(0)
    for s in np.concatenate([np.exp2(r.uniform(-1, 45, 5000)), [1, 2, 0.71, 1.41, 1.43, 967, 152064, 2.0 ** 31]]):
        h, l = logarithm(lib, F(s))
        # The series from t^3 on is at most 0.0038 (|t| <= 0.3 / 1.7).  Relative to it, in units of 2^-24: z counts once and once more in t z with that product's own
        # rounding less than 1 (together 2), p with the rounding of 1/3 less than 2, the fused sum, the one with n and the last 1 each: 7 in all.  It is taken
        # at t without t's own rest (at most 7.5e-9, times 2 t^2), what follows t^11 is 2.6e-11, and the pairs keep 2^-44 of h.
        assert abs(float(h) + float(l) - math.log(float(F(s)))) <= 7 * 2.0 ** -24 * 0.0038 + 2 * 0.0312 * 7.5e-9 + 2.6e-11 + abs(float(h)) * 2.0 ** -44


def test_scores_past_f32(lib):
    big, inf = float(np.finfo(F).max), float("inf")
    low, top = keys(lib, 0.0, [-inf], 0.0, 0.0)[0], keys(lib, inf, [0.0], 1.0, 0.0)[0]
    # a beam of +inf stays there, also beside a logit and a logarithm at the two ends of f32; a score below f32 is -inf
    assert (keys(lib, inf, [big, 1.0, -1.0, -big], big, 0.0) == top).all()
    assert keys(lib, 0.0, [-big], big, 0.0)[0] == low and keys(lib, -big, [-big], 0.0, 0.0)[0] == low
    finite = keys(lib, 0.0, [big, 0.0, -big], 1.0, 0.0)
    assert low < finite[2] < finite[1] < finite[0] < top


def test_a_larger_logit_can_have_the_smaller_key(lib):
    x = np.array([4.7683716e-7, 4.7683713e-7], F)                 # falling
    k = keys(lib, -37.7, x, 10.317374, 4.1082e-7)
    assert x[0] > x[1] and k[0] < k[1]
    k = loaded(lib, k)
    assert k[0] >= k[1]


def settings():
    for n in (200, 967, 1500, 2049, 4088):
        for cum in (-1.5, -38.486, -0.25, -100.0):
            yield n, cum


def test_merging_names_every_slot_where_keys_are_out_of_order(lib):
    """Equal beams of rows of neighbouring logits near half a step of the row's logarithm: unsorted lists leave slots of a round unwritten, loaded ones none, and
    the merged keys are the k best."""
    raw_stale = inverted = 0
    for n, cum in settings():
        step = float(np.spacing(F(math.log(n))))
        for half in (0.5, 1.0):
            for up in (2, 5, 9, 30):
                start = F(half * step)
                for _ in range(up):
                    start = np.nextafter(start, F(1))
                x = falling(start, n)
                lh, ll = row_log(lib, x)
                raw = keys(lib, cum, x[:64], lh, ll)
                inverted += int((raw[1:] > raw[:-1]).any())
                for beams, k in ((3, 64), (16, 32), (5, 33), (2, 64)):
                    raw_stale += merge(lib, [raw] * beams, k)[0] > 0
                    key = loaded(lib, raw[:k])
                    stale, best, place = merge(lib, [key] * beams, k)
                    assert stale == 0
                    assert np.array_equal(best, np.sort(np.concatenate([key] * beams))[::-1][:k])
                    assert len(set(place.tolist())) == k and place.min() >= 0 and place.max() < beams * k
                    # within a list in its order
                    for b in range(beams):
                        mine = place[place // k == b]
                        assert np.array_equal(mine, b * k + np.arange(len(mine)))
    assert inverted > 0 and raw_stale > 0                          # (the mechanism: what the running minimum is for)


def test_the_row_that_left_a_slot_unwritten(lib):
    # three equal beams of score -1.5 over 967 neighbouring logits from five steps above 2.38e-7 down, 64 candidates
    start = F(2.0 ** -22)
    for _ in range(5):
        start = np.nextafter(start, F(1))
    x = falling(start, 967)
    lh, ll = row_log(lib, x)
    raw = keys(lib, -1.5, x[:64], lh, ll)
    assert merge(lib, [raw] * 3, 64)[0] > 0
    assert merge(lib, [loaded(lib, raw)] * 3, 64)[0] == 0


@pytest.mark.parametrize("seed", range(4))
def test_merging_lists_of_all_lengths(lib, seed):
    r = np.random.default_rng(seed)
    for _ in range(400):
        left, k = int(r.integers(1, 65)), int(r.integers(1, 65))
        lists = [loaded(lib, r.integers(1, [4, 1 << 40][int(r.integers(2))], int(r.integers(0, k + 1))).astype(np.uint64)) for _ in range(left)]
        stale, best, place = merge(lib, lists, k)
        # equals: the earlier list, then the earlier entry
        entries = [(-int(x), q * k + j) for q, l in enumerate(lists) for j, x in enumerate(l)]
        want = sorted(entries)[:k]
        n = len(want)
        assert stale == 0 and (best[n:] == 0).all()
        assert [(-int(b), int(p)) for b, p in zip(best[:n], place[:n])] == want
