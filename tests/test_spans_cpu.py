"""Which tensors of a call share bytes, on the CPU: csrc/spans.cuh compiled by g++, against sets of bytes."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_mx_gb300", "csrc")
AT = 1 << 20


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("spans")
    (d / "spans.cc").write_text("""#include "spans.cuh"
using mxgb::span;
extern "C" int meet(const int64_t* a, const int64_t* b) {
  return mxgb::spans_meet(span((const void*)a[0], a[1], a[2], a[3], a[4], a[5]), span((const void*)b[0], b[1], b[2], b[3], b[4], b[5]));
}
extern "C" int apart(const int64_t* a) { return mxgb::rows_apart(a[1], a[2], a[3], a[4], a[5]); }
""")
    lib = str(d / "spans.so")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, str(d / "spans.cc"), "-o", lib])
    return ctypes.CDLL(lib)


def asked(lib, a, b):
    to = ctypes.c_int64 * 6
    one, other = lib.meet(to(*a), to(*b)), lib.meet(to(*b), to(*a))
    assert one == other
    return bool(one)


def covered(s):
    at, size, n0, step0, n1, step1 = s
    return {at + i * step0 + j * step1 + k for i in range(n0) for j in range(n1) for k in range(size)} if at else set()


def test_rows_in_two_directions(lib):
    rng, met = np.random.RandomState(0), []
    for trial in range(30000):
        s = [int(rng.choice([1, 2, 3, 4])) for _ in range(4)]
        steps = rng.randint(-24, 25, 4).tolist()
        if trial % 2:  # slices of one buffer
            steps[2:] = steps[:2]
        a = (AT, int(rng.randint(1, 9)), s[0], steps[0], s[1], steps[1])
        b = (AT + int(rng.randint(-60, 61)), int(rng.randint(1, 9)), s[2], steps[2], s[3], steps[3])
        met.append(bool(covered(a) & covered(b)))
        assert asked(lib, a, b) == met[-1], (a, b)
    assert 0.2 < np.mean(met) < 0.9  # (a word on the inputs)


def test_slices_of_a_projection(lib):
    """Queries, keys and values in one buffer [tokens][heads][size], by tokens or by heads first: only those that share
    heads meet."""
    size, heads, tokens = 8, 12, 5
    parts = [(0, 4), (4, 2), (6, 6), (3, 2), (0, 12), (11, 1)]
    for steps in ((heads * size, size), (size, tokens * size)):
        for (h0, n0), (h1, n1) in itertools.product(parts, parts):
            a, b = ((AT + h * steps[1], size, tokens, steps[0], n, steps[1]) for h, n in ((h0, n0), (h1, n1)))
            assert asked(lib, a, b) == (h0 < h1 + n1 and h1 < h0 + n0)


def test_rows_of_one_tensor(lib):
    rng, found = np.random.RandomState(1), []
    for _ in range(30000):
        s = (AT, int(rng.randint(1, 9)), int(rng.randint(0, 5)), int(rng.randint(-30, 31)), int(rng.randint(0, 5)), int(rng.randint(-30, 31)))
        found.append(len(covered(s)) == s[1] * s[2] * s[4])
        assert bool(lib.apart((ctypes.c_int64 * 6)(*s))) == found[-1], s
    assert 0.2 < np.mean(found) < 0.9


def test_none_and_empty_ones_meet_nothing(lib):
    whole = (AT, 1 << 16, 1, 0, 1, 0)
    for none in ((0, 64, 1, 0, 1, 0), (AT, 0, 1, 0, 1, 0), (AT, 64, 0, 64, 3, 64), (AT, 64, 3, 64, 0, 64)):
        assert not asked(lib, whole, none) and not asked(lib, none, none)
    assert asked(lib, whole, whole)


def test_large_ones_are_decided_at_once(lib):
    t, h, size = 1 << 20, 64, 256
    a, b = ((AT + at, size, t, (2 * h + 1) * size, h, size) for at in (0, h * size))
    assert not asked(lib, a, b)
    assert asked(lib, a, (b[0] - 1,) + b[1:]) and asked(lib, a, (b[0], b[1], b[2], b[3], h + 2, b[5]))
