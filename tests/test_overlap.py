"""CPU check of the operators' overlap test (csrc/overlap.h) against the bytes
themselves, through a small library built from the header."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import w4a4_quantized_gemm_smooth_b200 as S

SOURCE = """
#include "overlap.h"
extern "C" int both(const long long* a, const long long* b) {
  auto e = [](const long long* v) {
    return svdq::extent(reinterpret_cast<const void*>(v[0]), v[1], v[2], v[3], v[4], v[5]);
  };
  return svdq::overlap(e(a), e(b)) ? 1 : 0;
}
"""


@pytest.fixture(scope="module")
def both(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("overlap")
    src, so = d / "o.cpp", d / "o.so"
    src.write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(S.__file__), "csrc")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", csrc, str(src), "-o", str(so)], check=True)
    f = ctypes.CDLL(str(so)).both
    arr = ctypes.c_longlong * 6
    return lambda a, b: bool(f(arr(*a), arr(*b)))


def bytes_of(e):
    p, run, n0, n1, s0, s1 = e
    return {p + i * s0 + j * s1 + k for i in range(n0) for j in range(n1) for k in range(run)}


def test_against_the_bytes(both):
    rng = random.Random(1)
    hits = 0
    for _ in range(20000):
        def some():
            run = rng.randint(1, 6)
            steps = [rng.choice([0, 1, 4, 6, 8, 12, 24, 36]) for _ in range(2)]
            return (1000 + rng.randint(0, 60), run, rng.randint(1, 5), rng.randint(1, 4), *steps)
        a, b = some(), some()
        if rng.random() < 0.4:
            b = b[:4] + a[4:]                       # the same steps
        want = bool(bytes_of(a) & bytes_of(b))
        hits += want
        assert both(a, b) == want and both(b, a) == want, (a, b)
    assert 2000 < hits < 18000


def test_what_the_operators_meet(both):
    q = (1 << 30, 2 * 24 * 128, 1, 4608, 0, 2 * 9216)        # a third of the rows of a fused product
    k = ((1 << 30) + 2 * 24 * 128,) + q[1:]
    assert not both(q, k) and both(q, q)
    assert both(q, ((1 << 30) + 2 * 24 * 128 - 2,) + q[1:])
    far = (8, 16, 1 << 40, 1, 1 << 40, 0)                    # past 64 bits
    assert both(far, far) and not both(far, (40, 8, 1 << 40, 1, 1 << 40, 0))
    assert both(far, (8 + (1 << 42), 1, 1, 1, 0, 0))
    assert not both((0, 16, 4, 1, 16, 0), (0, 16, 4, 1, 16, 0))      # null pointers
    assert not both((64, 16, 0, 1, 16, 0), (64, 16, 4, 1, 16, 0))    # no rows
