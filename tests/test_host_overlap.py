"""The library's test for tensors that share memory (quantized_state_space_amd/csrc/common.hpp), built for the host, against sets
of bytes: never blind to a shared one, exact for equal strides and single rows, and for other strides wherever the
rows lie apart modulo the strides' greatest common divisor. CPU only."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("ho") / "libho.so")
    subprocess.check_call([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "host_overlap.cpp"), "-o", out])
    lib = ctypes.CDLL(out)

    def call(cases):
        c = np.ascontiguousarray(cases, np.int64).reshape(-1, 8)
        r = np.zeros(len(c), np.uint8)
        lib.host_overlap(ctypes.c_void_p(c.ctypes.data), ctypes.c_int64(len(c)), ctypes.c_void_p(r.ctypes.data))
        return r.astype(bool)
    return call


def bytes_of(p, rows, stride, width):
    return {p + i * stride + k for i in range(rows) for k in range(width)}


def test_against_sets_of_bytes(overlap):
    r = np.random.default_rng(7)
    cases = []
    for _ in range(20000):
        wa, wb = r.integers(1, 10, 2)
        sa = wa + r.integers(0, 13)
        sb = sa if r.random() < 0.5 else wb + r.integers(0, 13)
        cases.append((5000, r.integers(1, 7), sa, wa, 5000 + r.integers(-120, 121), r.integers(1, 7), sb, min(wb, sb)))
    got, back = overlap(cases), overlap([c[4:] + c[:4] for c in cases])
    shared = 0
    for c, o, ob in zip(cases, got, back):
        c = [int(v) for v in c]
        true = not bytes_of(*c[:4]).isdisjoint(bytes_of(*c[4:]))
        shared += true
        g = math.gcd(c[2], c[6])
        m = (c[4] - c[0]) % g
        if c[2] == c[6] or c[1] == 1 or c[5] == 1 or true or (c[3] <= m and m + c[7] <= g):
            assert o == true and ob == true, c
    assert 4000 < shared < 16000


def test_null_empty_and_far(overlap):
    far = 1 << 60
    assert overlap([(0, 4, 8, 8, 0, 4, 8, 8), (4096, 0, 8, 8, 4096, 4, 8, 8), (4096, 4, 8, 0, 4096, 4, 8, 8),
                    (4096, 4, 8, 8, 4128, 4, 8, 8), (4128, 4, 8, 8, 4096, 4, 8, 8), (4096, 4, 8, 8, 4127, 4, 8, 8),
                    (4096, 2, far, 64, 4096 + far - 1, 1, 8, 8), (4096, 2, far, 64, 4096 + far // 2, 1, 8, 8),
                    (4096, 2 ** 31 - 1, 2 ** 29, 64, 4096 + 2 ** 29 + 64, 2 ** 31 - 1, 2 ** 29, 64)]).tolist() == [
        False, False, False, False, False, True, True, False, False]
