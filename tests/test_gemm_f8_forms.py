"""Every form of the block-scaled e4m3 linear layer by name: on the CPU, that the library's choice takes the named tile form for
the shapes below; on the GPU, the forms against the oracle, with whole and partial last blocks, few blocks and many, and
rows of wider tensors; and the forms that other rules choose (few tokens, rows at any address)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["256x256", "256x128", "128x128", "64x64", "64x64 K2", "64x64 K4", "32x32 K4", "32x32 K4 deep"]
# name, M, N, K, fp16 y
SHAPES = [("256x256", 1284, 8962, 132, 1), ("256x256", 2568, 7698, 128, 1), ("256x256", 1036, 8679, 644, 1),
          ("256x128", 651, 8897, 132, 0), ("256x128", 771, 7579, 128, 1), ("256x128", 389, 8280, 644, 0), ("256x128", 388, 8361, 640, 1),
          ("128x128", 386, 7239, 132, 1), ("128x128", 390, 7032, 128, 0), ("128x128", 324, 8382, 644, 1), ("128x128", 385, 7117, 640, 0),
          ("64x64", 65, 8324, 132, 0), ("64x64", 67, 8211, 128, 1), ("64x64", 65, 8529, 644, 1), ("64x64", 68, 8339, 640, 0),
          ("64x64 K2", 19, 37, 132, 0), ("64x64 K2", 18, 31, 128, 1), ("64x64 K2", 33, 8217, 644, 1), ("64x64 K2", 34, 4304, 640, 0),
          ("32x32 K4", 34, 4324, 644, 0), ("32x32 K4", 34, 4169, 1024, 1), ("32x32 K4 deep", 19, 31, 644, 1), ("32x32 K4 deep", 19, 30, 640, 0),
          ("64x64 K4", 97, 4126, 6144, 0), ("64x64 K4", 97, 4223, 8196, 1)]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("forms") / "forms.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-std=c++17", os.path.join(ROOT, "tests", "host_gemm_f8_forms.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).host_form
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
    return f


@pytest.mark.parametrize("name,M,N,K,f16", SHAPES)
def test_choice(choose, name, M, N, K, f16):
    assert NAMES[choose(M, N, K, f16)] == name


def test_choice_covers_all_forms_and_never_the_wide_one_for_fp32(choose):
    assert {(s[0], s[4]) for s in SHAPES} >= {(n, y) for n in NAMES[1:] for y in (0, 1)} | {("256x256", 1)}
    r = np.random.default_rng(0)
    for _ in range(3000):
        M, N, K = (int(np.exp(r.uniform(np.log(a), np.log(b)))) for a, b in ((17, 1 << 20), (1, 1 << 20), (128, 1 << 20)))
        assert NAMES[choose(M, N, K, 0)] != "256x256"


@pytest.mark.gpu
@pytest.mark.parametrize("name,M,N,K,f16", SHAPES)
def test_form(dev, name, M, N, K, f16):
    from tests.test_gpu_f8 import check, operands
    print(f"\n[gemm_f8 {name} M={M} N={N} K={K}]", flush=True)
    i = SHAPES.index((name, M, N, K, f16))
    check(dev, operands(300 + i, M, N, K, bias=i % 2 == 0), f16=bool(f16), pads=((0, 0, 0, 0), (4, 8, 5, 3))[i % 2])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,pads,shift", [
    # up to 16 tokens: fewer blocks than waves, whole rounds, a rest, a partial last block, rows at any address
    (1, 17, 1, (0, 0, 0, 0), 0), (3, 16, 15, (1, 2, 0, 0), 1), (2, 33, 127, (0, 0, 0, 0), 0), (16, 100, 128, (0, 0, 0, 0), 0), (7, 130, 1024, (3, 1, 2, 5), 1),
    (15, 40, 8 * 128 * 4, (0, 0, 0, 0), 0), (16, 257, 8 * 128 * 4 + 128 * 3 + 5, (0, 5, 0, 0), 0), (5, 8, 8 * 128 * 9 + 64, (16, 16, 0, 0), 0),
    # rows at any address, and K of less than a block, above 16 tokens
    (17, 65, 100, (0, 0, 0, 0), 0), (64, 64, 129, (0, 0, 0, 0), 0), (130, 100, 15, (3, 0, 0, 1), 0), (70, 129, 640, (1, 2, 3, 4), 1), (200, 190, 1001, (0, 0, 0, 0), 0)])
def test_other_forms(dev, M, N, K, pads, shift):
    from tests.test_gpu_f8 import check, operands
    print(f"\n[gemm_f8 M={M} N={N} K={K} {pads}]", flush=True)
    for f16 in (False, True):
        check(dev, operands(M + N + K, M, N, K), f16=f16, pads=pads, shift=shift)
