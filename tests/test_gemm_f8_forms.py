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


# For an fp16 y: the tile forms, up to 16 tokens, and rows at any address
F16 = [(n, M, N, K, (0, 0, 0, 0)) for n, M, N, K, f16 in SHAPES if f16] + [
    ("few", 1, 700, 4096, (0, 0, 0, 0)), ("few", 16, 400, 8192 + 100, (0, 0, 0, 0)), ("any", 40, 300, 1500, (1, 3, 0, 0)), ("any", 130, 200, 4099, (0, 0, 0, 0))]


@pytest.mark.gpu
@pytest.mark.parametrize("name,M,N,K,pads", F16)
def test_fp16_sums_without_a_cut(dev, name, M, N, K, pads):
    """The codes of a row have one exponent in each block of 128, so all products of a block lie within two powers of two and
    have their last bits far above 2^-13 of the largest: the matrix cores cut nothing, and an fp16 y keeps the bound of an fp32
    one and its own rounding. A product more or less is seen: y is about sqrt(K) of them, its half step 2^-11 of that."""
    import oracle.packed as op
    from tests.test_gpu_f8 import product
    print(f"\n[gemm_f8 fp16 {name} M={M} N={N} K={K}]", flush=True)
    r = np.random.default_rng([57, M, N, K])
    kb, nb = -(-K // 128), -(-N // 128)

    def codes(rows):
        e = np.repeat(r.integers(5, 10, (rows, kb)), 128, axis=1)[:, :K]
        return (r.integers(0, 2, (rows, K)) << 7 | e << 3 | r.integers(0, 8, (rows, K))).astype(np.uint8)
    a, w = codes(M), codes(N)
    sa, sw = r.uniform(0.5, 1, (kb, M)).astype(np.float32), r.uniform(0.5, 1, (nb, kb)).astype(np.float32)
    bias = r.standard_normal(N).astype(np.float32)
    y = product(dev, a, sa, w, sw, bias, f16=True, pads=pads)
    want, e = op.gemm_f8(a, sa, w, sw, bias)
    e = e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25
    d = np.abs(y - want)
    assert np.abs(want).max() < 60000 and np.all(d <= e), (np.argwhere(~(d <= e))[:4], (d / e).max())


@pytest.mark.gpu
@pytest.mark.parametrize("normal", [True, False])
@pytest.mark.parametrize("name,M,N,K,pads", F16)
def test_fp16_sums_over_the_output(dev, name, M, N, K, pads, normal):
    """The cut is at most 6e-5 of the output, as root mean squares over it, for normal values and for codes of every exponent; an fp16 y's own
    rounding is uniform in a half step of at most 2^-11 of a value, so 2^-11 / sqrt(3) of it; the two are independent."""
    import oracle.packed as op
    from tests.test_gpu_f8 import operands, product
    print(f"\n[gemm_f8 fp16 rms {name} M={M} N={N} K={K} normal={normal}]", flush=True)
    a, sa, w, sw, bias = operands(400 + M + N, M, N, K, bias=False)
    sa, sw = sa / 64, sw / 64  # (no infinities)
    if normal:
        r = np.random.default_rng([58, M, N, K])
        a, w = (op.e4m3_encode((40 * r.standard_normal(s)).astype(np.float32), np.float32(1)) for s in (a.shape, w.shape))
    y = product(dev, a, sa, w, sw, bias, f16=True, pads=pads)
    want, _ = op.gemm_f8(a, sa, w, sw, bias)
    rms = lambda v: np.sqrt(np.mean(np.square(v)))  # noqa: E731
    assert np.abs(want).max() < 60000
    assert rms(y - want) <= np.hypot(6e-5, 2.0 ** -11 / np.sqrt(3)) * rms(want) + 2.0 ** -25, (rms(y - want) / rms(want),)
