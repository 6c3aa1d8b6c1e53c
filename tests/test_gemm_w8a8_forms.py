"""Every form of the W8A8 linear layer by name: on the CPU, that the library's choice takes the named form for the shapes below
(and that they cover each form's first steps, whole and partial, with few steps of K and many); on the GPU, the forms themselves
against the exact integer sums."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle.w8a8 as ow
from tests.test_gpu_gemm_w8a8 import bound, make

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["256x256", "256x128", "128x128", "128x64", "64x64", "split", "64x64 deep"]

# Rows that are multiples of 4 bytes (K and the rows' distance), fp32 y
DIRECT = [("256x256", 811, 8598, 128), ("256x256", 1040, 7263, 2048), ("256x256", 1043, 6778, 132), ("256x256", 930, 8313, 2052),
          ("256x128", 405, 8269, 128), ("256x128", 394, 9033, 2048), ("256x128", 540, 6600, 132), ("256x128", 406, 8411, 2052),
          ("128x128", 322, 8288, 1024), ("128x128", 206, 8806, 2048), ("128x128", 332, 8583, 644), ("128x128", 194, 8319, 2052),
          ("128x64", 328, 8546, 128), ("128x64", 324, 8578, 256), ("128x64", 76, 8293, 2048), ("128x64", 528, 5553, 260), ("128x64", 67, 8482, 2052),
          ("64x64", 78, 8675, 128), ("64x64", 74, 8371, 256), ("64x64", 132, 8432, 2048), ("64x64", 70, 8255, 132), ("64x64", 129, 8653, 2052),
          ("64x64 deep", 33, 70, 128), ("64x64 deep", 130, 70, 256), ("64x64 deep", 5, 8332, 2048), ("64x64 deep", 1, 8437, 644), ("64x64 deep", 3, 8207, 2052),
          ("split", 5, 70, 384), ("split", 20, 300, 2048), ("split", 33, 70, 260), ("split", 16, 257, 2052), ("split", 3, 130, 100)]
# Rows at any address
SHIFTED = [("256x256", 771, 8484, 127), ("256x256", 1080, 6713, 128), ("256x256", 3081, 2564, 2048), ("256x256", 863, 8337, 129), ("256x256", 1411, 5378, 2051),
           ("256x128", 386, 8527, 127), ("256x128", 398, 8234, 256), ("256x128", 410, 8893, 2048), ("256x128", 391, 8251, 129), ("256x128", 672, 5483, 2051),
           ("128x128", 457, 6238, 643), ("128x128", 203, 8446, 2048), ("128x128", 202, 8193, 2051),
           ("128x64", 598, 4935, 64), ("128x64", 396, 7249, 128), ("128x64", 75, 9380, 2048), ("128x64", 577, 4962, 129), ("128x64", 76, 8671, 2051),
           ("64x64", 1, 8421, 127), ("64x64", 9, 130, 15), ("64x64", 3, 8489, 128), ("64x64", 2, 8334, 2048), ("64x64", 1, 8259, 129), ("64x64", 3, 8227, 2051),
           ("split", 3, 130, 100), ("split", 40, 70, 256), ("split", 16, 257, 2048), ("split", 33, 70, 257), ("split", 20, 300, 2051)]


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("hf") / "libhf.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", os.path.join(ROOT, "tests", "host_gemm_w8a8_forms.cpp"), "-o", out])
    lib = ctypes.CDLL(out)
    lib.host_form.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2

    def name(M, N, K, f16, direct):
        r = lib.host_form(M, N, K, int(f16), int(direct))
        return NAMES[r & 15], bool(r & 16)
    return name


@pytest.mark.parametrize("want,M,N,K", DIRECT)
def test_direct_rows_take_the_named_form(form, want, M, N, K):
    assert K % 4 == 0 and form(M, N, K, False, True) == (want, False)


@pytest.mark.parametrize("want,M,N,K", SHIFTED)
def test_rows_at_any_address_take_the_named_form(form, want, M, N, K):
    assert form(M, N, K, False, False) == (want, True)


def test_shapes_cover_every_form():
    """Whole and partial first steps, few steps (at most 8 of 128 codes) and many; the shifted tiles shorter than a step too."""
    kinds = lambda rows, f: {(K % 128 != 0, K > 1024) for g, _, _, K in rows if g == f}  # noqa: E731
    every = {(False, False), (True, False), (False, True), (True, True)}
    for f in NAMES:
        assert kinds(DIRECT, f) == every, f
        if f != "64x64 deep":
            # (no shape under the limits tried takes the shifted 128x128 tile for fewer steps of a whole K)
            assert kinds(SHIFTED, f) == every - ({(False, False)} if f == "128x128" else set()), f
    assert {f for f, _, _, K in SHIFTED if K < 128} == {"256x256", "256x128", "128x64", "64x64", "split"}
    assert {M <= 16 for f, M, _, _ in DIRECT + SHIFTED if f == "split"} == {True, False}


def test_decode_batch_forms(form):
    """The projections of a decode batch, and short rows: the split form takes K from 16 on, a tile the rest."""
    assert form(256, 18560, 4096, True, True) == ("256x128", False)
    assert form(256, 4096, 8192, False, True) == ("64x64 deep", False)
    assert form(1, 100, 15, False, True) == ("64x64", True) and form(1, 100, 16, False, True) == ("split", False)
    assert form(1, 100, 0, False, True) == ("64x64", True)


def run(dev, M, N, K, pa, pw, oa, ow_, rows, f16=False):
    """y of the given rows from tensors whose rows lie pa and pw bytes further apart than K, from bytes oa and ow_ on; the
    bytes around them are 99."""
    import torch
    import quantized_state_space_amd as qs
    a, sa, w, sw, b = make(M + K, M, N, K)

    def place(t, pad, off):
        flat = torch.full((t.shape[0] * (K + pad) + off,), 99, dtype=torch.int8, device=dev)
        v = flat[off:].view(t.shape[0], K + pad)[:, :K]
        v.copy_(torch.from_numpy(t))
        return v
    y = torch.full((M, N), float("nan"), dtype=torch.float16 if f16 else torch.float32, device=dev)
    dv = lambda v: torch.from_numpy(v).to(dev)  # noqa: E731
    qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(place(a, pa, oa), dv(sa), place(w, pw, ow_), dv(sw), y, bias=dv(b)))
    torch.cuda.synchronize()
    assert not bool(torch.isnan(y).any())
    got = y[torch.from_numpy(rows).to(dev)].double().cpu().numpy()
    yb = ow.gemm_w8a8(a[rows], sa[rows], w, sw)
    want = yb + b.astype(np.float64)
    assert np.all(np.abs(got - want) <= bound(want, yb, f16))


def sampled(M, n):
    return np.unique(np.concatenate([[0, M - 1, M // 2], np.random.default_rng(M).integers(0, M, n)]))


@pytest.mark.gpu
@pytest.mark.parametrize("want,M,N,K", DIRECT)
def test_direct_forms(dev, want, M, N, K):
    print(f"\n[gemm_w8a8 {want} M={M} N={N} K={K}]", flush=True)
    run(dev, M, N, K, 0, 4, 0, 0, sampled(M, 100))


@pytest.mark.gpu
@pytest.mark.parametrize("want,M,N,K", SHIFTED)
def test_shifted_forms(dev, want, M, N, K):
    print(f"\n[gemm_w8a8 shifted {want} M={M} N={N} K={K}]", flush=True)
    run(dev, M, N, K, -K % 4 + 1, -K % 4 + 3, 1, 2, sampled(M, 100))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [255, 256])
def test_in_projection_of_a_decode_batch(dev, M):
    print(f"\n[gemm_w8a8 in-projection M={M} N=18560 K=4096]", flush=True)
    run(dev, M, 18560, 4096, 0, 0, 0, 0, sampled(M, 20), f16=True)
