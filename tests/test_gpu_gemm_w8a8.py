"""GPU parity of the W8A8 linear layer against the oracle's exact integer sums. Per element the kernel
rounds the sum (2^-24 relative), the product of the scales (2^-24), the fused multiply-add (2^-24 of the
result) and, for an fp16 y, the result once more (2^-11, or half the least denormal 2^-25): the bound
below counts exactly those, with 1 % for their second-order products."""
import numpy as np
import pytest

import oracle.w8a8 as ow

pytestmark = pytest.mark.gpu


def make(seed, M, N, K, per_row=True, bias=True):
    r = np.random.default_rng([92, seed])
    a = r.integers(-128, 128, (M, K)).astype(np.int8)
    w = r.integers(-128, 128, (N, K)).astype(np.int8)
    sa = np.exp(r.uniform(-3, 0, M if per_row else 1)).astype(np.float32)
    sw = (np.exp(r.uniform(-3, 0, N)) / 4096).astype(np.float32)
    return a, sa, w, sw, r.standard_normal(N).astype(np.float32) if bias else None


def bound(y, yb, f16):
    """yb: the oracle's y without the bias."""
    e = 2 * 2.0 ** -24 * np.abs(yb) + 2.0 ** -24 * np.abs(y)
    if f16:
        e = e + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
    return 1.01 * e + 2.0 ** -140


def padded(t, pad, dev, fill):
    import torch
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=dev)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]], wide


def run(dev, a, sa, w, sw, b, f16=False, pads=(0, 0, 0), offset=0):
    import torch
    import quantized_state_space_amd as qs
    M, N = a.shape[0], w.shape[0]
    at, _ = padded(torch.from_numpy(a).to(dev), pads[0], dev, 99)
    wt, _ = padded(torch.from_numpy(w).to(dev), pads[1], dev, 99)
    if offset:  # rows that start at an odd address
        flat = torch.zeros(a.size + offset, dtype=torch.int8, device=dev)
        flat[offset:] = torch.from_numpy(a).to(dev).reshape(-1)
        at = flat[offset:].view(a.shape)
    y, wide = padded(torch.full((M, N), float("nan"), dtype=torch.float16 if f16 else torch.float32, device=dev),
                     pads[2], dev, 7.0)
    dv = lambda v: None if v is None else torch.from_numpy(v).to(dev)  # noqa: E731
    args = qs.gemm_w8a8_args(at, dv(sa), wt, dv(sw), y, bias=dv(b))
    qs.qssm_gemm_w8a8(args)
    torch.cuda.synchronize()
    assert bool((wide[:, N:] == 7.0).all()), "columns behind the row were written"
    return y.float().cpu().numpy().astype(np.float64)


def check(dev, a, sa, w, sw, b, f16=False, **kw):
    y = run(dev, a, sa, w, sw, b, f16, **kw)
    yb = ow.gemm_w8a8(a, sa, w, sw)
    want = yb if b is None else yb + b.astype(np.float64)
    e = np.abs(y - want)
    assert np.all(e <= bound(want, yb, f16)), (np.argwhere(~(e <= bound(want, yb, f16)))[:5], e.max())


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 300, 512), (2, 257, 4096), (5, 64, 1000), (16, 128, 64), (17, 130, 192),
          (33, 1001, 1500), (64, 512, 2048), (65, 96, 80), (128, 128, 128), (129, 127, 129), (256, 640, 1024),
          (300, 333, 333), (513, 768, 1536), (1, 18560, 256), (40, 4096, 8192), (777, 1001, 500),
          (1024, 1024, 256), (1100, 1030, 2064), (2048, 520, 192), (1300, 2000, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_against_oracle(dev, M, N, K):
    print(f"\n[gemm_w8a8 M={M} N={N} K={K}]", flush=True)
    i = SHAPES.index((M, N, K))
    check(dev, *make(i, M, N, K, per_row=i % 3 != 2, bias=i % 2 == 0), f16=i % 4 == 1)
    check(dev, *make(i, M, N, K, per_row=True, bias=i % 2 == 1), f16=i % 4 != 1)


# Shapes that reach every form of the kernel with ragged edges in M, N and K: 256 x 256, 256 x 128, 128 x 128,
# 128 x 64 and 64 x 64 tiles, K split over four waves in 32 x 32 tiles (with 16 or 32 token rows loaded),
# each with few steps of K and many, whole and partial.
EVERY_FORM = [(4100, 4100, 964), (4000, 4090, 4096), (2300, 4300, 132), (4097, 3000, 64), (260, 9000, 132), (1030, 4000, 2052),
              (130, 6000, 100), (300, 4000, 700), (250, 4090, 4100), (256, 4096, 260), (70, 1000, 132), (16, 2000, 68), (9, 500, 2044),
              (1000, 4000, 4100), (60, 1000, 4100), (2000, 8000, 2000), (4000, 4000, 384), (250, 4000, 256), (50, 500, 128),
              # rows at odd addresses, in each of their tile sizes; rows shorter than a step
              (2000, 3001, 131), (4000, 1500, 2049), (1500, 1501, 197), (130, 700, 77), (200, 300, 63), (70, 70, 1),
              (300, 200, 65), (130, 130, 62)]


@pytest.mark.parametrize("M,N,K", EVERY_FORM)
def test_every_form(dev, M, N, K):
    """Every element for short rows of y, 300 sampled token rows (first and last among them) otherwise."""
    print(f"\n[gemm_w8a8 forms M={M} N={N} K={K}]", flush=True)
    a, sa, w, sw, b = make(M + K, M, N, K)
    f16 = K % 8 == 4
    y = run(dev, a, sa, w, sw, b, f16, pads=(0, 0, 3 if M % 4 else 0))
    rows = np.unique(np.concatenate([[0, M - 1, M // 2], np.random.default_rng(M).integers(0, M, 300)]))
    yb = ow.gemm_w8a8(a[rows], sa[rows], w, sw)
    want = yb + b.astype(np.float64)
    assert np.all(np.abs(y[rows] - want) <= bound(want, yb, f16))


# The tiles of 256 x 256, 256 x 128, 128 x 128, 128 x 64 and 64 x 64 (two shapes each) with rows of every alignment,
# and the shortest rows: (pads of a and w, offsets of a and w)
ROWS_ANYWHERE = [(4100, 4100, 965), (2300, 4300, 131), (1300, 4000, 513), (2048, 2049, 255), (521, 5536, 1021), (540, 5500, 2047),
                 (1281, 2309, 129), (521, 5463, 135), (300, 4000, 703), (70, 1000, 133), (3, 130, 1023), (4000, 700, 127), (65, 300, 126), (130, 70, 3),
                 (9, 33, 2), (1, 1, 125), (130, 130, 16), (66, 65, 15),
                 # K split over four waves, with 16 or 32 token rows
                 (1, 4001, 4095), (20, 3000, 2047), (32, 1000, 130), (7, 500, 17), (16, 260, 257), (33, 50, 639)]


@pytest.mark.parametrize("M,N,K", ROWS_ANYWHERE)
def test_rows_at_any_address(dev, M, N, K):
    """Rows 1 or 3 bytes further apart than a multiple of 4, and tensors that start at any byte; the bytes
    around and between the rows are 99."""
    import torch
    import quantized_state_space_amd as qs
    a, sa, w, sw, b = make(M + 2 * K, M, N, K)
    rows = np.unique(np.concatenate([[0, M - 1, M // 2], np.random.default_rng(M).integers(0, M, 150)]))
    yb = ow.gemm_w8a8(a[rows], sa[rows], w, sw)
    want = yb + b.astype(np.float64)
    for pa, pw, oa, ob in ((-K % 4 + 1, -K % 4 + 3, 0, 1), (-K % 4 + 3, -K % 4 + 4, 2, 3), (-K % 4, -K % 4 + 1, 1, 2), (-K % 4, -K % 4, 3, 3)):
        print(f"\n[gemm_w8a8 rows anywhere M={M} N={N} K={K} pads={pa, pw} offsets={oa, ob}]", flush=True)

        def place(t, pad, off):
            flat = torch.full((t.shape[0] * (K + pad) + off,), 99, dtype=torch.int8, device=dev)
            v = flat[off:].view(t.shape[0], K + pad)[:, :K]
            v.copy_(torch.from_numpy(t))
            return v
        y = torch.full((M, N), float("nan"), device=dev)
        dv = lambda v: torch.from_numpy(v).to(dev)  # noqa: E731
        qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(place(a, pa, oa), dv(sa), place(w, pw, ob), dv(sw), y, bias=dv(b)))
        got = y[torch.from_numpy(rows).to(dev)].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - want) <= bound(want, yb, False))
        assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("M,N,K,pads,offset", [
    (1, 200, 512, (16, 32, 3), 0), (40, 200, 512, (16, 16, 1), 0), (200, 300, 320, (16, 48, 5), 0),
    (40, 200, 513, (5, 1, 1), 0), (200, 300, 512, (0, 0, 0), 1), (3, 70, 256, (0, 0, 0), 8),
    (1200, 600, 256, (16, 16, 7), 0), (1200, 600, 256, (0, 16, 0), 4), (1200, 600, 250, (6, 6, 0), 0)])
def test_strides_and_alignment(dev, M, N, K, pads, offset):
    print(f"\n[gemm_w8a8 strides M={M} N={N} K={K} pads={pads} offset={offset}]", flush=True)
    check(dev, *make(M + N + K, M, N, K), pads=pads, offset=offset, f16=M == 200)


@pytest.mark.parametrize("M,N", [(1, 33), (70, 65), (1100, 520)])
def test_empty_sum_and_extremes(dev, M, N):
    """K = 0 gives the bias (0 without one); sums at the ends of their range; invalid scales."""
    print(f"\n[gemm_w8a8 extremes M={M} N={N}]", flush=True)
    a, sa, w, sw, b = make(M, M, N, 0)
    assert np.array_equal(run(dev, a, sa, w, sw, b), np.broadcast_to(b.astype(np.float64), (M, N)))
    assert np.all(run(dev, a, sa, w, sw, None) == 0)
    K = 4096
    for x, z in ((-128, -128), (-128, 127), (127, 127)):
        check(dev, np.full((M, K), x, np.int8), sa, np.full((N, K), z, np.int8), sw, b)
    a, sa, w, sw, b = make(M + 1, M, N, 320)
    sa[0], sw[3], sw[5], sw[N - 1] = np.inf, np.nan, 0.0, 2.0 ** -101
    y = run(dev, a, sa, w, sw, b)
    assert np.array_equal(y[0], b.astype(np.float64))
    assert np.array_equal(y[:, [3, 5, N - 1]], np.broadcast_to(b[[3, 5, N - 1]].astype(np.float64), (M, 3)))
    check(dev, a, sa, w, sw, b)


def test_longest_sum(dev):
    """K = 131071: the largest sums still fit 32 bits."""
    print("\n[gemm_w8a8 K=131071]", flush=True)
    K = 131071
    a, w = np.full((2, K), -128, np.int8), np.full((3, K), -128, np.int8)
    w[1] = 127
    check(dev, a, np.float32([1, 2]), w, np.float32([1, 1, 0.5]), None)
    a, w = np.full((2, 131056), -128, np.int8), np.full((40, 131056), -128, np.int8)
    check(dev, a, np.float32([1, 2]), w, np.ones(40, np.float32), None)


def test_side_stream_and_replay(dev):
    print("\n[gemm_w8a8 side stream, graph]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    for M, N, K in ((1, 512, 1024), (96, 640, 512), (1200, 700, 512)):
        a, sa, w, sw, b = make(M, M, N, K)
        t = [torch.from_numpy(v).to(dev) for v in (a, sa, w, sw, b)]
        y = torch.empty(M, N, device=dev)
        args = qs.gemm_w8a8_args(t[0], t[1], t[2], t[3], y, bias=t[4])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        qs.qssm_gemm_w8a8(args, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qs.qssm_gemm_w8a8(args)
        for k in range(3):
            t[0].copy_(torch.from_numpy(np.roll(a, k + 1, axis=1)))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            got = y.clone()
            y.fill_(float("nan"))
            qs.qssm_gemm_w8a8(args)
            torch.cuda.synchronize()
            assert torch.equal(got, y), (M, k)
            yb = ow.gemm_w8a8(np.roll(a, k + 1, axis=1), sa, w, sw)
            assert np.all(np.abs(y.cpu().numpy() - (yb + b)) <= bound(yb + b, yb, False)), (M, k)
