"""The W8A8 linear layer with scales from the whole valid range, whose product can leave fp32's: a sum of 0 then
still gives the bias, a sum that brings the value back into the range the value.

Per element the kernel rounds the sum (2^-24 relative), the product of the scales (2^-24) where it is a normal fp32
number (else it is exact in fp64), and the result (2^-24, or half the least denormal, 2^-150); an fp16 y once more (2^-11,
or 2^-25). 1 % covers the second-order products. A value of at least the largest finite number and half its last
place is an infinity; values nearer to that border than the bound may be either."""
import numpy as np
import pytest

import oracle.w8a8 as ow

pytestmark = pytest.mark.gpu

POWERS = [-100, -90, -75, -74, -64, -63, -62, -20, 0, 20, 62, 63, 64, 75, 100]


def make(seed, M, N, K):
    r = np.random.default_rng([101, seed])
    a = r.integers(-128, 128, (M, K)).astype(np.int8)
    w = r.integers(-128, 128, (N, K)).astype(np.int8)
    a[::3] = 0           # sums of 0 in every column
    a[1::7] = 0
    a[1::7, :1] = 1      # sums of one code
    m = lambda n: np.where(r.random(n) < 0.5, 1.0, r.uniform(1, 2, n))  # noqa: E731
    scale = lambda n: np.minimum(m(n) * 2.0 ** r.choice(POWERS, n), 2.0 ** 100).astype(np.float32)  # noqa: E731
    return a, scale(M), w, scale(N), r.standard_normal(N).astype(np.float32)


def check(got, want, yb, f16):
    top = 65504.0 if f16 else float(np.finfo(np.float32).max)
    border = top * (1 + (2.0 ** -12 if f16 else 2.0 ** -25))
    e = 1.01 * (2 * 2.0 ** -24 * np.abs(yb) + 2.0 ** -24 * np.abs(want) + 2.0 ** -150)
    if f16:
        e = e + 1.01 * (2.0 ** -11 * np.abs(want) + 2.0 ** -25)
    inside, outside = np.abs(want) + e < border, np.abs(want) - e > border
    assert not np.any(np.isnan(got))
    assert np.array_equal(got[outside], np.sign(want[outside]) * np.inf)
    d = np.abs(got[inside] - want[inside])
    assert np.all(d <= e[inside]), (np.argwhere(inside)[d > e[inside]][:5], d.max())
    assert np.all(np.abs(got[~inside & ~outside]) >= top * (1 - 2.0 ** -10))
    return int(outside.sum()), int(inside.sum())


# a 32 x 32 tile with K split over waves, and tiles of each size, rows at any address among them
@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (20, 260, 500), (40, 200, 64), (300, 333, 333), (600, 1100, 512),
                                   (1000, 1500, 132), (2100, 2300, 260), (130, 400, 65), (1300, 2000, 131)])
@pytest.mark.parametrize("f16", [False, True])
def test_scales_of_the_whole_range(dev, M, N, K, f16):
    print(f"\n[gemm_w8a8 scales M={M} N={N} K={K} f16={f16}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    a, sa, w, sw, b = make(M + N + K, M, N, K)
    t = [torch.from_numpy(v).to(dev) for v in (a, sa, w, sw, b)]
    for bias in (t[4], None):
        y = torch.full((M, N), float("nan"), dtype=torch.float16 if f16 else torch.float32, device=dev)
        qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(t[0], t[1], t[2], t[3], y, bias=bias))
        yb = ow.gemm_w8a8(a, sa, w, sw)
        over, _ = check(y.float().cpu().numpy().astype(np.float64), yb + (0.0 if bias is None else b.astype(np.float64)), yb, f16)
        if M > 1:
            assert over > 0
        zero = ~a.any(axis=1)
        want = np.zeros(N) if bias is None else (b.astype(np.float16) if f16 else b)
        assert np.array_equal(y.cpu().numpy()[zero], np.broadcast_to(want, (int(zero.sum()), N)).astype(y.cpu().numpy().dtype))


@pytest.mark.parametrize("M,N", [(1, 33), (70, 65), (1100, 520)])
def test_empty_sum_with_large_scales(dev, M, N):
    """K = 0 gives the bias, whatever the scales."""
    print(f"\n[gemm_w8a8 empty sum, scales of 2^100, M={M} N={N}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    b = torch.randn(N, device=dev)
    y = torch.full((M, N), float("nan"), device=dev)
    big = lambda n: torch.full((n,), 2.0 ** 100, device=dev)  # noqa: E731
    a, w = (torch.zeros(n, 0, dtype=torch.int8, device=dev) for n in (M, N))
    qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(a, big(M), w, big(N), y, bias=b))
    assert torch.equal(y, b.expand(M, N))


@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (200, 300, 256)])
def test_products_of_the_scales_below_the_normal_range(dev, M, N, K):
    """Scales of 2^-70: their product has few bits in fp32, the sums bring the value back."""
    print(f"\n[gemm_w8a8 scales of 2^-70 M={M} N={N} K={K}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    r = np.random.default_rng([102, M])
    a, w = np.full((M, K), 127, np.int8), np.full((N, K), 127, np.int8)
    sa, sw = ((r.uniform(1, 2, n) * 2.0 ** -70).astype(np.float32) for n in (M, N))
    y = torch.empty(M, N, device=dev)
    t = [torch.from_numpy(v).to(dev) for v in (a, sa, w, sw)]
    qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(*t, y))
    yb = ow.gemm_w8a8(a, sa, w, sw)
    assert yb.min() > 2.0 ** -126
    check(y.cpu().numpy().astype(np.float64), yb, yb, False)
