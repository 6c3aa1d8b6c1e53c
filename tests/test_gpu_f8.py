"""GPU parity of the block-scaled e4m3 operators: codes and scales of the quantizer bit for bit, the linear layer
within the roundings that oracle/packed.py counts."""
import numpy as np
import pytest

import oracle.packed as op

pytestmark = pytest.mark.gpu


def activations(seed, M, K, xt):
    r = np.random.default_rng([53, seed])
    x = r.standard_normal((M, K)) * np.exp(0.7 * r.standard_normal(K))
    kind = seed % 4
    if kind == 1:
        x[::2] *= 1e-6
        x[1::3] = 0
    if kind == 2:  # quotients on and beside the borders between codes
        grid = op.e4m3_values()[:127]
        mid = (grid[1:] + grid[:-1]) / 2
        x = r.choice(mid, (M, K)) * r.choice([-1, 1], (M, K)) * 2.0 ** r.integers(-8, 6, (M, 1))
        x[:, ::128] = 448 * 2.0 ** -3
    x = x.astype(xt)
    if kind == 3 and x.size > 20:
        x.flat[:: max(x.size // 11, 1)] = np.array([np.nan, np.inf, -np.inf, -0.0, np.finfo(xt).max, np.finfo(xt).tiny], xt)[
            np.arange(len(x.flat[:: max(x.size // 11, 1)])) % 6]
    return x


def wide(a, pad, shift, fill, dev):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    w = torch.full((t.shape[0], t.shape[1] + pad + shift), fill, device=dev).to(t.dtype)
    w[:, shift:shift + t.shape[1]] = t
    return w[:, shift:shift + t.shape[1]], w


def quantize(dev, x, pads=(0, 0, 0), shift=0):
    import torch
    import quantized_state_space_amd as qs
    M, K = x.shape
    xt, _ = wide(x, pads[0], shift, 1.0, dev)
    codes, cw = wide(np.zeros((M, K), np.uint8), pads[1], shift, 0x55, dev)
    scales, sw = wide(np.zeros((-(-K // 128), M), np.float32), pads[2], 0, 7.0, dev)
    qs.qssm_quant_f8(xt, codes.view(torch.float8_e4m3fn), scales)
    torch.cuda.synchronize()
    assert bool((cw[:, :shift] == 0x55).all()) and bool((cw[:, shift + K:] == 0x55).all()) and bool((sw[:, M:] == 7.0).all())
    return codes.cpu().numpy(), scales.cpu().numpy()


QUANT = [(1, 1), (1, 128), (1, 4096), (3, 129), (17, 500), (64, 1000), (100, 24), (33, 2048), (700, 1543), (257, 640), (5, 8192)]


@pytest.mark.parametrize("M,K", QUANT)
def test_quantizer(dev, M, K):
    print(f"\n[quant_f8 M={M} K={K}]", flush=True)
    i = QUANT.index((M, K))
    for j, xt in enumerate([np.float16, np.float32, np.float16, np.float32, np.float32]):
        x = activations(5 * i + j, M, K, xt)
        codes, scales = quantize(dev, x, pads=((0, 0, 0), (8, 16, 2), (3, 5, 1))[j % 3], shift=(0, 0, 1)[j % 3])
        want, ws = op.quant_f8(x)
        assert np.array_equal(scales, ws)
        assert np.array_equal(codes, want), (np.argwhere(codes != want)[:4], codes[codes != want][:4], want[codes != want][:4])


def test_quantizer_scale_range(dev):
    x = np.zeros((4, 256), np.float32)
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = 1e-38, 3e38, 2e-40, -1e25
    x[:, 200] = [1e-30, -2e30, 5, 0]
    codes, scales = quantize(dev, x)
    want, ws = op.quant_f8(x)
    assert np.array_equal(scales, ws) and np.array_equal(codes, want)


def operands(seed, M, N, K, bias=True):
    r = np.random.default_rng([54, seed])
    a, w = (r.integers(0, 256, s).astype(np.uint8) for s in ((M, K), (N, K)))
    for t in (a, w):  # no NaN, and few of the largest codes
        t[(t & 127) == 127] = 0x30
        t[(t & 0x78) > 0x60] -= 0x20
    kb, nb = -(-K // 128), -(-N // 128)
    sa = np.exp(r.uniform(-4, 0, (kb, M))).astype(np.float32)
    sw = np.exp(r.uniform(-4, 0, (nb, kb))).astype(np.float32)
    return a, sa, w, sw, r.standard_normal(N).astype(np.float32) if bias else None


def product(dev, a, sa, w, sw, b, f16=False, pads=(0, 0, 0, 0), shift=0):
    import torch
    import quantized_state_space_amd as qs
    M, N = a.shape[0], w.shape[0]
    f8 = lambda t: t.view(torch.float8_e4m3fn)  # noqa: E731
    at, _ = wide(a, pads[0], shift, 0x7F, dev)  # NaN beside the rows
    wt, _ = wide(w, pads[1], shift, 0xFF, dev)
    st, _ = wide(sa, pads[2], 0, float("nan"), dev)
    y, yw = wide(np.zeros((M, N), np.float16 if f16 else np.float32), pads[3], 0, 7.0, dev)
    dv = lambda t: None if t is None else torch.from_numpy(t).to(dev)  # noqa: E731
    y.fill_(float("nan"))
    args = qs.gemm_f8_args(f8(at), st, f8(wt), dv(sw), y, bias=dv(b))
    qs.qssm_gemm_f8(args)
    torch.cuda.synchronize()
    assert bool((yw[:, N:] == 7.0).all()), "columns behind the row were written"
    return y.double().cpu().numpy()


def check(dev, ops, f16=False, **kw):
    y = product(dev, *ops, f16=f16, **kw)
    want, e = op.gemm_f8(*ops, f16=f16)
    if f16:
        e = e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25
        want = np.where(np.abs(want) >= 65520, np.copysign(np.inf, want), want)
    big = np.isinf(want)
    assert np.array_equal(np.isinf(y), big)
    d = np.abs(np.where(big, 0, y) - np.where(big, 0, want))
    assert np.all(d <= e), (np.argwhere(~(d <= e))[:4], d.max())


PRODUCTS = [(1, 1, 1), (1, 16, 16), (1, 300, 512), (2, 257, 4096), (5, 64, 1000), (16, 128, 64), (17, 130, 192), (33, 1001, 1500),
            (64, 512, 2048), (65, 96, 80), (128, 128, 128), (129, 127, 129), (256, 640, 1024), (300, 333, 333), (513, 768, 1536),
            (1, 4096, 256), (40, 1024, 8192), (777, 1001, 500), (1024, 1024, 256), (1100, 1030, 2064), (2048, 520, 192), (4, 2000, 15)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(dev, M, N, K):
    print(f"\n[gemm_f8 M={M} N={N} K={K}]", flush=True)
    i = PRODUCTS.index((M, N, K))
    check(dev, operands(i, M, N, K, bias=i % 2 == 0), f16=i % 4 == 1)
    check(dev, operands(i + 100, M, N, K, bias=i % 2 == 1), f16=i % 4 != 1, pads=(16, 32, 3, 5))
    check(dev, operands(i + 200, M, N, K), pads=(5, 3, 0, 0), shift=i % 2)


def test_no_products(dev):
    ops = operands(7, 3, 5, 0)
    assert np.array_equal(product(dev, *ops), np.broadcast_to(ops[4].astype(np.float64), (3, 5)))


def test_scales_out_of_range_and_nan_codes(dev):
    for M, N, K in ((40, 300, 512), (2, 300, 512), (300, 300, 520)):
        a, sa, w, sw, b = operands(9, M, N, K)
        sa[1, 0], sa[2, 0], sa[0, 1] = np.nan, np.inf, 0.0
        sa[3, 1], sw[1, 2], sw[2, 1] = np.float32(2.0 ** 61), -1.0, np.float32(2.0 ** -61)
        sa[0, 0], sw[0, 0] = np.float32(2.0 ** 60), np.float32(2.0 ** -60)
        check(dev, (a, sa, w, sw, b))
        a[1, 5], w[7, 300] = 0x7F, 0xFF
        y = product(dev, a, sa, w, sw, b)
        nan = np.zeros((M, N), bool)
        nan[1], nan[:, 7] = True, True
        assert np.array_equal(np.isnan(y), nan)


def test_same_results_every_time(dev):
    ops = operands(11, 70, 700, 3000)
    y = [product(dev, *ops) for _ in range(3)]
    assert np.array_equal(y[0], y[1]) and np.array_equal(y[0], y[2])
