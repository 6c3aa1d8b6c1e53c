"""Pins of oracle/packed.py: each function against another way to the same numbers (numpy's convolution, the
closed form of a recurrence, torch's e4m3 type), and the library's host quantizer against it."""
import numpy as np
import pytest
import torch

import oracle.packed as op
import quantized_state_space_amd as qs


def test_conv_is_numpys_convolution():
    r = np.random.default_rng(0)
    x, w, b = r.standard_normal((40, 3)), r.standard_normal((3, 4)), r.standard_normal(3)
    init = r.standard_normal((2, 3, 3))
    y, v, s, final = op.causal_conv(x, w, b, False, [0, 25, 40], init)
    for i, (lo, hi) in enumerate(((0, 25), (25, 40))):
        rows = np.concatenate([init[i], x[lo:hi]])
        for c in range(3):
            assert np.allclose(y[lo:hi, c], np.convolve(rows[:, c], w[c, ::-1], "valid") + b[c])
        assert np.array_equal(final[i], rows[-3:])
    assert np.all(s >= np.abs(v) - 1e-12)


def test_conv_of_sequences_shorter_than_the_filter():
    x, w = np.arange(1.0, 4.0)[:, None], np.ones((1, 4))
    init = np.array([[[10.0], [20.0], [30.0]]] * 3)
    y, _, _, final = op.causal_conv(x, w, None, False, [0, 1, 1, 3], init)
    assert y[:, 0].tolist() == [61.0, 62.0, 55.0]
    assert [f[:, 0].tolist() for f in final] == [[20, 30, 1], [10, 20, 30], [30, 2, 3]]


def test_silu():
    assert op.silu(0.0) == 0.0 and abs(op.silu(1.0) - 1 / (1 + np.exp(-1))) < 1e-15 and op.silu(-800.0) == 0.0


@pytest.mark.parametrize("use_softplus", [False, True])
def test_scan_is_the_closed_form(use_softplus):
    """Constant inputs: h after n rows is a^n h0 + u B (1 - a^n) / (1 - a)."""
    n, A = 30, np.array([[-0.5, -1.5]])
    one = np.ones((n, 1))
    raw = 0.3
    dt = np.log(1 + np.exp(raw)) if use_softplus else raw
    B, C = np.tile([0.7, -0.2], (n, 1)), np.tile([1.1, 0.4], (n, 1))
    h0 = np.array([[[2.0, -3.0]]])
    y, ey, final, _ = op.selective_scan(2 * one, raw * one, A, B, C, [0.25], None, None, use_softplus, 1, [0, n], h0)
    a = np.exp(dt * A)
    for t in range(n):
        h = a ** (t + 1) * h0[0] + 2 * dt * B[0] * (1 - a ** (t + 1)) / (1 - a)
        assert np.allclose(y[t], (h * C[0]).sum() + 0.5)
    assert np.allclose(final[0], h) and np.all(ey < 1e-4) and np.all(ey > 0)


def test_scan_gate_bias_groups_and_empty_sequences():
    r = np.random.default_rng(1)
    x, dl, z = (r.standard_normal((6, 4)) for _ in range(3))
    B, C, A = r.standard_normal((6, 6)), r.standard_normal((6, 6)), -np.exp(r.standard_normal((4, 3)))
    bias, init = r.standard_normal(4), r.standard_normal((3, 4, 3))
    y, _, final, _ = op.selective_scan(x, dl, A, B, C, None, z, bias, True, 2, [0, 2, 2, 6], init)
    for d in range(4):
        h = init[2, d].copy()
        for t in range(2, 6):
            dt = np.log1p(np.exp(dl[t, d] + bias[d]))
            h = np.exp(dt * A[d]) * h + dt * x[t, d] * B[t, 3 * (d // 2):3 * (d // 2) + 3]
            assert np.isclose(y[t, d], (h @ C[t, 3 * (d // 2):3 * (d // 2) + 3]) * z[t, d] / (1 + np.exp(-z[t, d])))
        assert np.allclose(final[2][d], h) and np.allclose(final[1][d], init[1, d])


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(op.e4m3_values(), t, equal_nan=True)


def test_e4m3_encode():
    g = op.e4m3_values()
    fin = g[np.isfinite(g)]
    assert np.array_equal(g[op.e4m3_encode(fin, 1.0)], fin)
    # midpoints go to the even byte, a step beside them does not
    pos = g[:127]
    mid = ((pos[1:] + pos[:-1]) / 2).astype(np.float32)
    lo = np.arange(126)
    assert np.array_equal(op.e4m3_encode(mid, 1.0), np.where(lo % 2 == 0, lo, lo + 1))
    assert np.array_equal(op.e4m3_encode(np.nextafter(mid, np.float32(0)), 1.0), lo)
    assert np.array_equal(op.e4m3_encode(np.nextafter(mid, np.float32(1e9)), 1.0), lo + 1)
    assert op.e4m3_encode(np.float32([1e9, -np.inf, np.nan, -0.0, -1e-9]), 1.0).tolist() == [126, 254, 0, 128, 128]
    r = np.random.default_rng(2).standard_normal(5000).astype(np.float32) * 50
    want = torch.from_numpy(r).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(op.e4m3_encode(r, 1.0), want)


def weights(seed, N, K):
    r = np.random.default_rng([7, seed])
    w = (r.standard_normal((N, K)) * np.exp(r.standard_normal((N, 1)))).astype(np.float32)
    if seed == 1 and w.size > 8:
        w.flat[:5] = [np.nan, np.inf, -np.inf, 0.0, -0.0]
    if seed == 2:
        w[:128, :128] = 0.0
    if seed == 3:
        w *= np.float32(1e-30)
    if seed == 4:
        w = (np.float32(448) * op.e4m3_values()[r.integers(0, 127, (N, K))]).astype(np.float32)  # codes and
        w.flat[::3] *= np.float32(1.0625)                                                        # midpoints
    return w


@pytest.mark.parametrize("seed,N,K", [(0, 1, 1), (0, 130, 300), (1, 64, 129), (2, 257, 256), (3, 5, 128), (4, 128, 384), (0, 0, 4), (0, 4, 0)])
def test_host_weight_quantizer(seed, N, K):
    w = weights(seed, N, K)
    scales, codes = qs.qssm_quant_f8_weight(w)
    want_s, want = op.quant_f8_weight(w)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want)


def test_quant_f8_and_product():
    r = np.random.default_rng(3)
    x, w = r.standard_normal((5, 300)).astype(np.float32), r.standard_normal((140, 300)).astype(np.float32)
    c, s = op.quant_f8(x)
    back = op.e4m3_values()[c] * np.repeat(s.T.astype(np.float64), 128, 1)[:, :300]
    # half a step is 2^-4 of a value, or of a 2^-5 where the steps are 2^-9
    assert np.all(np.abs(back - x) <= np.abs(x) * 2.0 ** -4 + np.repeat(s.T, 128, 1)[:, :300] * 2.0 ** -10)
    ws, wc = op.quant_f8_weight(w)
    y, e = op.gemm_f8(c, s, wc, ws)
    wb = op.e4m3_values()[wc] * np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:140], 128, 1)[:, :300]
    assert np.allclose(y, back @ wb.T) and np.all(e > 0) and np.all(e < 1e-3 * np.abs(back) @ np.abs(wb).T + 1e-30)
