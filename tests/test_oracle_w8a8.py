"""Pins of the oracle's W8A8 block operators against exact rational arithmetic, closed forms and error
bounds, none of which share its code."""
from fractions import Fraction

import numpy as np
import pytest

import oracle.w8a8 as ow


def frac_code(v, s):
    """clamp(RNE(v / s)) in rational arithmetic."""
    q = Fraction(float(v)) / Fraction(float(s))
    return max(-128, min(127, round(q)))  # Fraction rounds half to even


def test_quant_matches_rational_arithmetic():
    r = np.random.default_rng(0)
    s = np.exp(r.uniform(-20, 20, 400)).astype(np.float32)
    k = r.integers(-130, 130, 400) + r.choice([0.0, 0.5, 0.4999, 0.5001], 400)
    v = (k * s).astype(np.float32)
    want = [frac_code(a, b) for a, b in zip(v, s)]
    assert ow.quant(v, s).tolist() == want
    v = np.float32([np.nan, np.inf, -np.inf, 1.0, 1.0, 1.0])
    s = np.float32([1, 1, 1, 0, np.inf, 2.0 ** -101])
    assert ow.quant(v, s).tolist() == [0, 127, -128, 0, 0, 0]


def test_row_scales_by_hand():
    v = np.float32([[0, 0, 0], [np.nan, -254, 127], [np.inf, 1, -2], [1e-38, 0, 0], [3e38, 0, 0]])
    want = np.float32([1, 2, np.float32(2) / np.float32(127), 2.0 ** -100, 2.0 ** 100])  # 2 c rounds as 2 / 127
    assert np.array_equal(ow.row_scales(v), want)


def test_rmsnorm_closed_forms():
    # constant rows: t / rms = sign, so v = +-w up to fp32 rounding, the scale is max w / 127
    w = np.float32([1.0, 0.5, 0.25, 1.0])
    x = np.float32([[3, -3, 3, 3], [-1e-3, -1e-3, 1e-3, 1e-3]])
    q, s, h = ow.rmsnorm_i8(x, w, eps=0.0)
    assert h is None
    assert q.tolist() == [[127, -64, 32, 127], [-127, -64, 32, 127]]
    assert np.allclose(s, 1 / 127, rtol=2.0 ** -22)
    # two groups of very different size normalize alike; a zero row has scale 1 and codes 0
    x = np.float32([[1000, -1000, 1, 1], [0, 0, 0, 0]])
    q, s, _ = ow.rmsnorm_i8(x, groups=2, eps=0.0 + 1e-30)
    assert q.tolist() == [[127, -127, 127, 127], [0, 0, 0, 0]] and s[1] == 1
    # the stream: h = x + residual in its type
    x, res = np.float16([[1, 2]]), np.float32([[2 ** -12, -2]])
    _, _, h = ow.rmsnorm_i8(x, residual=res, residual_dtype=np.float32)
    assert h.dtype == np.float32 and h.tolist() == [[1 + 2.0 ** -12, 0]]
    _, _, h = ow.rmsnorm_i8(x, residual=res.astype(np.float16), residual_dtype=np.float16)
    assert h.dtype == np.float16 and h.tolist() == [[1, 0]]
    # gate: silu(0) = 0, silu(large) = identity, silu(-large) = -0
    x, z = np.float32([[2, 2, 2, 4]]), np.float32([[0, 100, -1000, 100]])
    q, _, _ = ow.rmsnorm_i8(x, gate=z, eps=0.0)
    assert q.tolist() == [[0, 64, 0, 127]]


def test_rmsnorm_error_bound():
    """The value of every code is within half a step, plus the fp32 roundings of t r and w, of the real
    x / sqrt(mean x^2 + eps) * w."""
    r = np.random.default_rng(1)
    x = r.standard_normal((20, 96)).astype(np.float32)
    w = r.uniform(0.5, 2, 96).astype(np.float32)
    q, s, _ = ow.rmsnorm_i8(x, w, groups=3)
    x64 = x.astype(np.float64).reshape(20, 3, 32)
    v = (x64 / np.sqrt((x64 ** 2).mean(axis=2, keepdims=True) + np.float64(np.float32(1e-5)))).reshape(20, 96) * w
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - v) <= 0.5 * s[:, None] * (1 + 2.0 ** -20) + np.abs(v) * 2.0 ** -21)


def test_gemm_matches_rational_arithmetic():
    r = np.random.default_rng(2)
    a = r.integers(-128, 128, (3, 37)).astype(np.int8)
    w = r.integers(-128, 128, (5, 37)).astype(np.int8)
    sa, sw = np.float32([0.1, np.inf, 0.3]), np.float32([1, 2, 0, 4, 5e-3])
    y = ow.gemm_w8a8(a, sa, w, sw, np.ones(5, np.float32))
    for m in range(3):
        for n in range(5):
            acc = sum(int(p) * int(q) for p, q in zip(a[m], w[n]))
            ok = m != 1 and n != 2
            want = 1 + (acc * Fraction(float(sa[m])) * Fraction(float(sw[n])) if ok else 0)
            assert y[m, n] == pytest.approx(float(want), rel=1e-14)


def test_state_update_against_a_scalar_loop():
    r = np.random.default_rng(3)
    B, nh, P, N = 2, 2, 3, 4
    codes = r.integers(-127, 128, (B, nh, P, N)).astype(np.int8)
    sc = r.uniform(0.01, 0.1, (B, nh, P)).astype(np.float32)
    sc[0, 0, 0] = np.nan  # an invalid scale reads as 0
    xh, Bh, Ch = (r.standard_normal(s).astype(np.float32) for s in ((B, nh, P), (B, nh, N), (B, nh, N)))
    dt = r.uniform(0.01, 1, (B, nh)).astype(np.float32)
    A, D = np.float32([-1, -2]), np.float32([0.5, -1])
    y, q, s, h = ow.state_update(codes, sc, xh, Bh, Ch, dt, A, D)
    for b in range(B):
        for i in range(nh):
            for p in range(P):
                real = [(0 if np.isnan(sc[b, i, p]) else np.exp(float(dt[b, i]) * float(A[i])) * float(sc[b, i, p]) * codes[b, i, p, n])
                        + float(dt[b, i]) * float(xh[b, i, p]) * float(Bh[b, i, n]) for n in range(N)]
                # dA, its product with s, the two products of the input and the sum round once each
                assert np.allclose(h[b, i, p], real, rtol=0, atol=6 * 2.0 ** -24 * (max(map(abs, real)) + 15))
                assert y[b, i, p] == pytest.approx(float(np.dot(h[b, i, p].astype(float), Ch[b, i].astype(float))) + float(D[i]) * float(xh[b, i, p]))
                assert s[b, i, p] == np.float32(np.abs(h[b, i, p]).max()) * (np.float32(1) / np.float32(127))
                assert q[b, i, p].tolist() == [frac_code(v, s[b, i, p]) for v in h[b, i, p]]
