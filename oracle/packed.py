"""Oracle of the operators over packed sequences and in block-scaled 8-bit floating point (numpy, TEST
INFRASTRUCTURE ONLY): the causal convolution, the selective scan with a bound of the kernels' fp32
roundings beside it, the e4m3 quantizers and the linear layer. Everything is fp64 but for what a definition
rounds. Pinned by tests/test_oracle_packed.py.
"""
from __future__ import annotations

import numpy as np

from oracle.w8a8 import f32, quant

EPS = 2.0 ** -24  # half a step of fp32, relative


def silu(v):
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return v / (1.0 + np.exp(-v))


def equal_offsets(tokens, nseq):
    return np.arange(nseq + 1) * (tokens // max(nseq, 1))


def initial_states(state, nseq, shape, slots, has):
    """[nseq, *shape]: what each sequence starts from."""
    out = np.zeros((nseq, *shape))
    for i in range(nseq):
        k = i if slots is None else int(slots[i])
        if state is not None and 0 <= k < len(state) and (has is None or has[i]):
            out[i] = state[k]
    return out


def store_states(state_out, final, slots):
    """state_out with the sequences' final states in their slots."""
    out = state_out.copy()
    for i, f in enumerate(final):
        k = i if slots is None else int(slots[i])
        if 0 <= k < len(out):
            out[k] = f.astype(out.dtype)
    return out


def causal_conv(x, weight, bias, use_silu, offsets, init):
    """x [T, C]; init [nseq, W - 1, C]. Returns y and the sum v before SiLU (fp64, NaN in rows of no
    sequence), the sum of absolute values S that bounds its rounding, and the final states (x's type)."""
    x64 = np.asarray(x, np.float64)
    (T, C), W = x.shape, weight.shape[1]
    w = np.asarray(weight, np.float64)
    b = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    v, s = np.full((T, C), np.nan), np.full((T, C), np.nan)
    final = []
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(len(offsets) - 1):
            lo, hi = offsets[i], offsets[i + 1]
            rows = np.concatenate([init[i], x64[lo:hi]])
            n = hi - lo
            v[lo:hi] = b + sum(w[:, k] * rows[k:k + n] for k in range(W))
            s[lo:hi] = np.abs(b) + sum(np.abs(w[:, k] * rows[k:k + n]) for k in range(W))
            final.append(rows[n:].astype(x.dtype))
    return (silu(v) if use_silu else v), v, s, final


def conv_codes(y, scales_of_channel):
    return quant(f32(y), scales_of_channel[None, :])


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def selective_scan(x, delta, A, B, C, D, z, bias, use_softplus, groups, offsets, init, cut=0):
    """x, delta, z [T, D], B, C [T, groups * N], init [nseq, D, N]. Returns y [T, D] and the final states in fp64, and
    bounds on what the fp32 kernel may be off by in each: (y, ey, final, efinal). The recursions' errors:
      dt: (2 |v| + 12) eps relative (the sum's rounding, the exponent's, exp and rcp 2 eps each, products)
      a = e^(dt A): |dt A| (e_dt + 3 eps) + 2 eps relative (A log2 e, its product with dt, v_exp_f32)
      u B: e_dt + 2 eps relative;  h: eps of |h| (the fused multiply-add)
      y: N/4 + 4 additions of eps each of the sum of |C h|, the skip, the gate (8 + |z|) 2 eps
    cut: rows that a piece of a cut sequence may have; the sum of dt over it is off by at most cut eps / 4
    relative, and |A S| e^(-|A S|) <= 0.37, so an entering state is off by 0.1 cut eps of the largest |h| more.
    Where an exponential or a state has left fp32's range (2^127; negative steps make them grow), the bound is infinite."""
    x, delta, B, C = (np.asarray(t, np.float64) for t in (x, delta, B, C))
    A = np.asarray(A, np.float64)
    (T, d), N = x.shape, A.shape[1]
    of = np.arange(d) // (d // groups)
    v = delta if bias is None else delta + np.asarray(bias, np.float64)
    dt = softplus(v) if use_softplus else v
    e_dt = (2.0 * np.abs(v) + 12.0) * EPS
    y, ey = np.full((T, d), np.nan), np.full((T, d), np.nan)
    final, efinal = [], []
    Bt, Ct = B.reshape(T, groups, N), C.reshape(T, groups, N)
    skip = np.zeros(d) if D is None else np.asarray(D, np.float64)
    for i in range(len(offsets) - 1):
        h, e = init[i].astype(np.float64).copy(), np.zeros((d, N))
        top = np.abs(h)
        for t in range(offsets[i], offsets[i + 1]):
            m = dt[t][:, None] * A
            a = np.exp(m)
            ub = (dt[t] * x[t])[:, None] * Bt[t][of]
            er = e_dt[t][:, None]
            ah = a * h
            h = ah + ub
            e = a * e + np.abs(ah) * (np.abs(m) * (er + 3 * EPS) + 2 * EPS) + np.abs(ub) * (er + 2 * EPS) + EPS * np.abs(h)
            top = np.maximum(top, np.maximum(np.abs(h), a))
            e = np.where(top < 2.0 ** 127, e, np.inf)
            eh = e + (0.1 * cut * EPS) * top
            c = Ct[t][of]
            o = (c * h).sum(1) + skip * x[t]
            eo = (np.abs(c) * eh).sum(1) + (N / 4 + 4) * EPS * (np.abs(c * h).sum(1) + np.abs(skip * x[t])) + EPS * np.abs(o)
            if z is not None:
                zz = np.asarray(z[t], np.float64)
                g = silu(zz)
                eo = eo * np.abs(g) + np.abs(o * g) * ((8.0 + np.abs(zz)) * 2 * EPS + EPS)
                o = o * g
            y[t], ey[t] = o, 1.02 * eo + 1e-37
        final.append(h)
        efinal.append(1.02 * (e + (0.1 * cut * EPS) * top) + 1e-37)
    return y, ey, final, efinal


# ------------------------------------------------------------------------------------------------
# e4m3

def e4m3_values():
    """The value of each byte: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F and 0xFF are NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def e4m3_encode(v, s):
    """Bytes of the values nearest to v / s (fp32 operands), ties to the even byte, within +-448; NaN 0."""
    v = np.asarray(v, np.float32)
    s = np.broadcast_to(np.asarray(s, np.float32), v.shape)
    with np.errstate(invalid="ignore"):
        q = np.minimum(np.abs(v.astype(np.float64) / s.astype(np.float64)), 448.0)
    q = np.where(np.isnan(q), 0.0, q)
    grid = e4m3_values()[:127]
    up = np.searchsorted(grid, q)  # the first value at or above q
    lo = np.maximum(up - 1, 0)
    mid = (grid[lo] + grid[up]) / 2
    c = np.where(q > mid, up, np.where(q < mid, lo, np.where(lo % 2 == 0, lo, up)))
    c = np.where(grid[up] == q, up, c)
    return np.where(np.isnan(v), 0, c | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def block_scales(absmax, divide=False):
    """fl32(absmax * fl32(1/448)), or absmax / 448; 0 -> 1, within [2^-60, 2^60]."""
    a = np.asarray(absmax, np.float32)
    s = f32(a.astype(np.float64) / 448.0) if divide else f32(a.astype(np.float64) * np.float64(f32(1.0 / 448.0)))
    return np.where(a == 0, np.float32(1), np.clip(s, np.float32(2.0 ** -60), np.float32(2.0 ** 60))).astype(np.float32)


def quant_f8(x):
    """codes [M, K] and scales [ceil(K / 128), M] of x [M, K]."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((-(-K // 128), M), np.float32)
    for b in range(len(scales)):
        v = x[:, b * 128:(b + 1) * 128]
        scales[b] = block_scales(np.where(np.isfinite(v), np.abs(v), 0).max(axis=1))
        codes[:, b * 128:(b + 1) * 128] = e4m3_encode(v, scales[b][:, None])
    return codes, scales


def quant_f8_weight(w):
    w = np.asarray(w, np.float32)
    N, K = w.shape
    scales, codes = np.zeros((-(-N // 128), -(-K // 128)), np.float32), np.zeros((N, K), np.uint8)
    for i in range(scales.shape[0]):
        for b in range(scales.shape[1]):
            v = w[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128]
            scales[i, b] = block_scales(np.where(np.isfinite(v), np.abs(v), 0).max(), divide=True)
            codes[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128] = e4m3_encode(v, scales[i, b])
    return scales, codes


def gemm_f8(a, a_scales, w, w_scales, bias=None, f16=False):
    """y [M, N] in fp64, and a bound on the kernel's error: a block's 128 products are exact and summed in
    some order with at most 128 additions of 2^-23 each (truncating ones); then the scales' product, its
    fused multiply-add into the sum over the blocks and the bias, eps each. For an fp16 y the fp8 matrix
    instruction cuts each of 8 products at 2^-13 of the power of two of the largest: 8 * 2^-13 of it at most, and so
    2^-10 of the sum of their absolute values."""
    t = e4m3_values()
    (M, K), N = a.shape, w.shape[0]
    y, s = np.zeros((M, N)), np.zeros((M, N))
    ok = lambda v: np.where((v >= 2.0 ** -60) & (v <= 2.0 ** 60), v, 0).astype(np.float64)  # noqa: E731
    for b in range(-(-K // 128)):
        av, wv = t[a[:, b * 128:(b + 1) * 128]], t[w[:, b * 128:(b + 1) * 128]]
        sc = ok(a_scales[b])[:, None] * np.repeat(ok(w_scales[:, b]), 128)[None, :N]
        y += (av @ wv.T) * sc
        s += (np.abs(av) @ np.abs(wv).T) * sc
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    kb = -(-K // 128)
    return y, 1.01 * (s * ((2.0 ** -10 if f16 else 0.0) + min(K, 128) * 2.0 ** -23 + (kb + 2) * EPS) + EPS * np.abs(y)) + 1e-37
