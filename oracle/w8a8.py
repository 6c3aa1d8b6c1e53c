"""Oracle of the W8A8 block's operators around and inside the recurrence (numpy, TEST INFRASTRUCTURE
ONLY): the RMS norm with an int8 output, the W8A8 linear layer and the int8 recurrent state.

Values that the operators' definitions round to fp32 are rounded here at the same places, each
computed in fp64 from fp32 inputs; sums and transcendental functions are fp64. Pinned by
tests/test_oracle_w8a8.py.
"""
from __future__ import annotations

import numpy as np

LO, HI = np.float32(2.0 ** -100), np.float32(2.0 ** 100)


def f32(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(v, np.float64).astype(np.float32)


def scale_ok(s):
    s = np.asarray(s, np.float32)
    return (s >= LO) & (s <= HI)


def row_scales(v):
    """fl32(absmax * fl32(1/127)) over the last axis (finite values; 0 -> 1), in the valid range."""
    v = np.asarray(v, np.float32)
    a = np.where(np.isfinite(v), np.abs(v), np.float32(0)).max(axis=-1)
    s = np.clip(f32(a.astype(np.float64) * np.float64(f32(1.0 / 127.0))), LO, HI)
    return np.where(a == 0, np.float32(1), s).astype(np.float32)


def quant(v, s):
    """clamp(RNE(v / s), -128, 127); NaN and an invalid scale give 0. The fp64 quotient of two fp32
    values is a half-integer only where the exact quotient is."""
    v = np.asarray(v, np.float32).astype(np.float64)
    s = np.broadcast_to(np.asarray(s, np.float32), v.shape)
    ok = scale_ok(s) & ~np.isnan(v)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(np.where(ok, v, 0.0) / np.where(ok, s, 1.0).astype(np.float64)), -128, 127)
    return np.where(ok, q, 0).astype(np.int8)


def silu(z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return f32(z / (1.0 + np.exp(-z)))


def rmsnorm_i8(x, weight=None, eps=1e-5, residual=None, residual_dtype=None, gate=None, groups=1,
               scale=None):
    """x, residual, gate [M, D] (float16 or float32 arrays). residual_dtype: the stream's type when
    there is one (residual None: the stream starts with x). Returns q, scales, h."""
    M, D = x.shape
    with np.errstate(over="ignore", invalid="ignore"):
        t = np.asarray(x, np.float32)
        h = None
        if residual_dtype is not None:
            if residual is not None:
                t = t + np.asarray(residual, np.float32)
            h = t.astype(residual_dtype)
            t = h.astype(np.float32)
        if gate is not None:
            t = t * silu(gate)
        ms = (t.astype(np.float64) ** 2).reshape(M, groups, D // groups).sum(axis=2) / (D // groups)
        r = f32(1.0 / np.sqrt(ms + np.float64(np.float32(eps))))
        v = t.reshape(M, groups, D // groups) * r[:, :, None]
        v = v.reshape(M, D)
        if weight is not None:
            v = v * np.asarray(weight, np.float32)
    s = row_scales(v) if scale is None else np.full(M, scale, np.float32)
    return quant(v, s[:, None]), s, h


def gemm_w8a8(a, a_scales, w, w_scales, bias=None):
    """y [M, N] in fp64 from the exact integer sums; invalid scales give 0."""
    acc = np.asarray(a, np.float64) @ np.asarray(w, np.float64).T
    sa = np.where(scale_ok(a_scales), a_scales, 0).astype(np.float64).reshape(-1, 1)
    sw = np.where(scale_ok(w_scales), w_scales, 0).astype(np.float64)
    y = acc * sa * sw
    return y if bias is None else y + np.asarray(bias, np.float64)


def fma32(a, b, c):
    """fl32(a b + c) of fp32 values, rounded once. The product is exact in fp64 where its factors' bits are at most 53; the sum
    is rounded to odd there (its last bit set where it is not exact), which no tie of the rounding to fp32 survives."""
    a, b, c = (np.asarray(v, np.float32).astype(np.float64) for v in np.broadcast_arrays(a, b, c))
    with np.errstate(over="ignore", invalid="ignore"):
        p = a * b
        s = p + c
        t = s - p
        e = (p - (s - t)) + (c - t)  # the sum's error, exactly
    bits = s.view(np.int64).copy()
    fix = np.isfinite(s) & (e != 0) & ((bits & 1) == 0)
    bits[fix] += np.where((e[fix] > 0) == (s[fix] > 0), 1, -1)
    return f32(bits.view(np.float64))


def state_update(codes, scales, xh, Bh, Ch, delta, A, D=None):
    """One decode step on the int8 state: codes [B, nh, P, N], scales [B, nh, P]; xh [B, nh, P], Bh and
    Ch [B, nh, N] dequantized fp32 values (each head's group). Returns y (fp64), codes, scales, h."""
    d = np.asarray(delta, np.float32)
    dA = f32(np.exp((d * np.asarray(A, np.float32)).astype(np.float64)))
    keep = dA[:, :, None] * np.where(scale_ok(scales), scales, np.float32(0))
    add = (d[:, :, None] * xh)[..., None] * Bh[:, :, None, :]
    h = fma32(keep[..., None], codes.astype(np.float32), add)
    y = (h.astype(np.float64) * Ch[:, :, None, :].astype(np.float64)).sum(axis=3)
    if D is not None:
        y = y + np.asarray(D, np.float64)[None, :, None] * xh
    s = row_scales(h)
    return y, quant(h, s[..., None]), s, h
