"""Limits of the W8A8 block's entry points that keep their address arithmetic inside 64 bits, and the tensors that they
refuse for how they lie in memory. No GPU: every call here returns before any launch."""
import ctypes

import numpy as np
import pytest

import quantized_state_space_amd as qs
from tests.test_capi_w8a8 import INV, P, UNS, gemm, message, norm, update


@pytest.mark.parametrize("tensor", ["x", "q", "residual", "residual_out", "gate"])
def test_norm_refuses_rows_past_64_bits(tensor):
    """2^31 - 1 rows 2^40 elements apart each keep to their own limit, but end 2^73 bytes from the first."""
    for rows, stride in ((2 ** 31 - 1, 2 ** 40), (2 ** 31 - 1, 2 ** 27 + 1), (2 ** 20, 2 ** 38 + 8), (2 ** 18 + 1, 2 ** 40)):
        kw = {tensor: P, tensor + "_stride": stride}
        assert norm(rows=rows, **kw) == UNS and "2^58" in message(), (rows, stride)


def test_gemm_refuses_rows_past_64_bits():
    for M, stride in ((2 ** 27, 2 ** 40), (2 ** 27, 2 ** 31 + 1), (2 ** 18 + 1, 2 ** 40)):
        assert gemm(M=M, y_stride=stride) == UNS and "2^58" in message(), (M, stride)


def apart(n):
    """Addresses of n tensors far from each other."""
    return [(i + 1) << 32 for i in range(n)]


def norm_at(**kw):
    """A call on tensors apart from each other but for those given as (address, stride)."""
    x, q, sc, res, ro, gate, w = apart(7)
    a = dict(x=x, q=q, scales=sc, residual_dtype=qs.QSSM_F32, gate_dtype=qs.QSSM_F32)
    for name, at in dict(residual=res, residual_out=ro, gate=gate, weight=w).items():
        if name in kw and kw[name] is True:
            a[name] = at
            if name != "weight":
                a[name + "_stride"] = 64
    for k, v in kw.items():
        if v is not True:
            a[k] = v
    return norm(**a)


X, Q, SC, RES, RO, GATE, W = apart(7)


@pytest.mark.parametrize("kw,word", [
    # 4 rows of 64 fp32 values, 256 bytes apart: q's rows of 64 bytes
    (dict(q=X), "q "), (dict(q=X + 1023), "q "), (dict(q=X - 255), "q "), (dict(residual=True, q=RES + 512), "q "),
    (dict(gate=True, q=GATE + 255), "q "), (dict(weight=True, q=W + 255), "q "), (dict(q=SC - 255), "q "), (dict(q=SC + 15), "q "),
    (dict(residual_out=True, q=RO + 1023), "q "), (dict(q=X + 255, q_stride=256), "q "), (dict(compute_scales=0, q=SC + 3), "q "),
    # the stream over its own input, a row or an element off
    (dict(residual=True, residual_out=RES + 256, residual_out_stride=64), "residual_out"),
    (dict(residual=True, residual_out=RES - 256, residual_out_stride=64), "residual_out"),
    (dict(residual=True, residual_out=RES + 4, residual_out_stride=64), "residual_out"),
    (dict(residual=True, residual_out=RES - 4, residual_out_stride=64), "residual_out"),
    (dict(residual=True, residual_out=RES + 1020, residual_out_stride=64), "residual_out"),
    (dict(residual_out=X + 256, residual_out_stride=64), "residual_out"),
    (dict(residual_out=X, residual_out_stride=128), "residual_out"),
    (dict(residual_out=X, residual_out_stride=64, residual_dtype=qs.QSSM_F16), "residual_out"),
    (dict(residual_out=X, residual_out_stride=128, residual_dtype=qs.QSSM_F16), "residual_out"),
    (dict(weight=True, residual_out=W + 252, residual_out_stride=64), "residual_out"),
    (dict(residual_out=SC - 1020, residual_out_stride=64), "residual_out"),
    # columns of a tensor of 128 that meet by one element
    (dict(x_stride=128, residual_out=X + 252, residual_out_stride=128), "residual_out"),
    (dict(x_stride=128, residual_out=X - 252, residual_out_stride=128), "residual_out"),
    # scales that are written
    (dict(scales=X + 1020), "scales"), (dict(scales=X - 12), "scales"), (dict(residual=True, scales=RES + 4), "scales"),
    (dict(gate=True, scales=GATE), "scales"), (dict(weight=True, scales=W + 252), "scales")])
def test_norm_refuses_overlapping_tensors(kw, word):
    assert norm_at(**kw) == INV and "overlap" in message() and message().startswith(word.strip()), message()


def gemm_at(**kw):
    """M = 4, N = 8, K = 64 with y fp32 (rows of 32 bytes), every tensor apart but for those given."""
    return gemm(**dict(dict(a=X, w=W, y=RO, a_scales=SC, w_scales=RES, bias=GATE), **kw))


@pytest.mark.parametrize("kw", [
    dict(y=X), dict(y=X + 252), dict(y=X - 124), dict(y=W + 508), dict(y=W - 124), dict(y=SC + 12), dict(y=SC - 124),
    dict(a_per_row=0, y=SC), dict(y=RES + 28), dict(y=RES - 124), dict(y=GATE + 28), dict(y=GATE - 124),
    dict(y=X + 60, a_stride=128, y_stride=32),                 # columns of one tensor that meet by 4 bytes
    dict(y=X + 64, a_stride=128, y_stride=16),                 # rows of y in the gap, but twice as many
    dict(y=X + 62, y_dtype=qs.QSSM_F16, a_stride=80, y_stride=40)])
def test_gemm_refuses_an_overlapping_y(kw):
    assert gemm_at(**kw) == INV and "overlap" in message(), message()


@pytest.mark.parametrize("kw", [dict(a_scales=SC + 2), dict(a_scales=SC + 1, a_per_row=0), dict(w_scales=RES + 2), dict(bias=GATE + 3)])
def test_gemm_refuses_misaligned_scales(kw):
    assert gemm_at(**kw) == INV and "aligned" in message(), message()


@pytest.mark.parametrize("dtype,size", [(qs.QSSM_F32, 4), (qs.QSSM_F16, 2)])
def test_state_rows_refuse_overlapping_tensors(dtype, size):
    """10 rows of 16 values, their codes (160 bytes) and scales (40 bytes)."""
    at, lib = ctypes.c_void_p, qs.load()
    for v, c, s in ((X, X, SC), (X, X + 160 * size - 1, SC), (X, X - 159, SC), (X, Q, X + 160 * size - 4), (X, Q, X - 36),
                    (X, Q, Q + 156), (X, Q, Q - 36)):
        assert lib.qssm_state_quant(at(v), dtype, 10, 16, at(c), at(s), None) == INV and "overlap" in message()
        assert lib.qssm_state_dequant(at(c), at(s), 10, 16, at(v), dtype, None) == INV and "overlap" in message()


def test_state_update_refuses_codes_over_scales():
    """16 rows of 16 codes (256 bytes) and their scales (64 bytes), in or out."""
    at = ctypes.c_void_p
    for off in (-60, 0, 252):
        assert update(state=at(X), state_scales=at(X + off)) == INV and "overlap" in message()
        assert update(state=at(X), state_scales=at(SC), state_in=at(Q), scales_in=at(X + off)) == INV and "overlap" in message()
    for off in (-240, 0, 48):
        assert update(state=at(X), state_scales=at(SC), state_in=at(SC + off), scales_in=at(Q)) == INV and "overlap" in message()
