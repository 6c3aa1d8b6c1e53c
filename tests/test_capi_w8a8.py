"""Refusals of the W8A8 block's entry points (norm, linear layer, int8 state) and the host weight
quantizer. No GPU: every call here returns before any launch."""
import ctypes

import numpy as np
import pytest

import oracle.w8a8 as ow
import quantized_state_space_amd as qs

P = ctypes.c_void_p(4096)  # a non-null address that is never read
INV, UNS = qs.QSSM_ERR_INVALID_ARG, qs.QSSM_ERR_UNSUPPORTED


def message():
    return qs.load().qssm_last_error().decode()


def norm(**kw):
    a = qs.RmsnormArgs(rows=4, dim=64, norm_groups=1, x=P, x_stride=64, eps=1e-5, compute_scales=1,
                       scales=P, q=P, q_stride=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return qs.load().qssm_rmsnorm_i8(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), INV, "rows"), (dict(dim=0), INV, "dim"), (dict(norm_groups=0), INV, "norm_groups"),
    (dict(norm_groups=3), INV, "norm_groups"), (dict(x_dtype=qs.QSSM_I8), INV, "x_dtype"),
    (dict(residual=P, residual_dtype=qs.QSSM_I16, residual_stride=64), INV, "residual_dtype"),
    (dict(residual_out=P, residual_dtype=9, residual_out_stride=64), INV, "residual_dtype"),
    (dict(gate=P, gate_dtype=5, gate_stride=64), INV, "gate_dtype"),
    (dict(gate=P, gate_stride=64, residual=P, residual_stride=64), UNS, "gate"),
    (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"), (dict(eps=float("inf")), INV, "eps"),
    (dict(x_stride=63), INV, "stride"), (dict(q_stride=0), INV, "stride"),
    (dict(residual=P, residual_stride=63), INV, "stride"), (dict(gate=P, gate_stride=1), INV, "stride"),
    (dict(residual_out=P, residual_out_stride=-64), INV, "stride"),
    (dict(x_stride=2 ** 41), UNS, "stride"), (dict(rows=2 ** 31), UNS, "rows"),
    (dict(residual=P, residual_out=P, residual_stride=64, residual_out_stride=128), INV, "one stride"),
    (dict(dim=8193, x_stride=8193, q_stride=8193), UNS, "8192"),
    (dict(dim=32776, x_stride=32776, q_stride=32776), UNS, "8192"),
    (dict(dim=16384, x_stride=16384, q_stride=16384, x=ctypes.c_void_p(4098)), UNS, "8192"),
    (dict(x=None), INV, "null"), (dict(scales=None), INV, "null"), (dict(q=None), INV, "null")])
def test_norm_refusals(kw, status, word):
    assert norm(**kw) == status
    assert word in message()


@pytest.mark.parametrize("kw", [
    dict(x=ctypes.c_void_p(4098)), dict(x=ctypes.c_void_p(4097), x_dtype=qs.QSSM_F16),
    dict(residual=ctypes.c_void_p(4098), residual_stride=64), dict(weight=ctypes.c_void_p(4097)),
    dict(residual_out=ctypes.c_void_p(4097), residual_dtype=qs.QSSM_F16, residual_out_stride=64),
    dict(gate=ctypes.c_void_p(4098), gate_stride=64), dict(scales=ctypes.c_void_p(4098))])
def test_norm_refuses_misaligned_tensors(kw):
    assert norm(**kw) == INV
    assert "aligned" in message()


def test_state_rows_refuse_misaligned_tensors():
    lib, odd, half = qs.load(), ctypes.c_void_p(4097), ctypes.c_void_p(4098)
    for h, t, s in ((half, qs.QSSM_F32, P), (odd, qs.QSSM_F16, P), (P, qs.QSSM_F16, half)):
        assert lib.qssm_state_quant(h, t, 4, 16, P, s, None) == INV and "aligned" in message()
        assert lib.qssm_state_dequant(P, s, 4, 16, h, t, None) == INV and "aligned" in message()


def test_empty_calls_launch_nothing():
    lib = qs.load()
    assert norm(rows=0, x=None, q=None, scales=None) == qs.QSSM_OK
    assert gemm(M=0, a=None, y=None) == qs.QSSM_OK
    assert gemm(N=0, w=None, y=None) == qs.QSSM_OK
    assert lib.qssm_state_quant(None, 0, 0, 16, None, None, None) == qs.QSSM_OK
    assert lib.qssm_state_dequant(None, None, 0, 16, None, 0, None) == qs.QSSM_OK
    assert update(batch=0, state=None) == qs.QSSM_OK
    for f in ("qssm_rmsnorm_i8", "qssm_gemm_w8a8"):
        assert getattr(lib, f)(None, None) == INV and "null" in message()


def gemm(**kw):
    a = qs.GemmW8A8Args(M=4, N=8, K=64, a_per_row=1, y_dtype=0, a=P, a_stride=64, a_scales=P, w=P,
                        w_stride=64, w_scales=P, y=P, y_stride=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return qs.load().qssm_gemm_w8a8(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), INV, "negative"), (dict(N=-1), INV, "negative"), (dict(K=-1), INV, "negative"),
    (dict(y_dtype=qs.QSSM_I8), INV, "y_dtype"),
    (dict(K=131072, a_stride=131072, w_stride=131072), UNS, "131071"),
    (dict(a_stride=63), INV, "stride"), (dict(w_stride=63), INV, "stride"), (dict(y_stride=7), INV, "stride"),
    (dict(a_stride=2 ** 41), UNS, "stride"), (dict(w_stride=2 ** 22 + 64), UNS, "2^22"), (dict(M=2 ** 31), UNS, "2^27"), (dict(N=2 ** 27 + 1, y_stride=2 ** 27 + 1), UNS, "2^27"),
    (dict(M=2 ** 27, N=2 ** 27, y_stride=2 ** 27), UNS, "M * N"),
    (dict(a=None), INV, "null"), (dict(w=None), INV, "null"), (dict(y=None), INV, "null"),
    (dict(a_scales=None), INV, "null"), (dict(w_scales=None), INV, "null"),
    (dict(y=ctypes.c_void_p(4098)), INV, "aligned")])
def test_gemm_refusals(kw, status, word):
    assert gemm(**kw) == status
    assert word in message()


def update(state_in=None, scales_in=None, state_scales=P, **kw):
    a = qs.UpdateArgs(batch=1, nheads=2, headdim=8, dstate=16, ngroups=1, x_groups=1, bc_group_size=4,
                      state_dtype=qs.QSSM_I8, x=P, x_group_of=P, x_scales=P, B=P, C=P, B_scales=P,
                      C_scales=P, delta=P, A=P, state=P, y=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return qs.load().qssm_state_update_i8(ctypes.byref(a), state_in, scales_in, state_scales, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(state_dtype=qs.QSSM_F16), INV, "state_dtype"), (dict(dstate=8), UNS, "dstate"),
    (dict(dstate=48), UNS, "dstate"), (dict(dstate=512), UNS, "dstate"),
    (dict(headdim=20000), UNS, "headdim"), (dict(ngroups=3), INV, "ngroups"),
    (dict(state_in=P), INV, "together"), (dict(scales_in=P), INV, "together"),
    (dict(state_scales=None), INV, "null"), (dict(state=None), INV, "null"), (dict(delta=None), INV, "null"),
    (dict(state=ctypes.c_void_p(4104)), INV, "aligned"),
    (dict(state_in=ctypes.c_void_p(4104), scales_in=P), INV, "aligned"),
    (dict(y_dtype=qs.QSSM_I8), INV, "y_groups"), (dict(y_dtype=qs.QSSM_F16), INV, "y_dtype")])
def test_state_update_i8_refusals(kw, status, word):
    assert update(**kw) == status
    assert word in message()
    lib = qs.load()
    assert lib.qssm_state_update_i8(None, None, None, None, None) == INV


def test_state_update_i8_refuses_partly_overlapping_states():
    """16 rows of 16 codes: 256 bytes of codes and 64 of scales."""
    at = ctypes.c_void_p
    for off in (-240, -16, 16, 240):
        assert update(state_in=at(4096 + off), scales_in=P) == INV and "overlap" in message()
    for off in (-60, -4, 4, 60):
        assert update(state_in=P, scales_in=at(4096 + off)) == INV and "overlap" in message()


def test_fp_update_still_refuses_an_int8_state():
    a = qs.UpdateArgs(batch=1, nheads=2, headdim=8, dstate=16, ngroups=1, x_groups=1, bc_group_size=4,
                      state_dtype=qs.QSSM_I8)
    assert qs.load().qssm_state_update(ctypes.byref(a), None) == INV and "state_dtype" in message()


def test_state_rows_refusals():
    lib = qs.load()
    assert lib.qssm_state_quant(P, qs.QSSM_I8, 4, 16, P, P, None) == INV and "QSSM_F32" in message()
    assert lib.qssm_state_quant(P, 0, -1, 16, P, P, None) == INV
    assert lib.qssm_state_quant(P, 0, 4, 0, P, P, None) == INV
    assert lib.qssm_state_quant(P, 0, 2 ** 40, 2 ** 30, P, P, None) == UNS
    assert lib.qssm_state_quant(None, 0, 4, 16, P, P, None) == INV and "null" in message()
    assert lib.qssm_state_dequant(P, P, 4, 16, P, 7, None) == INV
    assert lib.qssm_state_dequant(P, None, 4, 16, P, 0, None) == INV and "null" in message()


@pytest.mark.parametrize("N,K", [(1, 1), (7, 100), (3, 0), (0, 5)])
def test_quant_w8_matches_oracle(N, K):
    r = np.random.default_rng(N + K)
    w = (r.standard_normal((N, K)) * np.exp(r.uniform(-3, 3, (N, 1)))).astype(np.float32)
    if N > 3:
        w[0, :4] = [np.nan, np.inf, -np.inf, 0.0]
        w[1] = 0.0
        w[2] = 1e-38
    s, q = qs.qssm_quant_w8(w)
    a = np.where(np.isfinite(w), np.abs(w), 0).max(axis=1, initial=0).astype(np.float32)
    want = np.where(a == 0, np.float32(1), np.maximum(a / np.float32(127), np.float32(2.0 ** -100)))
    assert np.array_equal(s, want)
    assert np.array_equal(q, ow.quant(w, want[:, None]))


def test_binding_refuses_mismatched_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        qs.rmsnorm_args(x, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="scales"):
        qs.rmsnorm_args(x, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(3))
    with pytest.raises(ValueError, match="w "):
        qs.gemm_w8a8_args(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4),
                          torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="shape"):
        qs.qssm_state_quant(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))


def test_state_binding_refusals():
    """Shapes, types and pairs that the binding refuses before it asks for a GPU."""
    import torch
    i8, f = torch.int8, torch.float32
    with pytest.raises(TypeError, match="int8"):
        qs.qssm_state_quant(torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4))
    with pytest.raises(ValueError, match="scales"):
        qs.qssm_state_dequant(torch.zeros(4, 8, dtype=i8), torch.zeros(3), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        qs.qssm_state_quant(torch.zeros(4, 8), torch.zeros(4, 8, dtype=i8), torch.zeros(4))
    a = qs.UpdateArgs()
    a._keep, a._state = [], torch.zeros(1, 2, 3, 16, dtype=i8)
    sc = torch.zeros(1, 2, 3, dtype=f)
    with pytest.raises(ValueError, match="together"):
        qs.qssm_state_update_i8(a, sc, state_in=a._state)
    with pytest.raises(ValueError, match="shape"):
        qs.qssm_state_update_i8(a, sc, state_in=torch.zeros(1, 2, 3, 32, dtype=i8), scales_in=sc)
    with pytest.raises(ValueError, match="scales"):
        qs.qssm_state_update_i8(a, torch.zeros(1, 2, 4))
    a._state = torch.zeros(1, 2, 3, 16)
    with pytest.raises(TypeError, match="int8"):
        qs.qssm_state_update_i8(a, sc)
