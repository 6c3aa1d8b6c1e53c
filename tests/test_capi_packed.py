"""What the entry points for packed sequences and block-scaled e4m3 refuse, on the CPU: every call here returns
before any launch. Addresses are made up and far from each other, but where a test lays tensors over each other."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_state_space_amd as qs

INV, UNS, WS = qs.QSSM_ERR_INVALID_ARG, qs.QSSM_ERR_UNSUPPORTED, qs.QSSM_ERR_WORKSPACE
X, Y, W, B, ST, SO, SL, HAS, G, SC, OFF, Z, A, DEL, BB, CC, WSP = [(i + 1) << 32 for i in range(17)]


def message():
    return qs.load().qssm_last_error().decode()


def conv(**kw):
    """10 rows of 64 channels in 2 sequences, fp16 to fp16."""
    a = qs.ConvArgs()
    f = dict(tokens=10, dim=64, nseq=2, width=4, silu=1, x_dtype=qs.QSSM_F16, y_dtype=qs.QSSM_F16, x=X, x_stride=64,
             weight=W, bias=B, y=Y, y_stride=64, state=ST, state_out=ST, slots=4, state_slots=SL, has_state=HAS)
    for k, v in {**f, **kw}.items():
        setattr(a, k, v)
    return qs.load().qssm_causal_conv(ctypes.byref(a), None)


def scan_args(**kw):
    """10 rows of 64 channels with 16 states in 2 sequences, fp16 to fp32."""
    a = qs.SscanArgs()
    f = dict(tokens=10, dim=64, dstate=16, nseq=2, ngroups=1, io_dtype=qs.QSSM_F16, y_dtype=qs.QSSM_F32,
             state_dtype=qs.QSSM_F32, delta_softplus=1, x=X, x_stride=64, delta=DEL, delta_stride=64, B=BB, B_stride=16,
             C=CC, C_stride=16, z=Z, z_stride=64, A=A, Dskip=B, delta_bias=W, y=Y, y_stride=64, state=ST, state_out=ST,
             slots=4, state_slots=SL, has_state=HAS)
    for k, v in {**f, **kw}.items():
        setattr(a, k, v)
    return a


def scan(ws=None, ws_bytes=0, **kw):
    return qs.load().qssm_selective_scan(ctypes.byref(scan_args(**kw)), ws, ws_bytes, None)


def quant(x=X, xt=qs.QSSM_F16, rows=4, K=256, xs=256, codes=Y, cs=256, scales=SC, ss=4):
    return qs.load().qssm_quant_f8(x, xt, rows, K, xs, codes, cs, scales, ss, None)


def gemm(**kw):
    """4 tokens, 256 channels of 384."""
    a = qs.GemmF8Args()
    f = dict(M=4, N=256, K=384, y_dtype=qs.QSSM_F32, a=X, a_stride=384, a_scales=SC, a_scales_stride=4, w=W, w_stride=384,
             w_scales=SL, bias=B, y=Y, y_stride=256)
    for k, v in {**f, **kw}.items():
        setattr(a, k, v)
    return qs.load().qssm_gemm_f8(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(tokens=-1), INV, "negative"), (dict(dim=-1), INV, "negative"), (dict(nseq=-1), INV, "negative"), (dict(slots=-1), INV, "negative"),
    (dict(tokens=11), INV, "multiple"), (dict(nseq=0), INV, "multiple"), (dict(tokens=2 ** 31), UNS, "2^31"),
    (dict(dim=2 ** 24 + 1), UNS, "2^24"), (dict(nseq=2 ** 24 + 1, tokens=0), UNS, "2^24"), (dict(width=1), UNS, "width"),
    (dict(width=5), UNS, "width"), (dict(x_dtype=qs.QSSM_I8), INV, "x_dtype"), (dict(y_dtype=qs.QSSM_I16), INV, "y_dtype"),
    (dict(reserved=1), INV, "reserved"), (dict(x_stride=63), INV, "x_stride"), (dict(y_stride=63), INV, "y_stride"),
    (dict(x_stride=2 ** 40 + 1), UNS, "2^40"), (dict(tokens=2 ** 30, nseq=1, y_stride=2 ** 30), UNS, "2^58"),
    (dict(x=None), INV, "null"), (dict(y=None), INV, "null"), (dict(weight=None), INV, "null"),
    (dict(x=X + 1), INV, "x is not aligned"), (dict(y=Y + 1), INV, "y is not aligned"), (dict(weight=W + 2), INV, "aligned"),
    (dict(bias=B + 2), INV, "aligned"), (dict(state=ST + 1), INV, "aligned"), (dict(state_slots=SL + 2), INV, "aligned"),
    (dict(seq_offsets=OFF + 2), INV, "aligned"), (dict(state_slots=None, slots=1), INV, "slots"), (dict(slots=2 ** 41), UNS, "slots"),
    (dict(slots=2 ** 40, dim=2 ** 20, x_stride=2 ** 20, y_stride=2 ** 20), UNS, "slots"),
    (dict(y_dtype=qs.QSSM_I8, y_groups=0), INV, "y_groups"), (dict(y_dtype=qs.QSSM_I8, y_groups=257), INV, "y_groups"),
    (dict(y_dtype=qs.QSSM_I8, y_groups=2, y_scales=SC), INV, "null"), (dict(y_dtype=qs.QSSM_I8, y_groups=2, y_group_of=G), INV, "null"),
    (dict(y_dtype=qs.QSSM_I8, y_groups=2, y_group_of=G, y_scales=SC + 1), INV, "aligned"),
    (dict(y=X), INV, "overlap"), (dict(y=X + 1278), INV, "overlap"), (dict(y=W), INV, "overlap"), (dict(y=B + 254), INV, "overlap"),
    (dict(y=ST), INV, "overlap"), (dict(state_out=ST + 2), INV, "overlap"), (dict(state_out=X, state=None), INV, "overlap"),
    (dict(y=SL + 6), INV, "overlap"), (dict(state_out=HAS), INV, "overlap"), (dict(seq_offsets=Y), INV, "overlap"),
    (dict(y_dtype=qs.QSSM_I8, y_groups=2, y_group_of=G, y_scales=SC, y=G + 63), INV, "overlap")])
def test_conv_refuses(kw, status, word):
    assert conv(**kw) == status and word in message(), message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(tokens=-1), INV, "negative"), (dict(tokens=11), INV, "multiple"), (dict(dstate=0), UNS, "dstate"), (dict(dstate=65), UNS, "dstate"),
    (dict(ngroups=0), INV, "ngroups"), (dict(ngroups=3), INV, "ngroups"), (dict(io_dtype=qs.QSSM_I8), INV, "io_dtype"),
    (dict(y_dtype=qs.QSSM_I8), INV, "y_dtype"), (dict(state_dtype=qs.QSSM_I8), INV, "state_dtype"), (dict(reserved=2), INV, "reserved"),
    (dict(x_stride=63), INV, "x_stride"), (dict(delta_stride=63), INV, "delta_stride"), (dict(B_stride=15), INV, "B_stride"),
    (dict(C_stride=15), INV, "C_stride"), (dict(z_stride=63), INV, "z_stride"), (dict(y_stride=63), INV, "y_stride"),
    (dict(ngroups=2, B_stride=31, C_stride=32), INV, "B_stride"), (dict(delta=None), INV, "null"), (dict(A=None), INV, "null"),
    (dict(B=None), INV, "null"), (dict(C=CC + 1), INV, "C is not aligned"), (dict(A=A + 2), INV, "aligned"), (dict(state=ST + 2), INV, "aligned"),
    (dict(slots=2 ** 40, dim=2 ** 20, x_stride=2 ** 20, delta_stride=2 ** 20, z_stride=2 ** 20, y_stride=2 ** 20), UNS, "slots"),
    (dict(y=X), INV, "overlap"), (dict(y=DEL + 4), INV, "overlap"), (dict(y=Z), INV, "overlap"), (dict(y=BB), INV, "overlap"),
    (dict(y=CC), INV, "overlap"), (dict(y=A + 4092), INV, "overlap"), (dict(y=ST), INV, "overlap"), (dict(state_out=ST + 4), INV, "overlap"),
    (dict(state_out=A, state=None), INV, "overlap"), (dict(state_out=Y), INV, "overlap")])
def test_scan_refuses(kw, status, word):
    assert scan(**kw) == status and word in message(), message()


def test_scan_workspace():
    lib = qs.load()
    size = lambda **kw: lib.qssm_selective_scan_workspace_size(ctypes.byref(scan_args(**kw)))  # noqa: E731
    assert size() == 0 and size(tokens=2) == 0 and size(tokens=0) == 0 and size(tokens=-4) == 0 and size(dstate=99) == 0
    long = dict(tokens=4096, nseq=1)
    need = size(**long)
    assert need > 0 and need % 4 == 0
    assert scan(**long) == WS and str(need) in message()
    assert scan(ws=WSP, ws_bytes=need - 1, **long) == WS
    assert scan(ws=WSP + 8, ws_bytes=need, **long) == INV and "16-byte" in message()
    for at in (X, Y, ST, A):
        assert scan(ws=at, ws_bytes=need, **long) == INV and "overlap" in message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), INV, "negative"), (dict(K=-1), INV, "negative"), (dict(xt=qs.QSSM_I8), INV, "x_dtype"), (dict(rows=2 ** 31), UNS, "rows"),
    (dict(K=2 ** 24 + 1), UNS, "K above"), (dict(xs=255), INV, "x_stride"), (dict(cs=255), INV, "codes_stride"), (dict(ss=3), INV, "scales_stride"),
    (dict(x=None), INV, "null"), (dict(codes=None), INV, "null"), (dict(scales=None), INV, "null"), (dict(x=X + 1), INV, "aligned"),
    (dict(scales=SC + 2), INV, "aligned"), (dict(codes=X), INV, "overlap"), (dict(scales=X), INV, "overlap"), (dict(scales=Y + 1020), INV, "overlap"),
    (dict(rows=2 ** 31 - 1, K=2 ** 10, xs=2 ** 10, cs=2 ** 10, ss=2 ** 31, codes=X + (1 << 50), scales=X + (1 << 51)), UNS, "too large")])
def test_quant_refuses(kw, status, word):
    assert quant(**kw) == status and word in message(), message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), INV, "negative"), (dict(y_dtype=qs.QSSM_I8), INV, "y_dtype"), (dict(reserved=1), INV, "reserved"),
    (dict(K=2 ** 20 + 1, a_stride=2 ** 21, w_stride=2 ** 21), UNS, "K above"), (dict(M=2 ** 27 + 1, a_scales_stride=2 ** 28), UNS, "M or N"),
    (dict(a_stride=383), INV, "a_stride"), (dict(w_stride=383), INV, "w_stride"), (dict(y_stride=255), INV, "y_stride"),
    (dict(a_scales_stride=3), INV, "a_scales_stride"), (dict(a_stride=2 ** 22 + 1), UNS, "2^22"), (dict(w_stride=2 ** 22 + 1), UNS, "2^22"),
    (dict(M=2 ** 27, a_scales_stride=2 ** 27, y_stride=2 ** 32), UNS, "2^58"), (dict(a=None), INV, "null"), (dict(w=None), INV, "null"),
    (dict(a_scales=None), INV, "null"), (dict(w_scales=None), INV, "null"), (dict(y=None), INV, "null"), (dict(y=Y + 2), INV, "aligned"),
    (dict(a_scales=SC + 1), INV, "aligned"), (dict(w_scales=SL + 2), INV, "aligned"), (dict(bias=B + 1), INV, "aligned"),
    (dict(M=2 ** 27, N=2 ** 20, a_scales_stride=2 ** 27, y_stride=2 ** 20), UNS, "too large"),
    (dict(y=X), INV, "overlap"), (dict(y=W + 4), INV, "overlap"), (dict(y=SC), INV, "overlap"), (dict(y=SL), INV, "overlap"), (dict(y=B), INV, "overlap")])
def test_gemm_refuses(kw, status, word):
    assert gemm(**kw) == status and word in message(), message()


def test_null_arguments_and_empty_calls():
    lib = qs.load()
    for f in (lib.qssm_causal_conv, lib.qssm_gemm_f8):
        assert f(None, None) == INV
    assert lib.qssm_selective_scan(None, None, 0, None) == INV and lib.qssm_selective_scan_workspace_size(None) == 0
    assert conv(nseq=0, tokens=0, slots=0) == qs.QSSM_OK and conv(dim=0, x=None, y=None) == qs.QSSM_OK
    assert scan(nseq=0, tokens=0, slots=0) == qs.QSSM_OK and scan(dim=0) == qs.QSSM_OK
    assert quant(rows=0) == qs.QSSM_OK and quant(K=0) == qs.QSSM_OK
    assert gemm(M=0, a_scales_stride=0) == qs.QSSM_OK and gemm(N=0) == qs.QSSM_OK
    assert lib.qssm_quant_f8_weight(None, -1, 4, None, None) == INV and lib.qssm_quant_f8_weight(None, 1, 4, None, None) == INV


# ------------------------------------------------------------------------------------------------
# The binding: shapes and types that it refuses before it asks for a GPU

z = torch.zeros
I32, U8, F8 = torch.int32, torch.uint8, torch.float8_e4m3fn


def conv_call(**kw):
    a = dict(x=z(6, 8), weight=z(8, 4), y=z(6, 8), bias=z(8), nseq=2, state=z(3, 3, 8), state_out=z(3, 3, 8),
             state_slots=z(2, dtype=I32), has_state=z(2, dtype=U8))
    a.update(kw)
    return qs.causal_conv_args(**a)


def scan_call(**kw):
    a = dict(x=z(6, 8), delta=z(6, 8), A=z(8, 4), B=z(6, 4), C=z(6, 4), y=z(6, 8), D=z(8), z=z(6, 8), delta_bias=z(8), nseq=2,
             state=z(3, 8, 4), state_out=z(3, 8, 4))
    a.update(kw)
    return qs.selective_scan_args(**a)


@pytest.mark.parametrize("kw,error,word", [
    (dict(x=z(6)), ValueError, "x must be"), (dict(weight=z(7, 4)), ValueError, "weight"), (dict(bias=z(7)), ValueError, "bias"),
    (dict(nseq=None), ValueError, "nseq"), (dict(nseq=3, seq_offsets=z(3, dtype=I32)), ValueError, "differ"),
    (dict(seq_offsets=z(0, dtype=I32), nseq=None), ValueError, "seq_offsets"), (dict(state=z(3, 3, 7)), ValueError, "state"),
    (dict(state=z(3, 2, 8)), ValueError, "state"), (dict(state=z(3, 3, 8, dtype=torch.float16)), TypeError, "state"),
    (dict(state_out=z(4, 3, 8)), ValueError, "one shape"), (dict(state_slots=z(3, dtype=I32)), ValueError, "state_slots"),
    (dict(has_state=z(1, dtype=U8)), ValueError, "has_state"), (dict(y=z(6, 8, dtype=torch.int8)), ValueError, "y_group_of")])
def test_conv_args_refuse(kw, error, word):
    with pytest.raises(error, match=word) as e:
        conv_call(**kw)
    assert "GPU" not in str(e.value)


@pytest.mark.parametrize("kw,error,word", [
    (dict(x=z(6)), ValueError, "x must be"), (dict(A=z(7, 4)), ValueError, "A"), (dict(D=z(7)), ValueError, "D must"),
    (dict(delta_bias=z(9)), ValueError, "delta_bias"), (dict(bc_groups=0), ValueError, "bc_groups"), (dict(bc_groups=1.5), ValueError, "bc_groups"),
    (dict(bc_groups=2 ** 33), ValueError, "bc_groups"), (dict(nseq=None), ValueError, "nseq"), (dict(state=z(3, 8, 5)), ValueError, "state"),
    (dict(state=z(3, 8, 4, dtype=torch.int8)), TypeError, "state"), (dict(state=z(3, 8, 4, dtype=torch.float16)), ValueError, "one shape and type")])
def test_scan_args_refuse(kw, error, word):
    with pytest.raises(error, match=word) as e:
        scan_call(**kw)
    assert "GPU" not in str(e.value)


def test_f8_args_refuse():
    a, w = z(4, 256, dtype=F8), z(130, 256, dtype=F8)
    for kw in (dict(a=z(4, 255, dtype=F8)), dict(w_scales=z(1, 2)), dict(w_scales=z(2, 3)), dict(bias=z(129)), dict(a=z(256, dtype=F8))):
        k = dict(a=a, a_scales=z(2, 4), w=w, w_scales=z(2, 2), y=z(4, 130))
        k.update(kw)
        with pytest.raises(ValueError) as e:
            qs.gemm_f8_args(**k)
        assert "GPU" not in str(e.value)
    with pytest.raises(ValueError, match="x must be"):
        qs.qssm_quant_f8(z(4), z(4, dtype=F8), z(1, 1))
    with pytest.raises(ValueError, match="GPU"):
        conv_call()
    with pytest.raises(ValueError, match="GPU"):
        scan_call()
