"""The strips of the causal convolution by their rows: on the CPU, that the library's choice gives the named ones; on the GPU,
strips of every length against the oracle, with sequences that begin anywhere in them. The oracle computes some of the channels,
the first and last and those on both sides of a wave's."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle.packed as op

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# rows of a strip, tokens, channels (an odd number: one a lane, of 64 in a wave; even: two, of 128)
STRIPS = [(64, 4200, 16384), (32, 2100, 16384), (16, 1100, 16384), (8, 530, 16384), (64, 4231, 8201), (32, 2105, 8201), (16, 1111, 8201), (8, 400, 8201),
          (64, 16384, 8192)]


@pytest.mark.parametrize("rows,T,C", STRIPS)
def test_choice(tmp_path_factory, rows, T, C):
    so = str(tmp_path_factory.mktemp("forms") / "forms.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-std=c++17", os.path.join(ROOT, "tests", "host_causal_conv_forms.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).host_strip
    f.argtypes, f.restype = [ctypes.c_int64] * 2, ctypes.c_int64
    assert f(T, -(-C // (64 if C % 2 else 128))) == rows


def offsets(r, T):
    """Long, short and empty sequences; some that begin right before, at and behind multiples of 8 and 64; rows of none at both ends."""
    at = [*r.integers(3, T - 5, 12), *(np.array([64, 65, 66, 127, 128, 134, 135, 136, 137, 200, 200, 256, 319, 321, 322])), *np.arange(330, 350, 2)]
    return np.concatenate([[3, 3], np.sort(at), [T - 5, T - 5]]).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("xt,yt", [("float16", "int8"), ("float16", "float16"), ("float32", "int8"), ("float32", "float32")])
@pytest.mark.parametrize("rows,T,C", STRIPS[:-1])
def test_strips_against_oracle(dev, rows, T, C, xt, yt):
    import torch
    import quantized_state_space_amd as qs
    from tests.test_gpu_causal_conv import bound
    print(f"\n[causal_conv strips of {rows} T={T} C={C} {xt} {yt}]", flush=True)
    r = np.random.default_rng([55, rows, C])
    g = torch.Generator(device=dev).manual_seed(rows + C)
    xt, yt = getattr(torch, xt), getattr(torch, yt)
    W = 4 if rows != 16 else 3
    n = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    off = offsets(r, T)
    nseq = len(off) - 1
    x, w, b = n(T, C).to(xt), 0.6 * n(C, W), n(C)
    state = n(nseq + 2, W - 1, C).to(xt)
    slot = r.permutation(nseq + 2)[:nseq].astype(np.int32)
    slot[4] = -1
    has = r.integers(0, 2, nseq).astype(np.uint8)
    gof = torch.from_numpy(r.integers(0, 4, C).astype(np.uint8)).to(dev)
    sc = torch.tensor([0.02, 0.004, 0.1, 0.5], device=dev)
    fill = 99 if yt == torch.int8 else 7.0
    y = torch.full((T, C), fill, dtype=yt, device=dev)
    pick = np.unique(np.concatenate([np.arange(8), np.arange(60, 70), np.arange(124, 132), np.arange(C - 70, C), r.integers(0, C, 40)]))
    at = torch.from_numpy(pick).to(dev)
    before = state[:, :, at].cpu().numpy()
    dv = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    qs.qssm_causal_conv(qs.causal_conv_args(x, w, y, bias=b, seq_offsets=dv(off), state=state, state_out=state, state_slots=dv(slot),
                                            has_state=dv(has), y_group_of=gof, y_scales=sc))
    torch.cuda.synchronize()
    init = op.initial_states(before, nseq, (W - 1, len(pick)), slot, has)
    want, v, s, final = op.causal_conv(x[:, at].cpu().numpy(), w[at].cpu().numpy(), b[at].cpu().numpy(), True, off, init)
    got = y[:, at].cpu().numpy()
    inside = slice(off[0], off[-1])
    if yt == torch.int8:
        codes = op.conv_codes(want, sc.cpu().numpy()[gof[at].cpu().numpy()])
        assert np.array_equal(got[inside], codes[inside])
    else:
        e = np.abs(got.astype(np.float64) - want)[inside]
        assert np.all(e <= bound(want, v, s, W, True, yt == torch.float16)[inside]), e.max()
    assert bool((y[:off[0]] == fill).all()) and bool((y[off[-1]:] == fill).all()), "rows of no sequence were written"
    assert np.array_equal(state[:, :, at].cpu().numpy(), op.store_states(before, final, slot))
