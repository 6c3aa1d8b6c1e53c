"""Rows whose offsets leave 32 bits (elements and bytes), and caches whose slots do: the operators over packed sequences and in
block-scaled e4m3 on columns of very wide tensors, against the same columns in small ones."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def far(t, stride, dev, dtype=None):
    """t [T, C] as the columns of rows `stride` elements apart."""
    import torch
    w = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype if dtype is None else dtype, device=dev)
    v = w.as_strided(t.shape, (stride, 1))
    v.copy_(t)
    return v


def test_convolution_and_quantizer(dev):
    import torch
    import quantized_state_space_amd as qs
    print("\n[conv and quantizer, rows 2^20 apart]", flush=True)
    r = np.random.default_rng(1)
    T, C, stride = 4300, 40, 1 << 20  # the last rows lie 4.5e9 elements, 9e9 bytes from the first
    x = torch.from_numpy(r.standard_normal((T, C)).astype(np.float16)).to(dev)
    w = torch.from_numpy(r.standard_normal((C, 4)).astype(np.float32)).to(dev)
    off = torch.tensor([0, 7, 2100, 4290, T], dtype=torch.int32, device=dev)
    xf = far(x, stride, dev)
    want, got = torch.zeros(T, C, device=dev), torch.zeros(T, C, device=dev)
    s0, s1 = (torch.zeros(4, 3, C, dtype=torch.float16, device=dev) for _ in range(2))
    qs.qssm_causal_conv(qs.causal_conv_args(x, w, want, seq_offsets=off, state_out=s0))
    qs.qssm_causal_conv(qs.causal_conv_args(xf, w, got, seq_offsets=off, state_out=s1))
    assert torch.equal(want, got) and torch.equal(s0, s1)
    y = far(torch.zeros(T, C, dtype=torch.int8, device=dev), stride, dev)
    g, sc = torch.zeros(C, dtype=torch.uint8, device=dev), torch.full((1,), 0.02, device=dev)
    yw = torch.zeros(T, C, dtype=torch.int8, device=dev)
    qs.qssm_causal_conv(qs.causal_conv_args(x, w, yw, seq_offsets=off, y_group_of=g, y_scales=sc))
    qs.qssm_causal_conv(qs.causal_conv_args(xf, w, y, seq_offsets=off, y_group_of=g, y_scales=sc))
    assert torch.equal(y, yw)
    f8 = torch.float8_e4m3fn
    c0, c1 = torch.zeros(T, C, dtype=f8, device=dev), far(torch.zeros(T, C, dtype=torch.uint8, device=dev), stride, dev).view(f8)
    a0, a1 = (torch.zeros(1, T, device=dev) for _ in range(2))
    qs.qssm_quant_f8(x, c0, a0)
    qs.qssm_quant_f8(xf, c1, a1)
    assert torch.equal(c0.view(torch.uint8), c1.view(torch.uint8)) and torch.equal(a0, a1)


def test_scan(dev):
    import torch
    import quantized_state_space_amd as qs
    print("\n[scan, rows 2^20 apart]", flush=True)
    r = np.random.default_rng(2)
    T, D, N, stride = 4200, 24, 16, 1 << 20
    n = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float16)).to(dev)  # noqa: E731
    x, dl, z, B, C = n(T, D), n(T, D), n(T, D), n(T, N), n(T, N)
    A = -torch.exp(torch.randn(D, N, device=dev))
    out = []
    for place in (lambda t: t, lambda t: far(t, stride, dev)):
        y = place(torch.zeros(T, D, dtype=torch.float16, device=dev))
        st = torch.zeros(2, D, N, device=dev)
        args = qs.selective_scan_args(place(x), place(dl), A, place(B), place(C), y, z=place(z), nseq=2, state=st, state_out=st)
        ws = torch.empty(qs.qssm_selective_scan_workspace_size(args), dtype=torch.uint8, device=dev)
        qs.qssm_selective_scan(args, ws)
        torch.cuda.synchronize()
        out.append((y.clone(), st))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_slots(dev):
    """Caches of more than 2^31 elements: single tokens and short prompts in their last slots."""
    import torch
    import quantized_state_space_amd as qs
    print("\n[slots past 2^31 elements]", flush=True)
    r = np.random.default_rng(3)
    D, N = 8192, 16
    slots = (1 << 31) // (D * N) + 5
    n = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float16)).to(dev)  # noqa: E731
    cache = torch.zeros(slots, D, N, device=dev)
    small = torch.zeros(3, D, N, device=dev)
    conv, csmall = torch.zeros((1 << 31) // (3 * D) + 5, 3, D, dtype=torch.float16, device=dev), torch.zeros(3, 3, D, dtype=torch.float16, device=dev)
    A, w = -torch.exp(torch.randn(D, N, device=dev)), torch.randn(D, 4, device=dev)
    at = torch.tensor([slots - 1, 0, slots - 3], dtype=torch.int32, device=dev)
    cat = torch.tensor([conv.shape[0] - 1, 0, conv.shape[0] - 2], dtype=torch.int32, device=dev)
    for rows in (2, 1, 1):
        x, dl, B, C = n(3 * rows, D), n(3 * rows, D), n(3 * rows, N), n(3 * rows, N)
        y0, y1 = (torch.zeros(3 * rows, D, device=dev) for _ in range(2))
        qs.qssm_selective_scan(qs.selective_scan_args(x, dl, A, B, C, y0, nseq=3, state=cache, state_out=cache, state_slots=at))
        qs.qssm_selective_scan(qs.selective_scan_args(x, dl, A, B, C, y1, nseq=3, state=small, state_out=small))
        assert torch.equal(y0, y1) and torch.equal(cache[at.long()], small)
        qs.qssm_causal_conv(qs.causal_conv_args(x, w, y0, nseq=3, state=conv, state_out=conv, state_slots=cat))
        qs.qssm_causal_conv(qs.causal_conv_args(x, w, y1, nseq=3, state=csmall, state_out=csmall))
        assert torch.equal(y0, y1) and torch.equal(conv[cat.long()], csmall)
    assert int(cache.count_nonzero()) == int(small.count_nonzero())


def test_linear_layer(dev):
    import torch
    import quantized_state_space_amd as qs
    print("\n[linear layer, rows 2^22 apart]", flush=True)
    r = np.random.default_rng(4)
    stride = 1 << 22
    f8 = torch.float8_e4m3fn
    for M, N, K in ((700, 600, 256), (12, 700, 256)):
        a, w = (torch.from_numpy(r.integers(0, 100, s).astype(np.uint8)).to(dev) for s in ((M, K), (N, K)))
        sa, sw = torch.rand(2, M, device=dev), torch.rand(-(-N // 128), 2, device=dev)
        want = torch.zeros(M, N, device=dev)
        qs.qssm_gemm_f8(qs.gemm_f8_args(a.view(f8), sa, w.view(f8), sw, want))
        af, wf = far(a, stride, dev).view(f8), far(w, stride, dev).view(f8)
        saf = far(sa, 1 << 31, dev)
        got = far(torch.zeros(M, N, device=dev), stride, dev)
        qs.qssm_gemm_f8(qs.gemm_f8_args(af, saf, wf, sw, got))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
