"""The operators over packed sequences and in block-scaled e4m3 together, as a Mamba1 block runs them: prompts, then
single tokens on the same caches. Every stage is checked against the oracle on the values that the stage before it
left on the GPU; then whole steps under HIP graph replay and on another stream against eager ones, bit for bit."""
import numpy as np
import pytest

import oracle.packed as op
from tests.test_gpu_causal_conv import bound as conv_bound

pytestmark = pytest.mark.gpu

DIM, D, N, R, W = 136, 200, 16, 12, 4


def params(seed):
    r = np.random.default_rng([61, seed])
    n = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    dt = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), D))
    return dict(w_in=n(2 * D, DIM) / 12, conv_w=n(D, W) / 2, conv_b=0.1 * n(D), w_x=n(R + 2 * N, D) / 10, w_dt=n(D, R) / 12,
                dt_b=(dt + np.log(-np.expm1(-dt))).astype(np.float32), A=-np.exp(n(D, N)), Dskip=n(D), w_out=n(DIM, D) / 14)


def host(t):
    return t.cpu().numpy().copy()


def check_linear(lin, x, y):
    """The quantizer's codes bit for bit, and the product within its roundings and an fp16 y's."""
    M = len(x)
    codes, scales = host(lin.codes[:M].view(__import__("torch").uint8)), host(lin.scales[:, :M])
    want_c, want_s = op.quant_f8(x)
    assert np.array_equal(codes, want_c) and np.array_equal(scales, want_s)
    want, e = op.gemm_f8(codes, scales, lin.w_host, lin.w_scales_host, f16=True)
    e = e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25
    assert np.all(np.abs(y.astype(np.float64) - want) <= e)


def check_step(blk, hidden, slots, offsets, has, before, cut):
    """A step that ran on `hidden` with the states `before`."""
    T = len(hidden)
    xz, x, dbc, dt, y, out = (host(t[:T]) for t in (blk.xz, blk.x, blk.dbc, blk.dt, blk.y, blk.out))
    check_linear(blk.proj_in, hidden, xz)
    nseq = len(slots)
    init = op.initial_states(before[0], nseq, (W - 1, D), slots, has)
    want, v, s, final = op.causal_conv(xz[:, :D], host(blk.conv_w), host(blk.conv_b), True, offsets, init)
    assert np.all(np.abs(x - want) <= conv_bound(want, v, s, W, True, True))
    assert np.array_equal(host(blk.conv_state), op.store_states(before[0], final, slots))
    check_linear(blk.proj_x, x, dbc)
    check_linear(blk.proj_dt, dbc[:, :R], dt)
    init = op.initial_states(before[1], nseq, (D, N), slots, has)
    want, ey, final, ef = op.selective_scan(x, dt, host(blk.A), dbc[:, R:R + N], dbc[:, R + N:], host(blk.Dskip), xz[:, D:],
                                            host(blk.dt_b), True, 1, offsets, init, cut=T if cut else 0)
    ey = ey + 2.0 ** -11 * (np.abs(want) + ey) + 2.0 ** -25
    assert np.all(np.abs(y - want) <= ey)
    state = host(blk.ssm_state)
    for i in range(nseq):
        assert np.all(np.abs(state[slots[i]] - final[i]) <= ef[i])
    keep = np.setdiff1d(np.arange(len(state)), slots)
    assert np.array_equal(state[keep], before[1][keep])
    check_linear(blk.proj_out, y, out)


def test_prompts_then_tokens_stage_by_stage(dev):
    import torch
    import quantized_state_space_amd.workloads as wl
    print("\n[f8 block]", flush=True)
    blk = wl.F8MambaBlock(params(1), 6, 300, dev)
    r = np.random.default_rng(1)
    blk.conv_state.copy_(torch.from_numpy(r.standard_normal((6, W - 1, D)).astype(np.float16)))
    blk.ssm_state.copy_(torch.from_numpy(r.standard_normal((6, D, N)).astype(np.float32)))
    slots = np.array([4, 0, 5], np.int32)
    offsets = np.array([0, 150, 151, 260], np.int32)
    has = np.array([0, 1, 0], np.uint8)
    dv = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    before = host(blk.conv_state), host(blk.ssm_state)
    hidden = r.standard_normal((260, DIM)).astype(np.float16)
    blk.step(dv(hidden), dv(slots), dv(offsets), dv(has))
    torch.cuda.synchronize()
    check_step(blk, hidden, slots, offsets, has, before, cut=True)
    for k in range(3):
        before = host(blk.conv_state), host(blk.ssm_state)
        hidden = r.standard_normal((3, DIM)).astype(np.float16)
        blk.step(dv(hidden), dv(slots))
        torch.cuda.synchronize()
        check_step(blk, hidden, slots, np.arange(4), None, before, cut=False)


@pytest.mark.parametrize("tokens", [False, True])
def test_steps_replay_from_graphs(dev, tokens):
    """A captured step replayed on new inputs, sequences and states, with eager work between the replays."""
    import torch
    import quantized_state_space_amd.workloads as wl
    print(f"\n[f8 block graph tokens={tokens}]", flush=True)
    T = 5 if tokens else 290
    a, b = (wl.F8MambaBlock(params(2), 7, T, dev) for _ in range(2))
    hidden = torch.zeros(T, DIM, dtype=torch.float16, device=dev)
    slots = torch.arange(5, dtype=torch.int32, device=dev)
    offsets = None if tokens else torch.tensor([0, 100, 100, 170, 180, T], dtype=torch.int32, device=dev)
    has = torch.ones(5, dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(hidden, slots, offsets, has)  # (the workspace grows outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(hidden, slots, offsets, has)
    for t in (a.conv_state, a.ssm_state):
        t.zero_()
    r = np.random.default_rng(2)
    for k in range(4):
        hidden.copy_(torch.from_numpy(r.standard_normal((T, DIM)).astype(np.float16)))
        slots.copy_(torch.from_numpy(r.permutation(7)[:5].astype(np.int32)))
        has.copy_(torch.from_numpy(r.integers(0, 2, 5).astype(np.uint8)))
        if offsets is not None and k == 2:
            offsets.copy_(torch.tensor([0, 10, 200, 201, 203, T - 3], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.step(hidden, slots, offsets, has)
        torch.cuda.synchronize()
        rows = slice(0, T - 3 if offsets is not None and k >= 2 else T)
        assert torch.equal(a.out[rows], b.out[rows]), k
        assert torch.equal(a.conv_state, b.conv_state) and torch.equal(a.ssm_state, b.ssm_state), k


def test_two_streams_at_once(dev):
    """Two blocks with caches and workspaces of their own, each on a stream that is not the tensors' own."""
    import torch
    import quantized_state_space_amd.workloads as wl
    p = params(3)
    blocks = [wl.F8MambaBlock(p, 2, 200, dev) for _ in range(4)]
    r = np.random.default_rng(3)
    hidden = [torch.from_numpy(r.standard_normal((200, DIM)).astype(np.float16)).to(dev) for _ in range(2)]
    slots = torch.tensor([1, 0], dtype=torch.int32, device=dev)
    offsets = torch.tensor([0, 130, 200], dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(5):
        for blk, h, st in zip(blocks, hidden, streams):
            with torch.cuda.stream(st):
                blk.step(h, slots, offsets)
    torch.cuda.synchronize()
    for blk, h in zip(blocks[2:], hidden):
        for k in range(5):
            blk.step(h, slots, offsets)
    torch.cuda.synchronize()
    for x, y in zip(blocks[:2], blocks[2:]):
        assert torch.equal(x.out, y.out) and torch.equal(x.ssm_state, y.ssm_state) and torch.equal(x.conv_state, y.conv_state)


def test_a_stream_that_is_given(dev):
    import torch
    import quantized_state_space_amd as qs
    x = torch.randn(64, 300, device=dev)
    out = []
    for st in (None, torch.cuda.Stream()):
        c = torch.zeros(64, 300, dtype=torch.float8_e4m3fn, device=dev)
        s, y = torch.zeros(3, 64, device=dev), torch.zeros(64, 64, device=dev)
        cy = torch.zeros(64, 300, device=dev)
        torch.cuda.synchronize()
        qs.qssm_quant_f8(x, c, s, stream=st)
        args = qs.gemm_f8_args(c, s, c, torch.ones(1, 3, device=dev), y)
        torch.cuda.synchronize()  # (the ones above are of the current stream)
        qs.qssm_gemm_f8(args, stream=st)
        qs.qssm_causal_conv(qs.causal_conv_args(x, torch.ones(300, 2, device=dev), cy, nseq=2), stream=st)
        torch.cuda.synchronize()
        out.append((c.view(torch.uint8), s, y, cy))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_a_captured_step_outlives_a_larger_one(dev):
    """A step is captured, then the same block runs a larger one, and memory that this might have freed is taken: replays give
    what they gave, and write nothing of others'."""
    import torch
    import quantized_state_space_amd.workloads as wl
    print("\n[f8 block, captured then larger]", flush=True)
    T = 1000
    a, b = (wl.F8MambaBlock(params(4), 9, T, dev) for _ in range(2))
    r = np.random.default_rng(4)
    dv = lambda x: torch.from_numpy(np.asarray(x)).to(dev)  # noqa: E731
    hidden = dv(r.standard_normal((T, DIM)).astype(np.float16))
    slots = torch.arange(9, dtype=torch.int32, device=dev)
    small, large = dv(np.array([0, 150], np.int32)), dv(np.array([0, 300, 470, 600, 601, 601, 780, 850, 900, T], np.int32))
    one = slots[:1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(hidden[:150], one, small)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    at = a.workspace.data_ptr()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(hidden[:150], one, small)
    for blk in (a, b):
        blk.conv_state.zero_()
        blk.ssm_state.zero_()
    a.step(hidden, slots, large)
    b.step(hidden, slots, large)
    torch.cuda.synchronize()
    assert a.workspace.data_ptr() == at
    taken = [torch.full((n,), 0x33, dtype=torch.uint8, device=dev) for n in (1 << 10, 1 << 14, 1 << 17, 1 << 18, 1 << 20) for _ in range(8)]
    for k in range(3):
        hidden.copy_(dv(r.standard_normal((T, DIM)).astype(np.float16)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.step(hidden[:150], one, small)
        torch.cuda.synchronize()
        assert torch.equal(a.out[:150], b.out[:150]) and torch.equal(a.ssm_state, b.ssm_state) and torch.equal(a.conv_state, b.conv_state)
        assert all(bool((t == 0x33).all()) for t in taken)
