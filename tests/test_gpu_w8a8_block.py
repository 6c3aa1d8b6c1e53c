"""The W8A8 block's operators together, as one decoded token runs through them: norm with the residual
stream -> in-projection -> state update on the int8 state -> gated, grouped norm -> out-projection.
Every stage is checked against the oracle on the values the stage before it left on the GPU (so that a
code that sits on a rounding boundary of an fp32 sum cannot spread), over several tokens; then the
whole step captured in a HIP graph against eager steps; and a prefill handing its state over."""
import numpy as np
import pytest

import oracle.w8a8 as ow
import qssm_synth as synth

pytestmark = pytest.mark.gpu

DIMS = dict(batch=5, nheads=8, headdim=64, dstate=128, ngroups=2)
D = 320


def params(cfg, dims=DIMS, d=D):
    p = synth.decode_params(cfg=cfg, **dims)
    r = np.random.default_rng([96, cfg])
    inner, gn = dims["nheads"] * dims["headdim"], dims["ngroups"] * dims["dstate"]
    p["w_in"] = (r.standard_normal((2 * inner + 2 * gn, d)) / np.sqrt(d)).astype(np.float32)
    p["w_out"] = (r.standard_normal((d, inner)) / np.sqrt(inner)).astype(np.float32)
    p["norm_w"] = r.uniform(0.5, 1.5, d).astype(np.float32)
    p["gate_w"] = r.uniform(0.5, 1.5, inner).astype(np.float32)
    return p


def token(cfg, k, dims=DIMS, d=D):
    r = np.random.default_rng([97, cfg, k])
    h = r.standard_normal((dims["batch"], d)).astype(np.float16)
    return h, np.log1p(np.exp(r.normal(-2, 0.5, (dims["batch"], dims["nheads"])))).astype(np.float32)


def host(t):
    return t.cpu().numpy()


def check_linear(lin, codes, scales):
    """Against the exact sums: 2 fp32 roundings of the scaled sum and one to the output's type."""
    want = ow.gemm_w8a8(codes, scales, lin.w_host, lin.w_scales_host)
    got = host(lin.y).astype(np.float64)
    e = 4 * 2.0 ** -24 * np.abs(want)
    if lin.y.dtype.itemsize == 2:
        e = e + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= e)


def test_block_stage_by_stage(dev):
    print("\n[w8a8 block, 3 tokens]", flush=True)
    import torch
    import quantized_state_space_amd.workloads as wl
    p = params(1)
    blk = wl.W8A8DecodeBlock(p, dev)
    B, nh, P, N, G = blk.core.shape
    stream = np.random.default_rng(1).standard_normal((B, D)).astype(np.float32)
    blk.residual.copy_(torch.from_numpy(stream))
    q, s = host(blk.core.state), host(blk.core.state_scales)
    assert np.array_equal(s, ow.row_scales(p["state0"])) and np.array_equal(q, ow.quant(p["state0"], s[..., None]))
    sx, group = host(blk.core.xs), blk.core.group_of
    for k in range(3):
        h, delta = token(1, k)
        blk.hidden.copy_(torch.from_numpy(h))
        blk.delta.copy_(torch.from_numpy(delta))
        blk.step()
        torch.cuda.synchronize()
        codes, scales, stream = ow.rmsnorm_i8(h, p["norm_w"], residual=stream, residual_dtype=np.float32)
        assert np.array_equal(host(blk.codes), codes) and np.array_equal(host(blk.scales), scales), k
        assert np.array_equal(host(blk.residual), stream), k
        for lin in blk.proj_in:
            check_linear(lin, codes, scales)
        # the update on the projected values
        sxc = sx[group].reshape(nh, P)
        xh = ow.quant(host(blk.core.x), sxc) * sxc
        of = (np.arange(G * N) // blk.core.gs).reshape(G, N)
        vals = [np.repeat(ow.quant(host(t), host(sc)[of]) * host(sc)[of], nh // G, axis=1)
                for t, sc in ((blk.core.Bm, blk.core.bs), (blk.core.Cm, blk.core.cs))]
        y, q, s, hh = ow.state_update(q, s, xh, vals[0], vals[1], delta, p["A"], p["D"])
        assert np.array_equal(host(blk.core.state), q) and np.array_equal(host(blk.core.state_scales), s), k
        err = (N + 2) * 2.0 ** -24 * ((np.abs(hh.astype(np.float64)) * np.abs(vals[1][:, :, None, :])).sum(3) +
                                      np.abs(p["D"][None, :, None].astype(np.float64) * xh))
        assert np.all(np.abs(host(blk.core.y) - y) <= err), k
        yc, ys, _ = ow.rmsnorm_i8(host(blk.core.y).reshape(B, nh * P), p["gate_w"], gate=host(blk.z), groups=G)
        assert np.array_equal(host(blk.y_codes), yc) and np.array_equal(host(blk.y_scales), ys), k
        check_linear(blk.out, yc, ys)


def test_block_replays(dev):
    """The captured step on successive tokens equals eager steps bit for bit; other work runs between."""
    print("\n[w8a8 block in a graph]", flush=True)
    import torch
    import quantized_state_space_amd.workloads as wl
    p = params(2)
    a, b = wl.W8A8DecodeBlock(p, dev), wl.W8A8DecodeBlock(p, dev)
    for blk in (a, b):
        blk.residual.zero_()
        blk.hidden.zero_()
        blk.delta.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step()
    torch.cuda.synchronize()
    a.core.state.copy_(b.core.state)
    a.core.state_scales.copy_(b.core.state_scales)
    a.residual.zero_()
    for k in range(4):
        h, delta = token(2, k)
        for blk in (a, b):
            blk.hidden.copy_(torch.from_numpy(h))
            blk.delta.copy_(torch.from_numpy(delta))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.step()
        torch.cuda.synchronize()
        for x, y in ((a.out.y, b.out.y), (a.core.state, b.core.state), (a.core.state_scales, b.core.state_scales),
                     (a.residual, b.residual), (a.y_codes, b.y_codes)):
            assert torch.equal(x, y), k


def test_block_other_state_types(dev):
    """fp32 and fp16 states in the same block: the int8 state's readout stays within its rounding of the
    fp32 one (half a scale per value, weighted by |C|) for the first token."""
    print("\n[w8a8 block, state types]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    import quantized_state_space_amd.workloads as wl
    p = params(3)
    h, delta = token(3, 0)
    out = {}
    for dt in (qs.QSSM_F32, qs.QSSM_F16, qs.QSSM_I8):
        blk = wl.W8A8DecodeBlock(p, dev, state_dtype=dt)
        blk.residual.zero_()
        blk.hidden.copy_(torch.from_numpy(h))
        blk.delta.copy_(torch.from_numpy(delta))
        blk.step()
        torch.cuda.synchronize()
        out[dt] = host(blk.core.y).astype(np.float64)
    B, nh, P, N, G = blk.core.shape
    cs = host(blk.core.cs)[(np.arange(G * N) // 16).reshape(G, N)]
    Ch = np.repeat(np.abs(ow.quant(host(blk.core.Cm), cs) * cs), nh // G, axis=1).sum(axis=2)[:, :, None]
    big = np.abs(p["state0"]).max(axis=3)
    room = 1e-4 * (np.abs(out[qs.QSSM_F32]) + Ch * (big + 1))
    assert np.all(np.abs(out[qs.QSSM_I8] - out[qs.QSSM_F32]) <= 0.5 * big / 127 * Ch + room)
    # half a step of fp16: 2^-11 of each value, or half its least denormal, 2^-25
    assert np.all(np.abs(out[qs.QSSM_F16] - out[qs.QSSM_F32]) <= (2.0 ** -11 * big + 2.0 ** -25) * Ch + room)


def test_prefill_state_handed_over(dev):
    """A chunked prefill's h_last written to the int8 state, one decoded token, and the state read back
    as the h0 of a following prefill: the same values as the oracle's rows."""
    print("\n[prefill -> int8 state -> decode -> prefill]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    import quantized_state_space_amd.workloads as wl
    inp = synth.ssd_inputs(cfg=98, batch=5, seqlen=70, nheads=8, headdim=64, dstate=128, ngroups=2, calib_len=256)
    pre = wl.SsdLayer(inp, dev)
    pre.step()
    p = params(4)
    dec = wl.DecodeLayer(p, dev, state_dtype=qs.QSSM_I8)
    dec.store_state(pre.h_last)
    dec.load_inputs(synth.decode_step_inputs(0, cfg=4, **DIMS))
    torch.cuda.synchronize()
    h = host(pre.h_last)
    s = ow.row_scales(h)
    assert np.array_equal(host(dec.state), ow.quant(h, s[..., None])) and np.array_equal(host(dec.state_scales), s)
    dec.step()
    h0 = torch.empty_like(pre.h_last)
    dec.load_state(h0)
    torch.cuda.synchronize()
    assert np.array_equal(host(h0), host(dec.state) * host(dec.state_scales)[..., None])
    nxt = dict(inp, h0=host(h0))
    cont = wl.SsdLayer(nxt, dev, with_h0=True)
    cont.step()
    torch.cuda.synchronize()
    assert np.all(np.isfinite(host(cont.y)))
