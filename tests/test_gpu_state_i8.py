"""GPU parity of the int8 recurrent state (write, read back, decode update) against the oracle. New codes
and scales are fixed bit for bit; y is an fp32 sum of N products and the skip term, each step rounding
by 2^-24: |error| <= (N + 2) 2^-24 (sum |C h| + |D x|), with x, B, C and h exactly the oracle's."""
import numpy as np
import pytest

import oracle.w8a8 as ow

pytestmark = pytest.mark.gpu


def special_rows(r, rows, N, dtype):
    h = (r.standard_normal((rows, N)) * np.exp(r.uniform(-8, 4, (rows, 1)))).astype(dtype)
    k = min(rows, 8)
    with np.errstate(over="ignore"):
        for i, f in enumerate([0, np.nan, np.inf, -np.inf, 1e-30, 1e36, 6e-8, 1.0][:k]):
            if i in (1, 2, 3):
                h[i, i % N] = f
            elif i == 7:
                h[i] = (np.arange(N) % 255 - 127) * 0.5  # ties when the absmax is 63.5
            else:
                h[i] = (h[i].astype(np.float64) * f).astype(dtype)
    return h


@pytest.mark.parametrize("rows,N,f16", [(1, 1, False), (9, 16, True), (40, 128, False), (33, 100, True),
                                        (17, 7, False), (1000, 64, False), (5, 300, True), (8, 4096, False),
                                        (301, 256, False), (64, 32, True)])
def test_write_and_read_back(dev, rows, N, f16):
    print(f"\n[state rows={rows} N={N} f16={f16}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    h = special_rows(np.random.default_rng([93, rows, N]), rows, N, np.float16 if f16 else np.float32)
    codes = torch.full((rows, N), -77, dtype=torch.int8, device=dev)
    sc = torch.full((rows,), float("nan"), device=dev)
    qs.qssm_state_quant(torch.from_numpy(h).to(dev), codes, sc)
    want_s = ow.row_scales(h)
    want = ow.quant(h.astype(np.float32), want_s[:, None])
    assert np.array_equal(sc.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want)
    if rows > 4:
        sc[2], sc[4] = float("inf"), 0.0  # not valid: read back as 0
        want_s[2] = want_s[4] = 0
    for dt in (torch.float32, torch.float16):
        out = torch.full((rows, N), float("nan"), dtype=dt, device=dev)
        qs.qssm_state_dequant(codes, sc, out)
        with np.errstate(over="ignore"):
            v = (want.astype(np.float32) * want_s[:, None]).astype(np.float16 if dt == torch.float16 else np.float32)
        assert np.array_equal(out.cpu().numpy(), v)


def test_unaligned_rows(dev):
    """Views that start at any element: the wide loads are only taken where the addresses allow them."""
    print("\n[state rows at odd addresses]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    r = np.random.default_rng(94)
    h = r.standard_normal(16 * 128 + 3).astype(np.float32)
    ht = torch.from_numpy(h).to(dev)
    for off in (1, 2, 3):
        hv = ht[off:off + 16 * 128].view(16, 128)
        cb = torch.zeros(16 * 128 + 3, dtype=torch.int8, device=dev)
        codes, sc = cb[off:off + 16 * 128].view(16, 128), torch.empty(16, device=dev)
        qs.qssm_state_quant(hv, codes, sc)
        want_s = ow.row_scales(hv.cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), ow.quant(hv.cpu().numpy(), want_s[:, None]))
        assert int(cb[:off].abs().sum()) == 0 and int(cb[off + 16 * 128:].abs().sum()) == 0
        ob = torch.zeros(16 * 128 + 3, device=dev)
        out = ob[off:off + 16 * 128].view(16, 128)
        qs.qssm_state_dequant(codes, sc, out)
        assert np.array_equal(out.cpu().numpy(), codes.cpu().numpy() * want_s[:, None])


def make(seed, B, nh, P, N, G, gs, xg=3):
    r = np.random.default_rng([95, seed])
    d = dict(x=r.standard_normal((B, nh, P)), B=r.standard_normal((B, G, N)), C=r.standard_normal((B, G, N)),
             x_scales=r.uniform(0.01, 0.05, xg), B_scales=r.uniform(0.01, 0.05, G * N // gs),
             C_scales=r.uniform(0.01, 0.05, G * N // gs), delta=np.log1p(np.exp(r.normal(-1, 1, (B, nh)))),
             A=-np.exp(r.uniform(0, 2, nh)), D=r.standard_normal(nh), scales=r.uniform(1e-3, 1e-1, (B, nh, P)))
    d = {k: v.astype(np.float32) for k, v in d.items()}
    d["group_of"] = r.integers(0, xg, nh * P).astype(np.uint8)
    d["codes"] = r.integers(-128, 128, (B, nh, P, N)).astype(np.int8)
    return d


def dequantized(d, gs):
    B, nh, P = d["x"].shape
    G, N = d["B"].shape[1:]
    sx = d["x_scales"][d["group_of"]].reshape(nh, P)
    xq = ow.quant(d["x"], sx)
    of = (np.arange(G * N) // gs).reshape(G, N)
    out = [xq * np.where(ow.scale_ok(sx), sx, 0).astype(np.float32)]
    for k in ("B", "C"):
        s = d[k + "_scales"][of]
        v = ow.quant(d[k], s) * np.where(ow.scale_ok(s), s, 0).astype(np.float32)
        out.append(np.repeat(v, nh // G, axis=1))
    return xq, out


class Update:
    def __init__(self, dev, d, gs, y_out=None, skip=True):
        import torch
        import quantized_state_space_amd as qs
        self.t = {k: torch.from_numpy(v).to(dev) for k, v in d.items()}
        t = self.t
        self.state = t["codes"].clone()
        self.y = torch.full(d["x"].shape, -77 if y_out else float("nan"),
                            dtype=torch.int8 if y_out else torch.float32, device=dev)
        yo = [None] * 3 if y_out is None else [torch.from_numpy(v).to(dev) for v in y_out]
        self.xq = torch.empty(d["x"].shape, dtype=torch.int8, device=dev)
        self.args = qs.update_args(t["x"], t["group_of"], t["x_scales"], t["B"], t["C"], t["B_scales"],
                                   t["C_scales"], gs, t["delta"], t["A"], self.state, self.y,
                                   Dskip=t["D"] if skip else None, xq_out=self.xq, y_group_of=yo[0],
                                   y_scales=yo[1], y_bias=yo[2])


CASES = [(1, 1, 1, 16, 1, 16), (2, 4, 64, 128, 2, 16), (3, 6, 48, 64, 3, 16), (1, 8, 80, 32, 1, 8),
         (2, 2, 33, 256, 1, 32), (4, 16, 64, 128, 8, 4), (1, 2, 5, 128, 2, 128), (2, 3, 300, 16, 3, 2)]


@pytest.mark.parametrize("B,nh,P,N,G,gs", CASES)
def test_update_against_oracle(dev, B, nh, P, N, G, gs):
    print(f"\n[state_update_i8 B={B} nh={nh} P={P} N={N} G={G} gs={gs}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(B + nh + P + N, B, nh, P, N, G, gs)
    d["scales"].reshape(-1)[0] = np.inf      # an invalid scale reads as 0
    d["codes"].reshape(-1, N)[-1] = 0        # an empty state
    if d["scales"].size > 8:
        d["scales"].reshape(-1)[5] = 1e30    # a state that dwarfs the input
        d["scales"].reshape(-1)[6] = 2e-30
        d["x"].reshape(-1)[7] = 0            # no input
        d["scales"].reshape(-1)[7] = 0       # ... and no state: scale 1, codes 0
    xq, (xh, Bh, Ch) = dequantized(d, gs)
    y, q, s, h = ow.state_update(d["codes"], d["scales"], xh, Bh, Ch, d["delta"], d["A"], d["D"])
    err = (N + 2) * 2.0 ** -24 * ((np.abs(h.astype(np.float64)) * np.abs(Ch[:, :, None, :])).sum(3) +
                                  np.abs(d["D"][None, :, None].astype(np.float64) * xh))
    # from another buffer, then in place
    u = Update(dev, d, gs)
    s_out = torch.full((B, nh, P), float("nan"), device=dev)
    u.state.fill_(-77)
    qs.qssm_state_update_i8(u.args, s_out, state_in=u.t["codes"], scales_in=u.t["scales"])
    torch.cuda.synchronize()
    assert np.array_equal(u.t["codes"].cpu().numpy(), d["codes"])
    assert np.array_equal(u.xq.cpu().numpy(), xq)
    v = Update(dev, d, gs)
    qs.qssm_state_update_i8(v.args, v.t["scales"])
    torch.cuda.synchronize()
    for st, sc, yy in ((u.state, s_out, u.y), (v.state, v.t["scales"], v.y)):
        assert np.array_equal(sc.cpu().numpy(), s)
        assert np.array_equal(st.cpu().numpy(), q), (st.cpu().numpy() != q).sum()
        assert np.all(np.abs(yy.cpu().numpy().astype(np.float64) - y) <= err)


def test_update_not_finite(dev):
    """delta of Inf or NaN, or a scale near the top of the range, makes rows that are not finite: NaN
    codes are 0, infinities saturate, the scale is that of the finite values; y follows the arithmetic."""
    print("\n[state_update_i8 not finite]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(1, 2, 4, 32, 128, 2, 16)
    d["delta"][0, 0], d["delta"][1, 1], d["delta"][1, 2] = np.nan, np.inf, 3e38
    d["scales"][0, 1] = 2.0 ** 100
    d["A"][2] = 0.01
    d["B_scales"][:4] = 2.0 ** 90
    with np.errstate(all="ignore"):
        _, (xh, Bh, Ch) = dequantized(d, 16)
        y, q, s, h = ow.state_update(d["codes"], d["scales"], xh, Bh, Ch, d["delta"], d["A"], None)
    u = Update(dev, d, 16, skip=False)
    qs.qssm_state_update_i8(u.args, u.t["scales"])
    torch.cuda.synchronize()
    assert not np.all(np.isfinite(h))
    assert np.array_equal(u.t["scales"].cpu().numpy(), s)
    assert np.array_equal(u.state.cpu().numpy(), q)


def test_update_int8_output(dev):
    """y as int8 codes: within one code of the exact rule on the oracle's y, and exact away from a
    rounding boundary."""
    print("\n[state_update_i8 int8 y]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(2, 3, 4, 64, 128, 2, 16)
    yg = (np.arange(256) % 3).astype(np.uint8)
    ys, yb = np.float32([0.05, 0.1, 0.02]), np.linspace(-0.1, 0.1, 256).astype(np.float32)
    _, (xh, Bh, Ch) = dequantized(d, 16)
    y, q, s, h = ow.state_update(d["codes"], d["scales"], xh, Bh, Ch, d["delta"], d["A"], d["D"])
    u = Update(dev, d, 16, y_out=(yg, ys, yb))
    qs.qssm_state_update_i8(u.args, u.t["scales"])
    torch.cuda.synchronize()
    sy = ys[yg].reshape(4, 64)
    t = (y + yb.reshape(4, 64)) / sy
    far = np.abs(t - np.floor(t) - 0.5) > 130 * 2.0 ** -24 * (np.abs(h) * np.abs(Ch[:, :, None, :])).sum(3) / sy + 1e-4
    got = u.y.cpu().numpy()
    want = np.clip(np.rint(t), -128, 127)
    assert np.array_equal(got[far], want[far]) and np.abs(got - want).max() <= 1 and far.mean() > 0.9
    assert np.array_equal(u.state.cpu().numpy(), q)


def test_steps_replay_and_drift(dev):
    """64 tokens through a captured update in place equal the oracle's step by step; the dequantized state
    stays within the accumulated rounding of an unrounded state: each step adds at most half a scale and
    the decay only shrinks what is there."""
    print("\n[state_update_i8 64 captured steps]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(3, 2, 4, 16, 64, 2, 16)
    u = Update(dev, d, 16)
    sc = u.t["scales"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qs.qssm_state_update_i8(u.args, sc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.qssm_state_update_i8(u.args, sc)
    torch.cuda.synchronize()
    u.state.copy_(torch.from_numpy(d["codes"]))
    sc.copy_(torch.from_numpy(d["scales"]))
    q, s = d["codes"], d["scales"]
    real = q.astype(np.float64) * s[..., None]
    drift = np.zeros(real.shape)
    for k in range(64):
        n = make(100 + k, 2, 4, 16, 64, 2, 16)
        for name in ("x", "B", "C", "delta"):
            d[name] = n[name]
            u.t[name].copy_(torch.from_numpy(n[name]))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _, (xh, Bh, Ch) = dequantized(d, 16)
        y, q, s, h = ow.state_update(q, s, xh, Bh, Ch, d["delta"], d["A"], d["D"])
        assert np.array_equal(u.state.cpu().numpy(), q), k
        assert np.array_equal(sc.cpu().numpy(), s), k
        dA = np.exp(d["delta"].astype(np.float64) * d["A"])[:, :, None, None]
        real = dA * real + (d["delta"].astype(np.float64)[:, :, None] * xh)[..., None] * Bh[:, :, None, :]
        drift = dA * drift + 0.5 * s[..., None] * (1 + 1e-5) + 1e-5 * np.abs(real).max()
        assert np.all(np.abs(q * s[..., None].astype(np.float64) - real) <= drift), k


def test_more_tiles_than_a_grid_dimension(dev):
    """2^23 + 5 sequences of one row each: the grid's second dimension."""
    print("\n[state_update_i8 2^23 + 5 sequences]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    B, N = 2 ** 23 + 5, 16
    g = torch.Generator(device=dev).manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, Bm, Cm = rn(B, 1, 1), rn(B, 1, N), rn(B, 1, N)
    one = lambda v, n=1: torch.full((n,), v, device=dev)  # noqa: E731
    delta = torch.rand(B, 1, generator=g, device=dev)
    codes = torch.randint(-127, 128, (B, 1, 1, N), dtype=torch.int8, generator=g, device=dev)
    sc = 0.01 + torch.rand(B, 1, 1, generator=g, device=dev)
    out, s_out, y = torch.empty_like(codes), torch.full_like(sc, float("nan")), torch.empty(B, 1, 1, device=dev)
    args = qs.update_args(x, torch.zeros(1, dtype=torch.uint8, device=dev), one(0.03), Bm, Cm, one(0.03), one(0.03), N,
                          delta, one(-0.7), out, y)
    qs.qssm_state_update_i8(args, s_out, state_in=codes, scales_in=sc)
    rows = torch.cat([torch.arange(4), torch.arange(2 ** 22 - 2, 2 ** 22 + 2), torch.arange(2 ** 23 - 3, B)]).to(dev)
    n = lambda t: t[rows].cpu().numpy()  # noqa: E731
    s3 = np.float32(0.03)
    xh, Bh, Ch = (ow.quant(n(t), s3) * s3 for t in (x, Bm, Cm))
    yr, q, s, h = ow.state_update(n(codes), n(sc), xh[:, :, 0][:, :, None], Bh, Ch, n(delta), np.float32([-0.7]))
    assert np.array_equal(n(out), q) and np.array_equal(n(s_out), s)
    err = (N + 2) * 2.0 ** -24 * (np.abs(h.astype(np.float64)) * np.abs(Ch[:, :, None, :])).sum(3)
    assert np.all(np.abs(n(y) - yr) <= err)
    assert not bool(torch.isnan(s_out).any())
