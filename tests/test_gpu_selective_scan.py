"""GPU parity of the selective scan over packed sequences against the fp64 oracle, within the bound that the oracle
carries along for the kernel's fp32 roundings (oracle/packed.py), and half a step of fp16 where y or the state is fp16."""
import numpy as np
import pytest

import oracle.packed as op
from tests.test_gpu_causal_conv import offsets_of

pytestmark = pytest.mark.gpu


def case(seed, T, D, N, groups, xt, off, st=np.float32, slow=False):
    r = np.random.default_rng([52, seed])
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    nseq = off if isinstance(off, int) else len(off) - 1
    slots = nseq + 2
    slot = r.permutation(slots)[:nseq].astype(np.int32)
    if nseq > 2:
        slot[0], slot[2] = slots, -3
    dt = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), D))
    return dict(x=n(T, D).astype(xt), delta=(0.5 * n(T, D)).astype(xt), z=n(T, D).astype(xt),
                B=n(T, groups * N).astype(xt), C=n(T, groups * N).astype(xt),
                A=(-np.arange(1, N + 1) * np.exp(0.1 * n(D, N)) * (0.02 if slow else 1.0)).astype(np.float32),
                D=n(D).astype(np.float32), bias=(dt + np.log(-np.expm1(-dt))).astype(np.float32), off=off, nseq=nseq,
                groups=groups, state=n(slots, D, N).astype(st), slot=slot, has=r.integers(0, 2, nseq).astype(np.uint8))


def run(dev, c, yt, gate=True, softplus=True, pad=0, in_place=True, state=True, slot=True, has=True, bias=True, skip=True):
    import torch
    import quantized_state_space_amd as qs
    T, D = c["x"].shape

    def dv(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    def wide(a):
        w = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device=dev).to(dv(a).dtype)
        w[:, :a.shape[1]] = dv(a)
        return w[:, :a.shape[1]]

    yw = torch.full((T, D + pad), 7.0, dtype=yt, device=dev)
    st = dv(c["state"]) if state else None
    so = st if in_place else (torch.full_like(st, 3.0) if state else None)
    kw = dict(nseq=c["off"]) if isinstance(c["off"], int) else dict(seq_offsets=dv(c["off"]))
    args = qs.selective_scan_args(wide(c["x"]), wide(c["delta"]), dv(c["A"]), wide(c["B"]), wide(c["C"]), yw[:, :D],
                                  D=dv(c["D"]) if skip else None, z=wide(c["z"]) if gate else None,
                                  delta_bias=dv(c["bias"]) if bias else None, delta_softplus=softplus, bc_groups=c["groups"],
                                  state=st, state_out=so, state_slots=dv(c["slot"]) if slot else None,
                                  has_state=dv(c["has"]) if has else None, **kw)
    need = qs.qssm_selective_scan_workspace_size(args)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)  # (as fp32: NaN)
    qs.qssm_selective_scan(args, ws)
    torch.cuda.synchronize()
    assert bool((yw[:, D:] == 7.0).all()), "columns behind the row were written"
    if state and not in_place:
        assert torch.equal(st, dv(c["state"])), "the state read was written"
    return yw[:, :D].cpu(), None if so is None else so.cpu().numpy(), need


def assert_near(g, want, e, f16):
    """fp16 adds half a step or half the least denormal, and is an infinity from 65520 on (its largest number is 65504 in
    steps of 32: what the bound lets reach 65520 may be either). Where the bound is infinite, fp32's range is left."""
    fine = np.isfinite(e) & np.isfinite(want)
    if f16:
        e = e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25
        with np.errstate(invalid="ignore"):
            fine &= ~((np.abs(want) + e >= 65520) & (g == np.copysign(np.inf, want)))
    with np.errstate(invalid="ignore"):
        bad = fine & ~(np.abs(g - want) <= e)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], e[bad][:4])


def check(dev, c, yt, gate=True, softplus=True, state=True, slot=True, has=True, bias=True, skip=True, in_place=True, **kw):
    import torch
    y, so, need = run(dev, c, yt, gate, softplus, in_place=in_place, state=state, slot=slot, has=has, bias=bias, skip=skip, **kw)
    T, D = c["x"].shape
    N = c["A"].shape[1]
    off = op.equal_offsets(T, c["nseq"]) if isinstance(c["off"], int) else c["off"]
    slots = c["slot"] if slot else None
    init = op.initial_states(c["state"] if state else None, c["nseq"], (D, N), slots, c["has"] if has else None)
    # a piece has at most as many rows as the call
    with np.errstate(over="ignore", invalid="ignore"):
        want, ey, final, ef = op.selective_scan(c["x"], c["delta"], c["A"], c["B"], c["C"], c["D"] if skip else None,
                                                c["z"] if gate else None, c["bias"] if bias else None, softplus, c["groups"],
                                                off, init, cut=T if need else 0)
    inside = np.zeros(T, bool)
    inside[off[0]:off[-1]] = True
    g = y.double().numpy()
    assert_near(g[inside], want[inside], ey[inside], yt == torch.float16)
    assert np.all(g[~inside] == 7.0), "rows of no sequence were written"
    if state:
        f16 = c["state"].dtype == np.float16
        written = []
        for i, (f, b) in enumerate(zip(final, ef)):
            k = i if slots is None else int(slots[i])
            if 0 <= k < len(so):
                written.append(k)
                assert_near(so[k].astype(np.float64), f, b, f16)
        keep = np.setdiff1d(np.arange(len(so)), written)
        assert np.array_equal(so[keep], c["state"][keep] if in_place else np.full_like(so[keep], 3.0))
    return need


SHAPES = [(1, 1, 1, 1, 1), (1, 64, 16, 1, 1), (5, 70, 16, 1, 5), (40, 128, 16, 2, 40), (17, 96, 64, 1, 17), (60, 100, 24, 2, 3),
          (33, 64, 16, 1, 1), (200, 65, 16, 1, "ragged"), (300, 192, 8, 3, "ragged"), (200, 40, 5, 1, "short"), (150, 130, 16, 1, "short"),
          (120, 66, 64, 2, "ragged"), (200, 64, 16, 1, "hole"), (100, 48, 32, 1, "ragged"), (97, 64, 33, 1, 1), (9, 8, 16, 1, [0, 0, 0, 9, 9]),
          (160, 64, 16, 1, [0, 31, 32, 33, 64, 65, 129, 160])]


@pytest.mark.parametrize("T,D,N,groups,kind", SHAPES)
def test_against_oracle(dev, T, D, N, groups, kind):
    import torch
    i = SHAPES.index((T, D, N, groups, kind))
    print(f"\n[selective_scan T={T} D={D} N={N} G={groups} {kind}]", flush=True)
    off = offsets_of(kind, T, np.random.default_rng(i))
    f16, f32 = np.float16, np.float32
    check(dev, case(10 * i, T, D, N, groups, f16, off), torch.float16)
    check(dev, case(10 * i + 1, T, D, N, groups, f32, off, st=f16), torch.float32, pad=3, in_place=False)
    check(dev, case(10 * i + 2, T, D, N, groups, f32, off), torch.float16, gate=False, softplus=False, bias=False, has=False)
    check(dev, case(10 * i + 3, T, D, N, groups, f16, off, slow=True), torch.float32, slot=False, skip=False, pad=8)
    check(dev, case(10 * i + 4, T, D, N, groups, f16, off, slow=True), torch.float32, state=False)


@pytest.mark.parametrize("T,D,N,kind", [(3000, 64, 16, 1), (2500, 128, 16, "ragged"), (2049, 20, 8, 1), (1500, 64, 64, "ragged"), (2600, 64, 16, 2),
                                        (4000, 16, 4, [0, 1, 3000, 3064, 4000]), (2800, 70, 16, [7, 2790])])
def test_long_sequences_are_cut(dev, T, D, N, kind):
    """Sequences of many pieces, with decays that carry a state over all of them."""
    import torch
    print(f"\n[selective_scan cut T={T} D={D} N={N} {kind}]", flush=True)
    off = offsets_of(kind, T, np.random.default_rng(T))
    c = case(500 + T, T, D, N, 1, np.float16, off, slow=True)
    assert check(dev, c, torch.float32) > 0
    assert check(dev, case(501 + T, T, D, N, 1, np.float32, off), torch.float16, in_place=False, pad=5) > 0


@pytest.mark.parametrize("T,N,begin", [(400, 16, 0), (400, 16, 3), (700, 5, 0), (500, 64, 1)])
def test_pieces_over_which_states_grow(dev, T, N, begin):
    """Steps below zero whose decay over a piece leaves fp32's range, on states of zero and on small ones, which row by row stay
    finite. Steps and their sums are exact, so the bound of single steps holds for their sum's exponential too."""
    import torch
    print(f"\n[selective_scan growing T={T} N={N} begin={begin}]", flush=True)
    off = 1 if begin == 0 else np.array([0, begin, T], np.int32)
    c = case(600 + T, T, 64, N, 1, np.float32, off)
    c["A"][:, :] = -1.0
    c["delta"][:] = 0.25
    c["has"][:] = 1
    c["slot"][:] = np.arange(c["nseq"])
    c["delta"][:, :16] = -2.0  # zero up to the last rows
    c["x"][:T - 10, :16] = 0.0
    c["state"][:, :16] = 0.0
    c["delta"][:, 16:32] = 0.0  # small, and e^96 over the second piece
    c["delta"][begin + 64:begin + 128, 16:32] = -1.5
    c["x"][:begin + 128, 16:32] = 0.0
    c["state"][:, 16:32] = 1e-37
    for gate in (True, False):
        y, so, need = run(dev, c, torch.float32, gate=gate, softplus=False, bias=False)
        assert need > 0 and bool(torch.isfinite(y).all()) and np.all(np.isfinite(so))
        check(dev, c, torch.float32, gate=gate, softplus=False, bias=False)


def test_channels_beside_growing_ones_keep_their_bits(dev):
    import torch
    c = case(620, 400, 64, 16, 1, np.float32, np.array([0, 3, 400], np.int32))
    c["A"][:, :] = -1.0
    c["delta"][:] = 0.25
    out = []
    for grows in (False, True):
        if grows:
            c["delta"][:, ::4] = -2.0
        y, so, need = run(dev, c, torch.float32, softplus=False, bias=False, slot=False)
        assert need > 0
        keep = np.arange(64) % 4 != 0
        out.append((y.numpy()[:, keep], so[:, keep]))
    assert np.array_equal(out[0][0], out[1][0]) and np.array_equal(out[0][1], out[1][1])


def test_no_tokens_hands_the_states_on(dev):
    import torch
    for off in (3, np.zeros(4, np.int32)):
        c = case(3, 0, 40, 16, 1, np.float32, off)
        check(dev, c, torch.float32, in_place=False)
        check(dev, c, torch.float32, in_place=True)


@pytest.mark.parametrize("T", [1, 70])
def test_values_at_the_borders(dev, T):
    """Infinite decays, steps of zero, infinite and NaN inputs in rows of one sequence do not reach another."""
    import torch
    off = 1 if T == 1 else np.array([0, 33, 70], np.int32)
    c = case(40, T, 64, 16, 1, np.float32, off)
    c["A"][:, 0] = -np.inf
    c["A"][:, 1] = -3e38
    c["A"][:, 2] = 0.0
    c["delta"][:, 5] = -np.inf   # softplus 0
    c["delta"][:, 6] = 200.0     # softplus the value
    c["delta"][:, 7] = -200.0
    if T > 1:
        c["B"][33:] = np.nan
        c["x"][33:] = np.inf
        c["z"][40:] = -np.inf
    c["z"][0, 8:12] = [-300, 300, -np.inf, np.inf]
    y, so, _ = run(dev, c, torch.float32, slot=False)
    n = 1 if T == 1 else 33
    A = np.where(np.isinf(c["A"]), np.float32(-3.4e38), c["A"])
    init = op.initial_states(c["state"], 1, (64, 16), None, c["has"][:1])
    with np.errstate(all="ignore"):
        want, ey, final, ef = op.selective_scan(c["x"][:n], np.maximum(c["delta"][:n], -1e30), A, c["B"][:n], c["C"][:n], c["D"], c["z"][:n],
                                                c["bias"], True, 1, [0, n], init)
    fine = np.isfinite(want) & np.isfinite(ey)
    g = y[:n].double().numpy()
    assert np.all(np.abs(g - want)[fine] <= ey[fine]) and fine.mean() > 0.9
    assert np.array_equal(np.isnan(g), np.isnan(want)) and np.array_equal(np.isinf(g), np.isinf(want))
    b = np.where(np.isfinite(ef[0]), ef[0], np.inf)
    assert np.all(np.isfinite(so[0])) and np.all(np.abs(so[0] - final[0]) <= b)
    if T > 1:
        assert np.all(np.isnan(so[1]))


def test_offsets_that_are_wrong_stay_inside(dev):
    import torch
    for off in ([-50, 10, 1000], [30, 20, 10], [5, 100, 3, 90], [2 ** 31 - 1, -2 ** 31, 7], [0, 0, -1, 2 ** 30]):
        c = case(72, 64, 72, 16, 1, np.float16, np.array(off, np.int32))
        y, so, _ = run(dev, c, torch.float16, pad=8)
        keep = np.setdiff1d(np.arange(len(so)), c["slot"])
        assert np.array_equal(so[keep], c["state"][keep])


def test_prompt_then_tokens(dev):
    """A prompt's state goes on token by token: with an fp32 cache the outputs are those of the whole prompt, within both bounds."""
    import torch
    c = case(90, 3 * 24, 64, 16, 1, np.float16, 3)
    whole, so, _ = run(dev, c, torch.float32, slot=False, has=False)
    part = lambda k, lo, hi: c[k].reshape(3, 24, -1)[:, lo:hi].reshape(3 * (hi - lo), -1)  # noqa: E731
    state, got = c["state"], []
    for lo, hi in [(0, 20)] + [(t, t + 1) for t in range(20, 24)]:
        cc = dict(c, off=3, state=state, **{k: part(k, lo, hi) for k in ("x", "delta", "z", "B", "C")})
        y, state, _ = run(dev, cc, torch.float32, slot=False, has=False)
        got.append(y.view(3, hi - lo, 64))
    init = op.initial_states(c["state"], 3, (64, 16), None, None)
    want, ey, _, _ = op.selective_scan(c["x"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"], c["bias"], True, 1,
                                       op.equal_offsets(72, 3), init)
    for g in (whole, torch.cat(got, 1).view(72, 64)):
        assert np.all(np.abs(g.double().numpy() - want) <= ey)
