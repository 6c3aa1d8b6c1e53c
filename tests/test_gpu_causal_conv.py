"""GPU parity of the causal convolution over packed sequences against the fp64 oracle: int8 codes and states bit for
bit, fp32 and fp16 outputs within the roundings counted in bound()."""
import numpy as np
import pytest

import oracle.packed as op

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def bound(y, v, s, W, use_silu, f16):
    """The sum: W fused multiply-adds of eps of at most s each, passed on by silu at most 1.1 times; silu: the
    exponent's rounding |v| eps, exponential and reciprocal 2 eps each, and four products and sums, under (8 + |v|) 2 eps
    of y; fp16: half a step, or half the least denormal."""
    e = W * EPS * s * (1.1 if use_silu else 1.0)
    if use_silu:
        e = e + (8.0 + np.abs(v)) * 2 * EPS * np.abs(y)
    if f16:
        e = e + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
    return 1.01 * e + 1e-37


def offsets_of(kind, T, r):
    """[nseq + 1] offsets: equal lengths as a number, or ragged ones with empty sequences and rows of none."""
    if isinstance(kind, int):
        return kind
    if kind == "ragged":
        return np.sort(np.concatenate([[0, T], r.integers(0, T + 1, 5)])).astype(np.int32)
    if kind == "short":  # many sequences of 0 to 4 rows
        return np.concatenate([[0], np.minimum(np.cumsum(r.integers(0, 5, T // 2 + 1)), T)]).astype(np.int32)
    if kind == "hole":  # rows before the first and behind the last sequence
        return np.array([5, 5, 40, 41, 41, T - 9], np.int32)
    return np.array(kind, np.int32)


def case(seed, T, C, W, xt, off, bias=True):
    r = np.random.default_rng([51, seed])
    x = (r.standard_normal((T, C)) * np.exp(0.4 * r.standard_normal(C))).astype(xt)
    w = (r.uniform(-1, 1, (C, W))).astype(np.float32)
    b = r.standard_normal(C).astype(np.float32) if bias else None
    nseq = off if isinstance(off, int) else len(off) - 1
    slots = nseq + 3
    state = r.standard_normal((slots, W - 1, C)).astype(xt)
    slot = r.permutation(slots)[:nseq].astype(np.int32)
    if nseq > 2:
        slot[1] = -1
        slot[2] = slots + 7
    has = r.integers(0, 2, nseq).astype(np.uint8)
    gof = r.integers(0, 5, C).astype(np.uint8)
    sc = np.array([0.02, 0.004, 0.1, 0.0, 0.5], np.float32)  # an invalid one among them
    return dict(x=x, w=w, b=b, off=off, nseq=nseq, state=state, slot=slot, has=has, gof=gof, sc=sc)


def run(dev, c, yt, use_silu=True, pads=(0, 0), in_place=True, shift=0, state=True, slot=True, has=True):
    """Runs the library on columns of wider tensors; returns y, the state written, and the rest of both."""
    import torch
    import quantized_state_space_amd as qs
    T, C = c["x"].shape
    dv = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    xw = torch.full((T, C + pads[0] + shift), 77.0, device=dev).to(dv(c["x"]).dtype)
    xw[:, shift:shift + C] = dv(c["x"])
    fill = 99 if yt == torch.int8 else 7.0
    yw = torch.full((T, C + pads[1] + shift), fill, dtype=yt, device=dev)
    y = yw[:, shift:shift + C]
    st = dv(c["state"]) if state else None
    so = st if in_place else (torch.full_like(st, 3.0) if state else None)
    kw = dict(nseq=c["off"]) if isinstance(c["off"], int) else dict(seq_offsets=dv(c["off"]))
    args = qs.causal_conv_args(xw[:, shift:shift + C], dv(c["w"]), y, bias=dv(c["b"]), silu=use_silu, state=st, state_out=so,
                               state_slots=dv(c["slot"]) if slot else None, has_state=dv(c["has"]) if has else None,
                               y_group_of=dv(c["gof"]), y_scales=dv(c["sc"]), **kw)
    qs.qssm_causal_conv(args)
    torch.cuda.synchronize()
    if shift:
        assert bool((yw[:, :shift] == fill).all())
    if pads[1]:
        assert bool((yw[:, shift + C:] == fill).all()), "columns behind the row were written"
    if state and not in_place:
        assert torch.equal(st, dv(c["state"])), "the state read was written"
    return y.cpu(), None if so is None else so.cpu().numpy(), args


def check(dev, c, yt, use_silu=True, state=True, slot=True, has=True, in_place=True, **kw):
    import torch
    y, so, _ = run(dev, c, yt, use_silu, state=state, slot=slot, has=has, in_place=in_place, **kw)
    T, C = c["x"].shape
    W = c["w"].shape[1]
    off = op.equal_offsets(T, c["nseq"]) if isinstance(c["off"], int) else c["off"]
    slots = c["slot"] if slot else None
    init = op.initial_states(c["state"] if state else None, c["nseq"], (W - 1, C), slots, c["has"] if has else None)
    want, v, s, final = op.causal_conv(c["x"], c["w"], c["b"], use_silu, off, init)
    inside = np.zeros(T, bool)
    inside[off[0]:off[-1]] = True
    if yt == torch.int8:
        sc = np.where(c["sc"] == 0, 0, c["sc"])[c["gof"]]
        codes = op.conv_codes(want, sc)
        assert np.array_equal(y.numpy()[inside], codes[inside])
        assert np.all(y.numpy()[~inside] == 99), "rows of no sequence were written"
    else:
        g = y.double().numpy()
        e = np.abs(g - want)[inside]
        lim = bound(want, v, s, W, use_silu, yt == torch.float16)[inside]
        assert np.all(e <= lim), (e.max(), np.argwhere(~(e <= lim))[:4])
        assert np.all(g[~inside] == 7.0), "rows of no sequence were written"
    if state:
        base = c["state"] if in_place else np.full_like(c["state"], 3.0)
        assert np.array_equal(so, op.store_states(base, final, slots))


# tokens, channels, width, sequences
SHAPES = [(1, 1, 4, 1), (1, 64, 4, 1), (7, 8, 2, 7), (256, 72, 4, 256), (33, 1543, 3, 33), (100, 40, 4, 4), (300, 512, 4, "ragged"),
          (300, 33, 3, "ragged"), (517, 520, 2, "short"), (400, 104, 4, "short"), (400, 7, 4, "short"), (200, 24, 4, "hole"),
          (1000, 1024, 4, 1), (2048, 64, 3, "ragged"), (3000, 1536, 4, "ragged"), (64, 16, 4, [0, 61, 64]), (130, 16, 4, [0, 62, 63, 64, 65, 66, 128, 130]),
          (9, 8, 4, [0, 0, 0, 9, 9]), (70, 200, 4, [0, 8, 15, 16, 17, 24, 31, 33, 41, 70])]


@pytest.mark.parametrize("T,C,W,kind", SHAPES)
def test_against_oracle(dev, T, C, W, kind):
    import torch
    i = SHAPES.index((T, C, W, kind))
    print(f"\n[causal_conv T={T} C={C} W={W} {kind}]", flush=True)
    off = offsets_of(kind, T, np.random.default_rng(i))
    for j, (xt, yt) in enumerate([(np.float16, torch.float16), (np.float32, torch.float32), (np.float16, torch.int8),
                                  (np.float32, torch.int8), (np.float16, torch.float32), (np.float32, torch.float16)]):
        c = case(10 * i + j, T, C, W, xt, off, bias=j != 1)
        check(dev, c, yt, use_silu=j != 4, in_place=j % 2 == 0, pads=((0, 0), (3, 5), (8, 16))[j % 3], shift=j % 3,
              has=j != 3, slot=j != 5)
    check(dev, c, torch.float32, state=False)


def test_long_packed_batch(dev):
    """More strips than fit the chip at once, sequences across their borders, and many empty ones."""
    import torch
    r = np.random.default_rng(8)
    off = np.sort(np.concatenate([[0, 9000], r.integers(0, 9001, 60), np.full(70, 4000), [8999] * 9])).astype(np.int32)
    c = case(900, 9000, 256, 4, np.float16, off)
    check(dev, c, torch.int8)
    check(dev, c, torch.float16, in_place=False, pads=(64, 0))


def test_no_tokens_hands_the_states_on(dev):
    import torch
    for off in (3, np.zeros(4, np.int32)):
        c = case(3, 0, 40, 4, np.float32, off)
        check(dev, c, torch.float32, in_place=False)
        check(dev, c, torch.float32, in_place=True)


@pytest.mark.parametrize("xt", [np.float16, np.float32])
@pytest.mark.parametrize("T", [1, 12])
def test_values_at_the_borders(dev, xt, T):
    """NaN, infinities, the largest values, gates far below zero, and sums that sit on a rounding border of the codes."""
    import torch
    c = case(70, T, 64, 4, xt, 1)
    x = c["x"]
    x[0, :8] = [np.nan, np.inf, -np.inf, 0, np.finfo(xt).max, -np.finfo(xt).max, 30, -30]
    x[T // 2, 8:16] = [np.nan, np.inf, -np.inf, -0.0, 1e-7, -1e-7, -120, 120]
    # bias + w x = (k + 1/2) s exactly, without silu
    c["w"][16:64] = [0, 0, 0, 1]
    c["b"][16:64] = 0
    c["gof"][:] = 0
    c["sc"][0] = 0.25
    x[:, 16:64] = (np.arange(48) - 24 + 0.5) * 0.25
    y, so, _ = run(dev, c, torch.int8, use_silu=False)
    init = op.initial_states(c["state"], 1, (3, 64), c["slot"], c["has"])
    for use_silu in (False, True):
        y, so, _ = run(dev, c, torch.int8, use_silu=use_silu)
        with np.errstate(invalid="ignore", over="ignore"):
            want, _, _, final = op.causal_conv(x, c["w"], c["b"], use_silu, [0, T], init)
            assert np.array_equal(y.numpy(), op.conv_codes(want, c["sc"][c["gof"]]))
        assert np.array_equal(so, op.store_states(c["state"], final, c["slot"]), equal_nan=True)
        y, _, _ = run(dev, c, torch.float32, use_silu=use_silu)
        assert np.array_equal(np.isnan(y.numpy()), np.isnan(want)) and np.array_equal(np.isinf(y.numpy()), np.isinf(f32(want)))


def f32(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return v.astype(np.float32)


def test_codes_near_rounding_borders(dev):
    """Millions of codes, a part of which the fp32 values leave open (sums that nearly cancel, small scales)."""
    import torch
    c = case(71, 2000, 512, 4, np.float32, 1)
    c["x"][:, ::2] *= 1000
    c["w"][::2, 1] = -c["w"][::2, 0]
    c["x"][1:, ::2] = c["x"][:-1, ::2] * np.float32(1 + 2.0 ** -12)
    c["sc"][:] = [1e-3, 1e-2, 0.1, 1.0, 3e-5]
    check(dev, c, torch.int8)
    check(dev, c, torch.int8, use_silu=False)


def test_offsets_that_are_wrong_stay_inside(dev):
    """Offsets outside the rows or out of order: which rows they name is undefined, but nothing else is touched."""
    import torch
    for off in ([-50, 10, 1000], [30, 20, 10], [5, 100, 3, 90], [2 ** 31 - 1, -2 ** 31, 7], [0, 0, -1, 2 ** 30]):
        c = case(72, 64, 72, 4, np.float16, np.array(off, np.int32))
        y, so, _ = run(dev, c, torch.float16, pads=(0, 8))
        keep = np.setdiff1d(np.arange(len(so)), c["slot"])
        assert np.array_equal(so[keep], c["state"][keep])


@pytest.mark.parametrize("off", [[2, 1, 60], [1, 0, 60], [1, 0, 2, 60], [2, 1, 1, 0, 64]])
def test_offsets_out_of_order_read_no_row_before_the_first(dev, off):
    """A sequence whose offset is above the next one's: the next one's rows begin behind its first, and what they need of
    rows before that lies before row 0."""
    import torch
    import quantized_state_space_amd as qs
    print(f"\n[causal_conv offsets {off}]", flush=True)
    for W in (2, 3, 4):
        wide = torch.full((67, 72), float("nan"), dtype=torch.float16, device=dev)
        wide[3:] = torch.randn(64, 72, device=dev).half()
        y = torch.full((64, 72), 7.0, device=dev)
        qs.qssm_causal_conv(qs.causal_conv_args(wide[3:], torch.randn(72, W, device=dev), y,
                                                seq_offsets=torch.tensor(off, dtype=torch.int32, device=dev)))
        torch.cuda.synchronize()
        assert bool(torch.isfinite(y).all()), W


def test_prompt_then_tokens_equals_the_prompt(dev):
    """A prompt cut anywhere, its rest token by token: the same outputs bit for bit."""
    import torch
    import quantized_state_space_amd as qs
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.standard_normal((3 * 20, 96)).astype(np.float16)).to(dev)
    w = torch.from_numpy(r.standard_normal((96, 4)).astype(np.float32)).to(dev)
    whole = torch.empty(60, 96, device=dev)
    qs.qssm_causal_conv(qs.causal_conv_args(x, w, whole, nseq=3))
    for cut in (0, 1, 2, 3, 11):
        st = torch.zeros(3, 3, 96, dtype=torch.float16, device=dev)
        head = x.view(3, 20, 96)[:, :cut].reshape(-1, 96).contiguous()
        yh = torch.empty(3 * cut, 96, device=dev)
        qs.qssm_causal_conv(qs.causal_conv_args(head, w, yh, nseq=3, state=None, state_out=st))
        outs = [yh.view(3, cut, 96)]
        for t in range(cut, 20):
            xt = x.view(3, 20, 96)[:, t].contiguous()
            y = torch.empty(3, 96, device=dev)
            qs.qssm_causal_conv(qs.causal_conv_args(xt, w, y, nseq=3, state=st, state_out=st))
            outs.append(y.view(3, 1, 96))
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(outs, 1).view(60, 96), whole), cut
