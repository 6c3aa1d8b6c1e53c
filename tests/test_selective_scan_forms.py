"""The forms of the selective scan: on the CPU, the rows of a piece and the form of single rows for named calls, that the
workspace's slots of all cut sequences are apart and inside, and its size; on the GPU, these calls against the oracle, and that
nothing behind the workspace is written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import quantized_state_space_amd as qs
from tests.test_capi_packed import scan_args

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OFF = 11 << 32  # an address that a size alone does not read


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("forms") / "forms.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-std=c++17", os.path.join(ROOT, "tests", "host_selective_scan_forms.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    i64 = ctypes.c_int64
    for f, args in ((lib.host_piece, [i64] * 3 + [ctypes.c_int]), (lib.host_first_slot, [ctypes.c_int] * 2), (lib.host_slots, [i64] * 3),
                    (lib.host_most, [i64] * 2), (lib.host_four, [i64] * 2 + [ctypes.c_int])):
        f.argtypes, f.restype = args, i64
    return lib


# rows of a piece, tokens, channels, states, sequences: a number of equal ones, or packed ones by their kind
PIECES = [(64, 3000, 64, 16, 1), (96, 6000, 1536, 16, "ragged"), (128, 8192, 1536, 16, 1), (128, 8190, 1500, 24, "ragged"), (192, 8192, 2304, 16, 1),
          (256, 16384, 4096, 16, "ragged"), (256, 12000, 4100, 8, 3)]
# four sequences a lane, sequences, channels, states, B/C groups
SINGLE = [(1, 256, 256, 16, 1), (1, 257, 256, 16, 2), (1, 258, 256, 5, 1), (1, 259, 250, 24, 2), (1, 260, 256, 32, 1), (1, 1030, 70, 16, 1), (1, 1029, 66, 8, 2),
          (0, 252, 256, 16, 1), (0, 300, 256, 33, 1), (0, 600, 70, 64, 2)]


def waves(D, groups=1):
    return 4 * groups * -(-(D // groups) // 64)


def npl(N):
    return 2 if N <= 8 else 4 if N <= 16 else 8 if N <= 32 else 16


@pytest.mark.parametrize("rows,T,D,N,kind", PIECES)
def test_piece(forms, rows, T, D, N, kind):
    assert forms.host_piece(T, 24 if kind == "ragged" else kind, waves(D), kind == "ragged") == rows


@pytest.mark.parametrize("four,nseq,D,N,groups", SINGLE)
def test_single_rows(forms, four, nseq, D, N, groups):
    assert forms.host_four(nseq, waves(D, groups) // 4, npl(N)) == four


def test_equal_sequences_that_fill_the_chip_run_whole(forms):
    assert forms.host_piece(16 * 1024, 16, waves(4096), 0) == 16 * 1024 and forms.host_piece(8 * 1024, 8, waves(1536), 0) == 128


@pytest.mark.parametrize("ordered", [True, False])
def test_slots_of_cut_sequences(forms, ordered):
    r = np.random.default_rng(5 + ordered)
    for _ in range(2000):
        T, nseq, piece = int(np.exp(r.uniform(0, 9))), int(np.exp(r.uniform(0, 6))), int(r.choice([3, 64, 96, 256]))
        off = r.integers(0, T + 1, nseq + 1)
        if ordered:
            off.sort()
        used, most = [], forms.host_slots(T, nseq, piece)
        for i in range(nseq):
            lo, hi = int(off[i]), max(int(off[i]), int(off[i + 1]))
            pieces = -(-(hi - lo) // piece)
            if pieces > 1:
                at = forms.host_first_slot(i, lo // piece)
                assert 0 <= at and at + pieces <= most, (T, nseq, piece, i)
                used += range(at, at + pieces)
        if ordered:
            assert len(set(used)) == len(used)
        assert most <= 2 * (T // piece)


def size(tokens, nseq, dim=4096, dstate=16, packed=True, groups=1):
    a = scan_args(tokens=tokens, nseq=nseq, dim=dim, dstate=dstate, ngroups=groups, seq_offsets=OFF if packed else None, slots=nseq)
    return qs.load().qssm_selective_scan_workspace_size(ctypes.byref(a))


def test_workspace_does_not_grow_with_sequences_that_are_not_cut():
    """16384 rows of 4096 channels, in pieces of 256: 64 slots for one sequence behind the last, two for each 256 rows at most."""
    slot = 4096 * (16 + 1) * 4
    assert size(16384, 1) == 65 * slot
    assert size(16384, 24) == 88 * slot
    assert size(16384, 64) == size(16384, 1024) == size(16384, 16384) == size(16384, 1 << 24) == 128 * slot


@pytest.mark.parametrize("dim,dstate,groups", [(1, 1, 1), (200, 16, 1), (1536, 16, 1), (4096, 8, 2), (8192, 64, 1), (5000, 33, 5)])
def test_workspace_bound_covers_every_call(dim, dstate, groups):
    """Of fewer rows too, with and without offsets, and it is one of them where the sequences are many."""
    bound = lambda t: qs.qssm_selective_scan_workspace_bound(t, dim, dstate, groups)  # noqa: E731
    most, last = 0, 0
    for t in [*range(1, 1500), *range(1500, 40000, 37)]:
        for nseq, packed in ((1, True), (t, True), (1, False), (2, False), (3, False)):
            if packed or t % nseq == 0:
                most = max(most, size(t, nseq, dim, dstate, packed, groups))
        assert last <= bound(t) and most <= bound(t)
        last = bound(t)
    assert bound(39000) <= most * 1.1
    assert bound(0) == 0 and bound(-1) == 0
    assert qs.qssm_selective_scan_workspace_bound(100, 64, 65) == 0 and qs.qssm_selective_scan_workspace_bound(100, 64, 16, 0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,kind", [(1500, 64, "one"), (3000, 40, "short"), (1400, 70, "mixed"), (700, 64, "wrong")])
def test_nothing_behind_the_workspace_is_written(dev, T, D, kind):
    import torch
    print(f"\n[selective_scan workspace T={T} D={D} {kind}]", flush=True)
    r = np.random.default_rng(T)
    off = {"one": [0, T], "short": np.minimum(np.arange(T + 2) * 3, T), "wrong": [600, 0, 700, 20, 690, -5, 10 ** 6],
           "mixed": np.sort(np.concatenate([[0, T, T], r.integers(0, T, 40), [5] * 30, [200, 700]]))}[kind]
    off = torch.tensor(np.asarray(off, np.int32), device=dev)
    n = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
    args = qs.selective_scan_args(n(T, D), n(T, D), -torch.rand(D, 16, device=dev), n(T, 16), n(T, 16), n(T, D), seq_offsets=off)
    need = qs.qssm_selective_scan_workspace_size(args)
    assert need > 0
    ws = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device=dev)
    qs.qssm_selective_scan(args, ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all())


@pytest.mark.gpu
@pytest.mark.parametrize("four,nseq,D,N,groups", SINGLE)
def test_single_rows_against_oracle(dev, four, nseq, D, N, groups):
    import torch
    from tests.test_gpu_selective_scan import case, check
    print(f"\n[selective_scan single rows nseq={nseq} D={D} N={N} G={groups}]", flush=True)
    f16, f32 = np.float16, np.float32
    i = SINGLE.index((four, nseq, D, N, groups))
    for j, (xt, st, yt) in enumerate([(f16, f32, torch.float16), (f32, f16, torch.float32), (f16, f16, torch.float32)]):
        c = case(700 + 10 * i + j, nseq, D, N, groups, xt, nseq, st=st)
        c["slot"][[5, 11, nseq - 1]] = -1, len(c["state"]), 2 ** 31 - 1  # no slot, in every place of the four
        check(dev, c, yt, in_place=j != 1, pad=(0, 3, 8)[j], gate=j != 2, softplus=j != 2, bias=j != 2)
        if j == 0:
            check(dev, c, yt, slot=False, has=False, skip=False)


@pytest.mark.gpu
@pytest.mark.parametrize("xt", ["float16", "float32"])
@pytest.mark.parametrize("rows,T,D,N,kind", PIECES)
def test_pieces_against_oracle(dev, rows, T, D, N, kind, xt):
    """The oracle computes some of the channels, the first and last and those on both sides of a workgroup's."""
    import torch
    import oracle.packed as op
    from tests.test_gpu_selective_scan import assert_near
    print(f"\n[selective_scan pieces of {rows} T={T} D={D} N={N} {kind} {xt}]", flush=True)
    r = np.random.default_rng([56, T, D])
    g = torch.Generator(device=dev).manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if kind == "ragged":
        off = np.concatenate([[2], np.sort(r.integers(2, T - 3, 19)), [T - 700, T - 700, T - 699, T - 3]]).astype(np.int32)
        off.sort()
        where, nseq = dict(seq_offsets=torch.from_numpy(off).to(dev)), len(off) - 1
    else:
        off, where, nseq = op.equal_offsets(T, kind), dict(nseq=kind), kind
    xt = getattr(torch, xt)
    x, delta, z, B, C = n(T, D).to(xt), (0.5 * n(T, D)).to(xt), n(T, D).to(xt), n(T, N).to(xt), n(T, N).to(xt)
    A = -0.1 * torch.rand(D, N, generator=g, device=dev) * torch.arange(1, N + 1, device=dev)
    skip, bias = n(D), -3 + n(D)
    state = n(nseq + 2, D, N)
    slot = r.permutation(nseq + 2)[:nseq].astype(np.int32)
    has = r.integers(0, 2, nseq).astype(np.uint8)
    has[0] = 1
    y = torch.full((T, D), 7.0, device=dev)
    pick = np.unique(np.concatenate([[0, 1, 63, 64, 127, 128], np.arange(D - 3, D), r.integers(0, D, 4)]) % D)
    at = torch.from_numpy(pick).to(dev)
    before = state[:, at].cpu().numpy()
    dv = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    args = qs.selective_scan_args(x, delta, A, B, C, y, D=skip, z=z, delta_bias=bias, state=state, state_out=state, state_slots=dv(slot),
                                  has_state=dv(has), **where)
    ws = torch.full((qs.qssm_selective_scan_workspace_size(args),), 0xFF, dtype=torch.uint8, device=dev)
    assert ws.numel() > 0
    qs.qssm_selective_scan(args, ws)
    torch.cuda.synchronize()
    h = lambda t: t.cpu().numpy()  # noqa: E731
    init = op.initial_states(before, nseq, (len(pick), N), slot, has)
    want, ey, final, ef = op.selective_scan(h(x[:, at]), h(delta[:, at]), h(A[at]), h(B), h(C), h(skip[at]), h(z[:, at]), h(bias[at]), True, 1,
                                            off, init, cut=rows)
    inside = slice(off[0], off[-1])
    assert_near(h(y[:, at]).astype(np.float64)[inside], want[inside], ey[inside], False)
    assert bool((y[:off[0]] == 7.0).all()) and bool((y[off[-1]:] == 7.0).all()), "rows of no sequence were written"
    got = h(state[:, at])
    for i in range(nseq):
        assert_near(got[slot[i]].astype(np.float64), final[i], ef[i], False)
    keep = np.setdiff1d(np.arange(nseq + 2), slot)
    assert np.array_equal(got[keep], before[keep])
