"""How the selective scan cuts sequences: on the CPU, the rows of a piece for named calls, that the workspace's slots of all cut
sequences are apart and inside, and its size; on the GPU, that nothing behind the workspace is written."""
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
                    (lib.host_most, [i64] * 2)):
        f.argtypes, f.restype = args, i64
    return lib


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
