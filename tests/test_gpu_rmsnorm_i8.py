"""GPU parity of the RMS norm with an int8 output against the oracle: codes and scales are fixed bit for
bit by the operator's definition (fp32 roundings at stated places, sums and silu in fp64, the exact
quantization rule), so they must be equal, and the residual stream too."""
import numpy as np
import pytest

import oracle.w8a8 as ow

pytestmark = pytest.mark.gpu

DT = {"f16": np.float16, "f32": np.float32}


def make(seed, M, D, xt, rt, gt, outliers=True):
    r = np.random.default_rng([91, seed])
    ch = np.exp(r.uniform(-1, 1, D)) * np.where(r.random(D) < 0.02, 30, 1)
    x = (r.standard_normal((M, D)) * (ch if outliers else 1)).astype(DT[xt])
    w = (1 + 0.3 * r.standard_normal(D)).astype(np.float32)
    res = (2 * r.standard_normal((M, D))).astype(DT[rt]) if rt else None
    z = (2 * r.standard_normal((M, D))).astype(DT[gt]) if gt else None
    return x, w, res, z


def to(a, dev, pad=0):
    """Device tensor; with pad the rows lie that much further apart than they are wide."""
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    if not pad:
        return t.to(dev)
    wide = torch.zeros(a.shape[0], a.shape[1] + pad, dtype=t.dtype, device=dev)
    wide[:, :a.shape[1]] = t.to(dev)
    return wide[:, :a.shape[1]]


def run(dev, x, w, res, z, groups=1, static=None, pad=0, eps=1e-5, stream_out=True, inplace=False):
    import torch
    import quantized_state_space_amd as qs
    M, D = x.shape
    buf = torch.full((M, D + pad), -77, dtype=torch.int8, device=dev)
    q = buf[:, :D]
    sc = torch.full((M,), float("nan"), device=dev) if static is None else torch.full((1,), static, device=dev)
    xt, rt, zt = to(x, dev, pad), to(res, dev, pad), to(z, dev, pad)
    ro = None
    if res is not None:
        ro = rt if inplace else (torch.empty_like(rt) if stream_out else None)
    qs.qssm_rmsnorm_i8(qs.rmsnorm_args(xt, q, sc, weight=to(w, dev), eps=eps, residual=rt,
                                       residual_out=ro, gate=zt, norm_groups=groups,
                                       compute_scales=static is None))
    torch.cuda.synchronize()
    if pad:
        assert bool((buf[:, D:] == -77).all()), "columns behind the row were written"
    return q.cpu().numpy(), sc.cpu().numpy(), None if ro is None else ro.cpu().numpy()


def check(dev, x, w, res, z, groups=1, static=None, **kw):
    q, s, h = run(dev, x, w, res, z, groups, static, **kw)
    eps = kw.get("eps", 1e-5)
    oq, os_, oh = ow.rmsnorm_i8(x, w, eps=eps, residual=res, residual_dtype=None if res is None else res.dtype,
                                gate=z, groups=groups, scale=static)
    if static is None:
        assert np.array_equal(s, os_), np.flatnonzero(s != os_)[:5]
    assert np.array_equal(q, oq), (np.argwhere(q != oq)[:5], (q != oq).sum())
    if h is not None:
        assert np.array_equal(h, oh, equal_nan=True)


@pytest.mark.parametrize("M,D,groups,xt,rt,gt,static,pad", [
    (1, 4096, 1, "f16", "f32", None, None, 0),
    (3, 8192, 8, "f16", None, "f16", None, 64),
    (1, 1, 1, "f32", None, None, None, 0),
    (5, 1, 1, "f16", "f16", None, None, 3),
    (7, 64, 1, "f32", "f16", None, None, 0),
    (33, 768, 1, "f16", "f32", None, 0.05, 0),
    (9, 1543, 1, "f32", "f32", None, 0.02, 0),
    (9, 1543, 1, "f32", "f32", None, None, 5),
    (4, 8192, 1, "f32", None, "f32", None, 0),
    (4, 8191, 1, "f16", "f16", None, None, 1),
    (4, 8190, 9, "f32", None, "f16", None, 0),
    (2, 16384, 2, "f16", "f32", None, None, 8),
    (2, 32768, 1, "f32", "f32", None, None, 0),
    (2, 24584, 7, "f16", None, "f32", 0.03, 8),
    (6, 1000, 125, "f16", None, "f16", None, 0),
    (6, 1000, 1000, "f32", None, None, None, 0),
    (11, 520, 1, "f16", None, None, None, 8),
    (300, 2048, 2, "f16", None, "f16", None, 0),
])
def test_against_oracle(dev, M, D, groups, xt, rt, gt, static, pad):
    print(f"\n[rmsnorm M={M} D={D} groups={groups} x={xt} residual={rt} gate={gt} static={static} pad={pad}]", flush=True)
    check(dev, *make(M * 31 + D, M, D, xt, rt, gt), groups=groups, static=static, pad=pad)


@pytest.mark.parametrize("M,D,groups,xt,rt,gt,static,pad", [
    (512, 5001, 1, "f16", None, None, None, 0),
    (515, 8191, 1, "f32", "f32", None, None, 1),
    (513, 2050, 2, "f16", None, "f32", None, 0),
    (600, 2048, 64, "f32", None, "f16", None, 3),
    (700, 130, 1, "f16", "f32", None, 0.05, 0),
    (1000, 1001, 7, "f32", "f16", None, None, 0),
    (520, 8192, 8, "f16", None, "f16", None, 0),
    (520, 4104, 1, "f16", "f32", None, None, 8),
    (530, 24576, 1, "f32", None, "f32", None, 0),
])
def test_many_rows(dev, M, D, groups, xt, rt, gt, static, pad):
    """The launch shapes taken from 512 rows on."""
    print(f"\n[rmsnorm M={M} D={D} groups={groups} x={xt} residual={rt} gate={gt} static={static} pad={pad}]", flush=True)
    check(dev, *make(M * 31 + D, M, D, xt, rt, gt), groups=groups, static=static, pad=pad)


@pytest.mark.parametrize("D,rt", [(1001, "f16"), (1001, "f32"), (1000, "f16")])
def test_columns_behind_the_stream_are_left(dev, D, rt):
    """residual_out as a slice of a wider tensor, whose other columns keep what they hold."""
    print(f"\n[rmsnorm residual_out in a wider tensor D={D} residual={rt}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    x, w, res, _ = make(8, 600, D, "f16", rt, None)
    wide = torch.full((600, 1008), -7.0, dtype=torch.from_numpy(res).dtype, device=dev)
    q, sc = torch.empty(600, D, dtype=torch.int8, device=dev), torch.empty(600, device=dev)
    qs.qssm_rmsnorm_i8(qs.rmsnorm_args(to(x, dev), q, sc, weight=to(w, dev), residual=to(res, dev),
                                       residual_out=wide[:, :D]))
    oq, os_, oh = ow.rmsnorm_i8(x, w, residual=res, residual_dtype=res.dtype)
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sc.cpu().numpy(), os_)
    assert np.array_equal(wide[:, :D].cpu().numpy(), oh)
    assert bool((wide[:, D:] == -7.0).all())


def test_stream_in_place_and_absent(dev):
    print("\n[rmsnorm residual in place, without an output, starting from x, no weight]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    x, w, res, _ = make(5, 17, 768, "f16", "f32", None)
    check(dev, x, w, res, None, inplace=True)
    check(dev, x, w, res, None, stream_out=False)
    check(dev, x, None, res, None)
    q = torch.empty(17, 768, dtype=torch.int8, device=dev)
    sc, ro = torch.empty(17, device=dev), torch.empty(17, 768, dtype=torch.float16, device=dev)
    xt = (torch.from_numpy(x).float() * 1.001).to(dev)
    qs.qssm_rmsnorm_i8(qs.rmsnorm_args(xt, q, sc, weight=to(w, dev), residual_out=ro))
    oq, os_, oh = ow.rmsnorm_i8(xt.cpu().numpy(), w, residual_dtype=np.float16)
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sc.cpu().numpy(), os_)
    assert np.array_equal(ro.cpu().numpy(), oh)


@pytest.mark.parametrize("D,groups", [(64, 1), (64, 4), (63, 3)])
def test_special_rows(dev, D, groups):
    """Zero rows, NaN and infinities (their group's codes are 0, its others stay), fp16 overflow of the
    stream, denormals, huge and tiny fp32 values, exact ties; eps 0; weights that are 0, NaN, Inf."""
    print(f"\n[rmsnorm special rows D={D} groups={groups}]", flush=True)
    x, w, _, _ = make(6, 12, D, "f32", None, None)
    x[0] = 0
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, D - 1] = -np.inf
    x[4] *= np.float32(1e-30)
    x[5] *= np.float32(1e36)
    x[6] = np.float32(1e-45)
    x[7] = np.arange(D) % 3 - 1  # equal magnitudes
    x[8, 0], x[8, 1:] = 2, 1    # v / s = 63.5 exactly after the common factor
    x[9] = np.float32(3e38)
    for ww in (w, None):
        check(dev, x, ww, None, None, groups=groups)
        check(dev, x, ww, None, None, groups=groups, static=0.01)
        check(dev, x[4:], ww, None, None, groups=groups, eps=0.0)
    for bad in (np.nan, np.inf, 0.0):
        wb = w.copy()
        wb[2] = bad
        check(dev, x, wb, None, None, groups=groups)
    for s in (np.inf, np.nan, 0.0, 2.0 ** -101, 1e-3):  # invalid static scales give codes 0
        check(dev, x, w, None, None, groups=groups, static=float(s))
    big = np.full((2, D), 60000, np.float16)
    check(dev, big, w, big, None, groups=groups)  # the fp16 stream overflows to Inf
    z = np.tile(np.float32([0, -0.0, 1e-40, 88, -88, 104, -104, 800, -800, 3e38, -3e38, 1, -1, 0.5, 20, -20]), 64)
    check(dev, np.ones((2, D), np.float32), w, None, np.stack([z[:D], z[D:2 * D]]), groups=groups)
    z = z[:D].copy()
    z[1], z[7], z[D - 2] = np.nan, np.inf, -np.inf
    check(dev, np.ones((1, D), np.float32), w, None, z[None], groups=groups)


def test_another_stream_and_replay(dev):
    """On a side stream, and captured once and replayed on new inputs with eager work between, bit for bit."""
    print("\n[rmsnorm side stream, graph]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    x, w, res, _ = make(8, 40, 1024, "f16", "f32", None)
    xt, wt, rt = to(x, dev), to(w, dev), to(res, dev)
    q, sc, ro = torch.empty(40, 1024, dtype=torch.int8, device=dev), torch.empty(40, device=dev), torch.empty_like(rt)
    args = qs.rmsnorm_args(xt, q, sc, weight=wt, residual=rt, residual_out=ro)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qs.qssm_rmsnorm_i8(args, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.qssm_rmsnorm_i8(args)
    for k in range(3):
        xk = (x * np.float16(1 + k)).astype(np.float16)
        xt.copy_(torch.from_numpy(xk))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        oq, os_, oh = ow.rmsnorm_i8(xk, w, residual=res, residual_dtype=np.float32)
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sc.cpu().numpy(), os_), k
        assert np.array_equal(ro.cpu().numpy(), oh), k


def test_more_rows_than_a_grid_dimension(dev):
    """2^21 + 3 rows: the grid's second dimension (a dimension holds fewer than 2^32 threads)."""
    print("\n[rmsnorm 2^21 + 3 rows]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    M, D = 2 ** 21 + 3, 8
    x = torch.randn(M, D, device=dev)
    q, sc = torch.full((M, D), -77, dtype=torch.int8, device=dev), torch.full((M,), float("nan"), device=dev)
    qs.qssm_rmsnorm_i8(qs.rmsnorm_args(x, q, sc))
    rows = torch.cat([torch.arange(5), torch.arange(M // 2 - 4, M // 2 + 4), torch.arange(2 ** 21 - 4, M)]).to(dev)
    oq, os_, _ = ow.rmsnorm_i8(x[rows].cpu().numpy())
    assert np.array_equal(q[rows].cpu().numpy(), oq) and np.array_equal(sc[rows].cpu().numpy(), os_)
    assert not bool(torch.isnan(sc).any())
