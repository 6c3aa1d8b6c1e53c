"""The norm on tensors that lie in one buffer without sharing an element, and on a stream that replaces x."""
import numpy as np
import pytest

import oracle.w8a8 as ow
from tests.test_gpu_rmsnorm_i8 import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,D", [(5, 64), (700, 1001), (600, 2048)])
def test_columns_of_one_tensor(dev, M, D):
    """x, residual, residual_out and the codes as columns of one fp32 tensor, an unused column behind each."""
    print(f"\n[rmsnorm columns of one tensor M={M} D={D}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    x, w, res, _ = make(110, M, D, "f32", "f32", None)
    wide = torch.full((M, 4 * (D + 8)), -7.0, device=dev)
    cols = [wide[:, k * (D + 8):k * (D + 8) + D] for k in range(3)]
    cols[0].copy_(torch.from_numpy(x))
    cols[1].copy_(torch.from_numpy(res))
    before = wide.clone()
    q = wide.view(torch.int8)[:, 12 * (D + 8):12 * (D + 8) + D]
    sc = torch.empty(M, device=dev)
    qs.qssm_rmsnorm_i8(qs.rmsnorm_args(cols[0], q, sc, weight=torch.from_numpy(w).to(dev), residual=cols[1], residual_out=cols[2]))
    oq, os_, oh = ow.rmsnorm_i8(x, w, residual=res, residual_dtype=np.float32)
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sc.cpu().numpy(), os_)
    assert np.array_equal(cols[2].cpu().numpy(), oh)
    cols[2].fill_(-7.0)
    q.copy_(before.view(torch.int8)[:, 12 * (D + 8):12 * (D + 8) + D])
    assert torch.equal(wide, before), "something else was written"


@pytest.mark.parametrize("xt", ["f16", "f32"])
@pytest.mark.parametrize("M,D", [(3, 64), (700, 1001), (600, 4096)])
def test_stream_in_place_of_x(dev, xt, M, D):
    """residual_out is x itself, with a residual of its type and without one."""
    print(f"\n[rmsnorm stream in place of x M={M} D={D} {xt}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    x, w, res, _ = make(111, M, D, xt, xt, None)
    wt = torch.from_numpy(w).to(dev)
    for r in (res, None):
        xd = torch.from_numpy(x).to(dev)
        q, sc = torch.empty(M, D, dtype=torch.int8, device=dev), torch.empty(M, device=dev)
        qs.qssm_rmsnorm_i8(qs.rmsnorm_args(xd, q, sc, weight=wt, residual=None if r is None else torch.from_numpy(r).to(dev), residual_out=xd))
        oq, os_, oh = ow.rmsnorm_i8(x, w, residual=r, residual_dtype=x.dtype)
        assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(sc.cpu().numpy(), os_)
        assert np.array_equal(xd.cpu().numpy(), oh)
