"""The W8A8 linear layer's y as columns of the tensor that holds its activations."""
import numpy as np
import pytest

import oracle.w8a8 as ow
from tests.test_gpu_gemm_w8a8 import bound, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (20, 64, 256), (300, 200, 516)])
def test_y_beside_its_activations(dev, M, N, K):
    print(f"\n[gemm_w8a8 y beside a M={M} N={N} K={K}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    a, sa, w, sw, b = make(M, M, N, K)
    wide = torch.full((M, K // 4 + N + 1), -7.0, device=dev)
    codes, y = wide.view(torch.int8)[:, :K], wide[:, K // 4:K // 4 + N]
    codes.copy_(torch.from_numpy(a))
    dv = lambda v: torch.from_numpy(v).to(dev)  # noqa: E731
    qs.qssm_gemm_w8a8(qs.gemm_w8a8_args(codes, dv(sa), dv(w), dv(sw), y, bias=dv(b)))
    yb = ow.gemm_w8a8(a, sa, w, sw)
    assert np.all(np.abs(y.cpu().numpy() - (yb + b)) <= bound(yb + b, yb, False))
    assert np.array_equal(codes.cpu().numpy(), a) and bool((wide[:, -1] == -7.0).all())
