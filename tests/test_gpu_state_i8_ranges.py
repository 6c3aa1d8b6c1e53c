"""The int8 state update with scales and inputs from the whole range, where the state and what is added to it are many powers of
two apart: one rounding of the fused sum, codes and scales bit for bit."""
import numpy as np
import pytest

import oracle.w8a8 as ow
from tests.test_gpu_state_i8 import Update, dequantized, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,nh,P,N,G,gs", [(5, 10, 25, 64, 2, 16), (4, 3, 105, 128, 3, 2), (3, 10, 98, 64, 2, 1), (3, 9, 165, 32, 3, 16),
                                           (3, 2, 183, 16, 2, 16), (2, 12, 64, 256, 3, 4)])
def test_update_of_scales_from_the_whole_range(dev, B, nh, P, N, G, gs):
    print(f"\n[state_update_i8 scales of the whole range B={B} nh={nh} P={P} N={N} G={G} gs={gs}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(B + nh + P, B, nh, P, N, G, gs)
    r = np.random.default_rng([103, P])
    d["scales"] = np.exp(r.uniform(-69, 69, d["scales"].shape)).astype(np.float32)
    _, (xh, Bh, Ch) = dequantized(d, gs)
    y, q, s, h = ow.state_update(d["codes"], d["scales"], xh, Bh, Ch, d["delta"], d["A"], d["D"])
    u = Update(dev, d, gs)
    qs.qssm_state_update_i8(u.args, u.t["scales"])
    torch.cuda.synchronize()
    assert np.array_equal(u.t["scales"].cpu().numpy(), s)
    assert np.array_equal(u.state.cpu().numpy(), q)
    total = (np.abs(h.astype(np.float64)) * np.abs(Ch[:, :, None, :])).sum(3) + np.abs(d["D"][None, :, None].astype(np.float64) * xh)
    assert np.all(np.abs(u.y.cpu().numpy().astype(np.float64) - y) <= (N + 2) * 2.0 ** -24 * total)
