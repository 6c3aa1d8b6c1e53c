"""The int8 state update's readout y in rows that are not finite or whose scale is clamped, where the update takes its
general path: y follows the arithmetic, y = sum C h + D x with every step rounded to fp32."""
import numpy as np
import pytest

import oracle.w8a8 as ow
from tests.test_gpu_state_i8 import Update, dequantized, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("skip", [False, True])
def test_readout_of_rows_that_are_not_finite(dev, skip):
    """Where the finite products of a row sum to less than fp32's largest in magnitude, y is of the oracle's kind (NaN, an
    infinity's sign, or finite), and finite ones are within (N + 2) roundings of 2^-24."""
    print(f"\n[state_update_i8 readout not finite skip={skip}]", flush=True)
    import torch
    import quantized_state_space_amd as qs
    d = make(1, 2, 4, 32, 128, 2, 16)
    N = 128
    d["delta"][0, 0], d["delta"][1, 1] = np.nan, np.inf
    d["scales"][0, 1] = 2.0 ** 100                 # values of ~2^106: the new scales are at the end of their range
    d["scales"][1, 2], d["A"][2] = 2.0 ** 100, 3.0  # beyond it: growth past 127 * 2^100 ...
    d["delta"][1, 2] = 2.0                          # ... by e^6, still finite
    d["scales"][1, 3], d["A"][3], d["delta"][1, 3] = 2.0 ** 100, 2.5 * np.log(2.0), 10.0  # by 2^25: infinite from code 8 on,
    d["codes"][1, 3, :, 1:] = 0                     # ... in one value a row, the only one that is read out
    d["C"][1, 1, 0], d["C"][1, 1, 1:] = 1.0, 0.0
    with np.errstate(all="ignore"):
        _, (xh, Bh, Ch) = dequantized(d, 16)
        y, q, s, h = ow.state_update(d["codes"], d["scales"], xh, Bh, Ch, d["delta"], d["A"], d["D"] if skip else None)
        h64, c64 = h.astype(np.float64), Ch[:, :, None, :].astype(np.float64)
        total = np.where(np.isfinite(h64), np.abs(h64 * c64), 0.0).sum(3)
        if skip:
            total = total + np.abs(d["D"][None, :, None].astype(np.float64) * xh)
    sure = total < 1e38
    u = Update(dev, d, 16, skip=skip)
    qs.qssm_state_update_i8(u.args, u.t["scales"])
    torch.cuda.synchronize()
    got = u.y.cpu().numpy().astype(np.float64)
    assert np.array_equal(u.t["scales"].cpu().numpy(), s) and np.array_equal(u.state.cpu().numpy(), q)
    nan, inf = np.isnan(y) & sure, np.isinf(y) & sure
    fine = np.isfinite(y) & sure
    big = fine & (np.abs(h64).max(axis=3, initial=0, where=np.isfinite(h64)) > 127 * 2.0 ** 100)
    assert nan.any() and inf.any() and fine.any() and big.any()
    assert np.all(np.isnan(got[nan]))
    assert np.array_equal(got[inf], y[inf])
    assert np.all(np.abs(got[fine] - y[fine]) <= (N + 2) * 2.0 ** -24 * total[fine])
