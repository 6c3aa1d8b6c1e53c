"""The gated norm's fp32 gates far below zero, where silu is -0 whatever the gate's size: rows and groups in
which nothing larger hides a value that should have vanished. Codes and scales bit for bit."""
import numpy as np
import pytest

from tests.test_gpu_rmsnorm_i8 import check

pytestmark = pytest.mark.gpu

LOWEST = -3.4028235e38
FAR = [-127.0, -200.0, -1e4, -2.0 ** 31, -4e9, -1e12, -1e20, -3e38, LOWEST]


@pytest.mark.parametrize("D,groups", [(64, 1), (64, 4), (63, 3), (1001, 1)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_every_gate_far_below_zero(dev, D, groups, eps):
    """Rows of one gate value: codes 0 and scale 1."""
    print(f"\n[rmsnorm gates far below zero D={D} groups={groups} eps={eps}]", flush=True)
    z = np.repeat(np.float32(FAR)[:, None], D, axis=1)
    x = np.random.default_rng([98, D]).standard_normal(z.shape).astype(np.float32)
    with np.errstate(divide="ignore"):
        check(dev, x, np.ones(D, np.float32), None, z, groups=groups, eps=eps)
        check(dev, (1e30 * x).astype(np.float32), None, None, z, groups=groups, eps=eps)


@pytest.mark.parametrize("D,groups", [(64, 1), (64, 4), (63, 3)])
def test_far_gates_beside_small_ones(dev, D, groups):
    """Gates whose silu is tiny but not 0 (0, 1e-30, -100, 1e-38) beside far ones, a group of far ones alone,
    and an infinite one."""
    print(f"\n[rmsnorm far gates beside small ones D={D} groups={groups}]", flush=True)
    r = np.random.default_rng([99, D])
    small = np.float32([0.0, -0.0, 1e-30, -1e-30, 1e-38, -100.0, -103.0])
    rows = []
    for far in FAR:
        z = small[r.integers(0, len(small), D)]
        z[r.random(D) < 0.5] = far
        z[:D // groups] = far
        rows.append(z)
    z = np.stack(rows + [rows[-1], rows[0]])
    z[-2, D // 2], z[-1, D // 2] = -np.inf, np.inf
    x = r.standard_normal(z.shape).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        for eps in (0.0, 1e-30, 1e-5):
            check(dev, x, np.ones(D, np.float32), None, z.astype(np.float32), groups=groups, eps=eps)


def test_fp16_gates_at_the_end_of_their_range(dev):
    print("\n[rmsnorm fp16 gates of -65504]", flush=True)
    z = np.full((3, 64), -65504, np.float16)
    z[1], z[2, ::2] = 65504, 0
    x = np.random.default_rng(100).standard_normal((3, 64)).astype(np.float32)
    with np.errstate(divide="ignore"):
        check(dev, x, np.ones(64, np.float32), None, z, groups=2)
        check(dev, x, np.ones(64, np.float32), None, z, eps=0.0)
