"""Shapes and numbers that the binding of the W8A8 block's operators refuses, on the CPU: every call here ends
before it asks for a GPU."""
import pytest
import torch

import quantized_state_space_amd as qs

I8 = torch.int8


def update_tensors(B=2, nh=4, P=8, N=16, G=2, gs=8):
    z = torch.zeros
    return dict(x=z(B, nh, P), x_group_of=z(nh * P, dtype=torch.uint8), x_scales=z(1), Bm=z(B, G, N), Cm=z(B, G, N),
                B_scales=z(G * N // gs), C_scales=z(G * N // gs), gs=gs, delta=z(B, nh), A=z(nh),
                state=z(B, nh, P, N, dtype=I8), y=z(B, nh, P), Dskip=z(nh), xq_out=z(B, nh, P, dtype=I8),
                Bq_out=z(B, G, N, dtype=I8), Cq_out=z(B, G, N, dtype=I8))


@pytest.mark.parametrize("name,label,shape", [
    ("Bm", "B", (1, 2, 16)), ("Bm", "B", (3, 2, 16)), ("Cm", "C", (1, 2, 16)), ("Cm", "C", (2, 2, 8)), ("delta", "delta", (1, 4)),
    ("A", "A", (3,)), ("x_group_of", "x_group_of", (31,)), ("B_scales", "B_scales", (2,)), ("C_scales", "C_scales", (5,)),
    ("state", "state", (1, 4, 8, 16)), ("y", "y", (2, 4, 4)), ("Dskip", "Dskip", (1,)), ("xq_out", "xq_out", (1, 4, 8)),
    ("Bq_out", "Bq_out", (1, 2, 16)), ("Cq_out", "Cq_out", (1, 2, 16))])
def test_update_args_refuses_tensors_of_other_sizes(name, label, shape):
    t = update_tensors()
    t[name] = torch.zeros(shape, dtype=t[name].dtype)
    with pytest.raises(ValueError, match=f"^{label} must have shape"):
        qs.update_args(**t)


@pytest.mark.parametrize("groups,error", [(0, ValueError), (-1, ValueError), (65, ValueError), (2 ** 32 + 1, ValueError),
                                          (2 ** 40 + 2, ValueError), (2.5, ValueError), (None, TypeError)])
def test_norm_refuses_group_counts(groups, error):
    """Among them counts that a 32-bit field or a conversion would turn into another one."""
    with pytest.raises(error) as e:
        qs.rmsnorm_args(torch.zeros(4, 64), torch.zeros(4, 64, dtype=I8), torch.zeros(4), norm_groups=groups)
    assert "GPU" not in str(e.value)
