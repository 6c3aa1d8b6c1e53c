"""Limits of the W8A8 block's entry points that keep their address arithmetic inside 64 bits, and the tensors that they
refuse for how they lie in memory. No GPU: every call here returns before any launch."""
import pytest

import quantized_state_space_amd as qs
from tests.test_capi_w8a8 import INV, P, UNS, gemm, message, norm


@pytest.mark.parametrize("tensor", ["x", "q", "residual", "residual_out", "gate"])
def test_norm_refuses_rows_past_64_bits(tensor):
    """2^31 - 1 rows 2^40 elements apart each keep to their own limit, but end 2^73 bytes from the first."""
    for rows, stride in ((2 ** 31 - 1, 2 ** 40), (2 ** 31 - 1, 2 ** 27 + 1), (2 ** 20, 2 ** 38 + 8), (2 ** 18 + 1, 2 ** 40)):
        kw = {tensor: P, tensor + "_stride": stride}
        assert norm(rows=rows, **kw) == UNS and "2^58" in message(), (rows, stride)


def test_gemm_refuses_rows_past_64_bits():
    for M, stride in ((2 ** 27, 2 ** 40), (2 ** 27, 2 ** 31 + 1), (2 ** 18 + 1, 2 ** 40)):
        assert gemm(M=M, y_stride=stride) == UNS and "2^58" in message(), (M, stride)
