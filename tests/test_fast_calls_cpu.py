"""The native marshalling (csrc/fast_calls.cpp) leaves every call that is not a
plain one to the Python wrappers: tensors off the GPU, other objects, other
types and counts of arguments give None and nothing happens."""
import pytest
import torch

import fp8_precision_quant_amd as fq
from fp8_precision_quant_amd import _fast

F, I8 = torch.zeros(4, 32), torch.zeros(4, 32, dtype=torch.int8)
V = torch.zeros(4)


@pytest.mark.parametrize("f,args", [
    (_fast.layer_norm_forward, (F, None, None, 1e-5)), (_fast.layer_norm_forward, (F, F[0], F[0], 1e-5)),
    (_fast.layer_norm_forward, (None, None, None, 1e-5)), (_fast.layer_norm_forward, (F, "w", 3, "eps")),
    (_fast.layer_norm_forward, ()), (_fast.layer_norm_forward, (F,)),
    (_fast.layer_norm_backward, (F, F, V, V, F[0])), (_fast.layer_norm_backward, (F, F, V, V, None)),
    (_fast.layer_norm_backward, (1, 2, 3, 4, 5)), (_fast.layer_norm_backward, ()),
    (_fast.int8_quant_rows, (F,)), (_fast.int8_quant_rows, ([1.0],)), (_fast.int8_quant_rows, ()),
    (_fast.int8_quant_rows, (torch.zeros(4, 32).to_sparse(),)), (_fast.int8_quant_rows, (torch.zeros(4, 32, device="meta"),)),
    (_fast.int8_gemm, (I8, V, I8, V, None, True)), (_fast.int8_gemm, (None,) * 6), (_fast.int8_gemm, (I8, V)),
    (_fast.adamw_multi_step, ()), (_fast.adamw_multi_step, (None,) * 18),
    (_fast.adamw_multi_step, ([], 0, 0, [], *(None,) * 14)), (_fast.adamw_multi_step, ([V], 0, 0, [V], *(None,) * 14)),
])
def test_other_calls_are_left_to_the_wrappers(f, args):
    assert f(*args) is None


def test_product_of_more_columns_than_a_launch_counts():
    """A launch's threads are counted in 32 bits: 2^28 channels of 16 a workgroup of 256 would pass them."""
    p = 1 << 20
    for M, N, status in ((1, 1 << 28, fq.ERR_UNSUPPORTED), (1 << 27, 129, fq.ERR_UNSUPPORTED), (1 << 13, 1 << 22, fq.ERR_UNSUPPORTED)):
        got = fq._lib.fp8q_int8_gemm(M, N, 16, p, 16, p, p, 16, p, None, p, (N + 15) // 16 * 16, fq.BF16, p, 1 << 40, None)
        assert got == status
