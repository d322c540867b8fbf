"""Which of the two kernels of the block-scaled product a call takes, and both of them over the shapes and forms that their
users meet."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref
from tests.test_gpu_fp8 import _check_product, _experts, _expected, _fp8_weights, _gen, _ok, _operands, _product

pytestmark = pytest.mark.gpu


def _names(run):
    """Names of the launches of run(), and what it returns."""
    moe.trace_enable(True)
    moe.trace_read()
    try:
        out = run()
        torch.cuda.synchronize()
        return [n for n, _ in moe.trace_read()], out
    finally:
        moe.trace_enable(False)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("M,N", [(128, 4096), (128, 4608), (96, 4096), (96, 6016), (64, 9472), (32, 18944), (33, 9472), (33, 9600),
                                 (160, 3584), (128, 4864), (8, 18944), (256, 2304), (256, 2432), (320, 4096)])
def test_a_single_matrix_fills_the_gpu_or_not(M, N):
    """Tiles of 32 rows x 128 outputs, no more of them than SMs: the few-row kernel, whatever M is a multiple of.  More of
    them and more than 8 rows: the other one."""
    K = 288
    a, sa, b, sb = _operands(M, 1, N, K, "e4m3", "e4m3", M + N)
    names, out = _names(lambda: _product(a, sa, b, sb, None, torch.float32))
    tiles = -(-M // 32) * -(-N // 128)
    assert names == ["fp8_gemm" if tiles <= _sms() or M <= 8 else "fp8_gemm_rows"], tiles
    _check_product(out, a, sa, b, sb, [0, M])
