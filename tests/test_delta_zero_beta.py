"""Tokens that write nothing (beta = 0): no gradient for their values, exactly."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make
from tests.test_packed import off_of


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
def test_no_gradient_for_values_not_written(cuda_ok, dtype, path, d):
    T, off = 150, off_of([70, 80])
    x, randn = make(T, 1, 2, d, dtype, d)
    x["beta"][3::5] = 0.0
    do, dS = randn(T, 2, d).to(dtype), 0.1 * randn(2, 2, d, d)
    dv = bd.delta_backward(*x.values(), off, do, dS_out=dS, path=path)[2]
    zero = x["beta"] == 0
    assert (dv[zero] == 0).all() and (dv[~zero] != 0).any(-1).all()
