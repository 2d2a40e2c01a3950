"""A NaN in packed attention's inputs reaches every gradient that depends on it."""
import math

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_packed import make, off_of


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
@pytest.mark.parametrize("row", range(64, 72))
def test_nan_in_a_query_reaches_its_gradients(cuda_ok, row, dtype, path, d):
    """dq of the row and dk, dv of every key it sees, wherever the row lies in a tile; no other row's dq, no other
    sequence and no other key head."""
    gen = torch.Generator(device="cuda").manual_seed(row)
    q, k, v = make(140, 4, d, dtype, gen), make(140, 2, d, dtype, gen), make(140, 2, d, dtype, gen)
    do, off = make(140, 4, d, dtype, gen), off_of([100, 40])

    def both():
        out, lse = bd.packed_forward(q, k, v, off, path=path)
        return bd.packed_backward(q, k, v, out, lse, do, off, path=path)

    clean = both()
    q[row, 1, 3] = math.nan
    dq, dk, dv = both()
    assert dq[row, 1].isnan().all() and dk[:row + 1, 0].isnan().all() and dv[:row + 1, 0].isnan().all()
    same = torch.ones(140, 4, dtype=torch.bool, device="cuda")
    same[row, 1] = False
    assert torch.equal(dq[same], clean[0][same])
    for x, y in zip((dk, dv), clean[1:]):
        assert torch.equal(x[:, 1], y[:, 1]) and torch.equal(x[100:], y[100:])
