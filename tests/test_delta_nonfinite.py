"""A NaN gate in the gated delta rule: it is not a reset. From its token on the
state, and all that is read from it, is NaN, in its sequence and head only."""
import math

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make
from tests.test_packed import off_of

TYPES = [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_TC)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("lens,row", [([30, 5], 0), ([30, 5], 29), ([7, 6], 3), ([150, 20], 0), ([150, 20], 70),
                                      ([150, 20], 149)])
def test_nan_gate(cuda_ok, lens, row, dtype, path, d):
    """Token by token (up to 8 and up to 48 tokens), in chunks, and backward."""
    n, T = lens[0], sum(lens)
    x, randn = make(T, 2, 4, d, dtype, row + n)
    off, S0, dS1 = off_of(lens), 0.3 * randn(2, 4, d, d), 0.1 * randn(2, 4, d, d)
    do = randn(T, 4, d).to(dtype)

    def both():
        out, S = bd.delta_forward(*x.values(), off, S_in=S0, max_len=max(lens), path=path)
        return (out, S, *bd.delta_backward(*x.values(), off, do, S_in=S0, dS_out=dS1, max_len=max(lens), path=path))

    clean = both()
    x["g"][row, 1] = math.nan
    got = both()
    out, S, dq, dk, dv, dg, dbeta, dS = got
    assert out[row:n, 1].isnan().all() and S[0, 1].isnan().all()
    assert dq[row:n, 0].isnan().all() and dS[0, 1].isnan().all() and dv[:row, 1].isnan().all() and dg[row, 1].isnan()
    for i, (a, b) in enumerate(zip(got, clean)):
        state, per_key = i in (1, 7), i in (2, 3)
        other = slice(1, None) if state else slice(n, None)  # the other sequence
        assert torch.equal(a[other], b[other]), i
        for h in ((1,) if per_key else (0, 2, 3)):           # the other heads (key head 0 has value heads 0 and 1)
            assert torch.equal(a[:, h], b[:, h]), (i, h)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_gate_of_a_step(cuda_ok, dtype, d):
    x, randn = make(3, 1, 2, d, dtype, 4)
    S = 0.3 * randn(3, 2, d, d)
    x["g"][1, 1] = math.nan
    S2 = torch.empty_like(S)
    out = bd.delta_step(*x.values(), S, S_out=S2)
    hit = torch.zeros(3, 2, dtype=torch.bool, device="cuda")
    hit[1, 1] = True
    assert out[hit].isnan().all() and S2[hit].isnan().all()
    assert out[~hit].isfinite().all() and S2[~hit].isfinite().all()
