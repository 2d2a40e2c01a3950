"""Elements that are not finite in packed attention: a NaN reaches what depends
on it and is never taken for a query that sees no key."""
import math

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_packed import make, off_of

FORWARD = [(torch.float32, bd.INFINI_PATH_SIMT), (torch.float32, bd.INFINI_PATH_SPLIT),
           (torch.bfloat16, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SPLIT),
           (torch.bfloat16, bd.INFINI_PATH_TC)]


def forward(q, k, v, off, k_off, path):
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[1::-1], 7.0, device="cuda")
    bd.packed_forward(q, k, v, off, k_off, out=out, lse=lse, path=path)
    return out, lse.t()  # both by rows and heads


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", FORWARD)
@pytest.mark.parametrize("row", [0, 70, 199, 203])
def test_nan_in_a_query(cuda_ok, row, dtype, path, d):
    """out and lse of that row and head are NaN, everything else is bit for bit what it was."""
    gen = torch.Generator(device="cuda").manual_seed(row + d)
    q, k, v = make(240, 4, d, dtype, gen), make(240, 2, d, dtype, gen), make(240, 2, d, dtype, gen)
    off = off_of([200, 40])
    out, lse = forward(q, k, v, off, off, path)
    q[row, 1, 3] = math.nan
    hit = torch.zeros(240, 4, dtype=torch.bool, device="cuda")
    hit[row, 1] = True
    o2, l2 = forward(q, k, v, off, off, path)
    assert o2[hit].isnan().all() and l2[hit].isnan().all()
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", FORWARD)
@pytest.mark.parametrize("key", [0, 50, 128, 199])
def test_nan_in_a_key(cuda_ok, key, dtype, path, d):
    """Rows that see the key are NaN (the first may see nothing else), the rest of the sequence and the others are not."""
    gen = torch.Generator(device="cuda").manual_seed(key + d)
    q, k, v = make(240, 4, d, dtype, gen), make(240, 2, d, dtype, gen), make(240, 2, d, dtype, gen)
    off = off_of([200, 40])
    out, lse = forward(q, k, v, off, off, path)
    k[key, 0, 5] = math.nan
    hit = torch.zeros(240, 4, dtype=torch.bool, device="cuda")
    hit[key:200, :2] = True
    o2, l2 = forward(q, k, v, off, off, path)
    assert o2[hit].isnan().all() and l2[hit].isnan().all()
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", FORWARD)
def test_nan_in_a_query_that_sees_no_key(cuda_ok, dtype, path):
    """Such a row is 0 and -inf whatever it holds."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = make(70, 4, 64, dtype, gen), make(20, 2, 64, dtype, gen), make(20, 2, 64, dtype, gen)
    q[10] = math.nan
    out, lse = forward(q, k, v, off_of([70]), off_of([20]), path)
    assert (out[:50] == 0).all() and (lse[:50] == -math.inf).all()
    assert out[50:].isfinite().all() and lse[50:].isfinite().all()
