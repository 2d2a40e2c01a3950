"""Write strengths next to nothing (a saturated gate): dbeta keeps its digits.

With du the gradient of a token's pseudo-value and err = v - S'^T k, dbeta = du .
err does not depend on beta. The kernels that go through tensors of the row type
round du and err (times beta) once each, u = 2^-8 of every term, and the result;
the state's and fp32 sums' errors are some 2^-14 of a term and more than covered
by counting four u."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make, recur, reverse
from tests.test_packed import off_of


@pytest.mark.gpu
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_TC])
@pytest.mark.parametrize("beta", [0.0, 2.0 ** -100, 2.0 ** -112, -2.0 ** -118, 2.0 ** -120, 2.0 ** -126, -2.0 ** -127,
                                  2.0 ** -130, 2.0 ** -133])
def test_gradient_of_a_small_beta(cuda_ok, beta, path):
    T, d = 90, 64
    x, randn = make(T, 1, 1, d, torch.bfloat16, 3)
    x["beta"][5::4] = beta
    assert float(x["beta"][5]) == beta
    do = randn(T, 1, d).bfloat16()
    g = bd.delta_backward(*x.values(), off_of([T]), do, path=path)
    q, k, v, lg, b = (t.double().cpu()[:, 0] for t in x.values())
    a, zero, scale = lg.exp(), torch.zeros(d, d, dtype=torch.float64), d ** -0.5
    _, _, kept = recur(q, k, v, a, b, zero, scale, -1)
    do = do.double().cpu()[:, 0]
    want = reverse(q, k, v, a, b, do, zero, scale, kept, -1)["dbeta"]
    # the sizes of the terms, on the same way back
    dS, size = zero, torch.zeros(T, dtype=torch.float64)
    for t in reversed(range(T)):
        X = dS + scale * torch.outer(q[t], do[t])
        du = k[t] @ X
        size[t] = (du * kept[t][1]).abs().sum()
        dS = (X - torch.outer(k[t], b[t] * du)) * a[t]
    off = (g[4].double().cpu()[:, 0] - want).abs()
    assert (off <= 4 * 2.0 ** -8 * size).all(), float((off / size).max())
    assert (want.abs() > 4 * 2.0 ** -8 * size)[5::4].float().mean() > 0.5  # zeros would not do
