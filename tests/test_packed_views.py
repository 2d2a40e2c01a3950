"""Outputs that interleave with other tensors of the call: views of one buffer
that share no element are no overlap, whichever of its dimensions they alternate
in, and views that share one are."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make as make_delta
from tests.test_packed import make, off_of

D = 64


def rows(layout, i, T, H, n=3):
    """View i of n: [T][H][n][d], [H][T][n][d], [T][n][H][d] or [H][n][T][d], bf16."""
    at, st, sh = {"THnd": (D, H * n * D, n * D), "HTnd": (D, n * D, T * n * D), "TnHd": (H * D, n * H * D, D),
                  "HnTd": (T * D, D, n * T * D)}[layout]
    return bd.infini_rows(0x10000000 + 2 * i * at, st, sh)


def backward_of_no_sequence(dq, dk, dv, T, H):
    """The argument checks alone: with no sequence nothing is launched."""
    s = bd.infini_packed_shape(0, T, T, H, H, D, T, T, bd.INFINI_BF16, 0.125)
    far = lambda i: bd.infini_rows((i + 1) << 36, H * D, D)  # noqa: E731
    return bd._lib.infini_attn_packed_backward(s, far(1), far(2), far(3), far(4), 6 << 36, far(6), None, None, None, None,
                                               dq, dk, dv, 9 << 36, 1 << 30, bd.INFINI_PATH_AUTO, None)


@pytest.mark.parametrize("layout", ["THnd", "HTnd", "TnHd", "HnTd"])
@pytest.mark.parametrize("T,H", [(5, 4), (1, 4), (5, 1), (1, 1), (8, 2)])
def test_interleaved_views_do_not_overlap(layout, T, H):
    a, b, c = (rows(layout, i, T, H) for i in range(3))
    assert backward_of_no_sequence(a, b, c, T, H) == bd.INFINI_OK
    assert backward_of_no_sequence(c, a, b, T, H) == bd.INFINI_OK
    assert backward_of_no_sequence(a, b, b, T, H) == bd.INFINI_ERR_ALIAS
    half = bd.infini_rows(b.ptr + D, b.stride_t, b.stride_h)  # half of b's, half of the next one's elements
    assert backward_of_no_sequence(a, half, b, T, H) == bd.INFINI_ERR_ALIAS
    assert backward_of_no_sequence(half, a, c, T, H) == bd.INFINI_ERR_ALIAS


def test_different_grids_overlap():
    """Two views of one buffer whose steps do not fit each other are refused."""
    T, H = 8, 4
    a = bd.infini_rows(0x10000000, H * 3 * D, 3 * D)
    b = bd.infini_rows(0x10000000 + 2 * D, H * 2 * D, 2 * D)
    assert backward_of_no_sequence(a, b, bd.infini_rows(8 << 36, H * D, D), T, H) == bd.INFINI_ERR_ALIAS


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_beside_each_other_by_heads(cuda_ok, dtype):
    """q, k, v and their gradients per head in one projection's output, [T, H, 3, d]; g and beta as [T, H, 2]."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    T, H, off = 150, 4, off_of([90, 60])
    x, do = make(T, H * 3, D, dtype, gen).view(T, H, 3, D), make(T, H, D, dtype, gen)
    q, k, v = x.unbind(2)
    out, lse = bd.packed_forward(q, k, v, off)
    want = bd.packed_backward(q, k, v, out, lse, do, off)
    dx = torch.full_like(x, 7.0)
    bd.packed_backward(q, k, v, out, lse, do, off, dq=dx[:, :, 0], dk=dx[:, :, 1], dv=dx[:, :, 2])
    assert all(torch.equal(a, b) for a, b in zip(want, dx.unbind(2)))
    y, _ = make_delta(T, H, H, D, dtype, 3)
    want = bd.delta_backward(*y.values(), off, do)
    gb = torch.full((T, H, 2), 7.0, dtype=dtype, device="cuda")
    dx = torch.full_like(x, 7.0)
    bd.delta_backward(*y.values(), off, do, dq=dx[:, :, 0], dk=dx[:, :, 1], dv=dx[:, :, 2], dg=gb[:, :, 0], dbeta=gb[:, :, 1])
    assert all(torch.equal(a, b) for a, b in zip(want[:5], (*dx.unbind(2), *gb.unbind(2))))
