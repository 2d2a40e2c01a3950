"""Extents of rows beyond what an address can hold."""
import pytest

from compressive_memory_segment_b200 import binding as bd

D = 64


@pytest.mark.parametrize("st,sh", [(1 << 38, 1 << 38), (1 << 38, D)])
def test_extents_beyond_an_address_space_are_refused(st, sh):
    """Strides whose product with the sizes leaves 64 bits must not pass the checks with a wrapped extent."""
    s = bd.infini_packed_shape(0, 1 << 29, 8, 4, 4, D, 8, 8, bd.INFINI_BF16, 0.125)
    far = lambda i: bd.infini_rows((i + 1) << 40, 4 * D, D)  # noqa: E731
    q = bd.infini_rows(1 << 36, st, sh)
    rc = bd._lib.infini_attn_packed_forward(s, q, far(2), far(3), None, None, None, None, far(4), None, 9 << 42, 1 << 40,
                                            bd.INFINI_PATH_SIMT, None)
    assert rc == bd.INFINI_ERR_SIZE
