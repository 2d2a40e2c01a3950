"""The automatic choice between the split keys and the tiles, by what was
measured on both sides (no GPU: the choice is the host's)."""
import pytest

from compressive_memory_segment_b200 import binding as bd
from tests.test_packed import shape

SPLIT, TC, SIMT = bd.INFINI_PATH_SPLIT, bd.INFINI_PATH_TC, bd.INFINI_PATH_SIMT


@pytest.mark.parametrize("dtype,n,Hq,Hkv,d,nq,nk,path", [
    # many sequences: tiles as soon as the rows make more work than the heads
    (bd.INFINI_BF16, 256, 8, 8, 64, 64, 512, TC),        # 117 us, split 260
    (bd.INFINI_BF16, 256, 8, 8, 64, 16, 16, SPLIT),      # 40 us, tiles 61
    (bd.INFINI_BF16, 16, 8, 8, 64, 64, 512, TC),         # 17 us, split 30
    (bd.INFINI_BF16, 256, 32, 8, 128, 16, 512, SPLIT),   # 414 us, tiles 454
    (bd.INFINI_BF16, 2000, 4, 2, 64, 20, 20, SPLIT),     # 170 us, tiles 205
    (bd.INFINI_BF16, 256, 16, 1, 128, 4, 512, SPLIT),    # 77 us, tiles 236
    (bd.INFINI_BF16, 48, 32, 8, 128, 16, 4096, SPLIT),   # 514 us, tiles 635
    (bd.INFINI_BF16, 48, 32, 8, 128, 64, 4096, TC),      # 654 us, split 1977
    (bd.INFINI_F32, 256, 8, 8, 64, 64, 512, SIMT),       # 569 us, split 2759
    (bd.INFINI_F32, 256, 32, 8, 128, 16, 512, SIMT),     # 2405 us, split 5660
    (bd.INFINI_F32, 256, 32, 8, 128, 4, 4, SPLIT),       # 121 us, tiles 212
    (bd.INFINI_F32, 16, 32, 8, 128, 16, 512, SIMT),      # 176 us, split 231
    # one sequence: its keys have to be spread
    (bd.INFINI_BF16, 1, 8, 8, 64, 64, 512, SPLIT),       # 14 us, tiles 16
    (bd.INFINI_BF16, 1, 32, 8, 128, 16, 8192, SPLIT),    # 43 us, tiles 109
    (bd.INFINI_F32, 1, 32, 8, 128, 16, 512, SPLIT),      # 24 us, tiles 59
    (bd.INFINI_F32, 1, 8, 8, 64, 64, 512, SPLIT),        # 22 us, tiles 34
])
def test_choice(dtype, n, Hq, Hkv, d, nq, nk, path):
    s = shape(n_seq=n, Tq=n * nq, Tk=n * nk, Hq=Hq, Hkv=Hkv, d=d, max_q=nq, max_k=nk, dtype=dtype)
    assert bd._lib.infini_attn_packed_select_path(s) == path


@pytest.mark.parametrize("dtype", [bd.INFINI_BF16, bd.INFINI_F32])
def test_rows_of_the_split_path_end_before_32_bits_do(dtype):
    """Its loop over rows steps up to 1024 beyond the last one in 32 bits: within that of 2^31 the path is not taken."""
    for Tq, fits in (((1 << 29) - 1, False), ((1 << 29) - 256, False), ((1 << 29) - 257, True)):
        s = shape(n_seq=1, Tq=Tq, Hq=4, Hkv=1, max_q=1, max_k=8, dtype=dtype)
        assert (bd._lib.infini_attn_packed_select_path(s) == SPLIT) == fits, Tq
        assert (bd._lib.infini_attn_packed_workspace_size(s, SPLIT) > 0) == fits
