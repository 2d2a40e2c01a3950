"""Steps of very many sequences and key heads against their caches."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_packed import close, make, off_of, reference, shape


def test_path_does_not_end_at_a_grid_dimension():
    """Few rows a key head take the split path for any number of sequences that the sizes allow."""
    sel = bd._lib.infini_attn_packed_select_path
    for n, Hkv, dtype in ((8191, 8, bd.INFINI_BF16), (8192, 8, bd.INFINI_BF16), (100000, 8, bd.INFINI_BF16),
                          (70000, 1, bd.INFINI_F32)):
        s = shape(n_seq=n, Tq=n, Tk=n * 16, Hq=4 * Hkv, Hkv=Hkv, max_q=1, max_k=16, dtype=dtype)
        assert sel(s) == bd.INFINI_PATH_SPLIT, (n, Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,Hkv", [(70000, 1), (9000, 8)])
def test_more_sequences_times_heads_than_a_grid_dimension(cuda_ok, n, Hkv, dtype):
    gen = torch.Generator(device="cuda").manual_seed(Hkv)
    q, k, v = make(n, Hkv, 64, dtype, gen), make(2 * n, Hkv, 64, dtype, gen), make(2 * n, Hkv, 64, dtype, gen)
    k_len = (torch.arange(n, device="cuda") % 3).int()
    one = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse = bd.packed_forward(q, k, v, one, one * 2, k_len=k_len, max_q=1, max_k=2, path=bd.INFINI_PATH_SPLIT)
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
    some = [0, 1, 2, n // 2, n // 2 + 1, n // 2 + 2, n - 3, n - 2, n - 1, 65535 % n, 65536 % n, 65537 % n]
    ref, bound = reference(q, k, v, [(s, 1) for s in some], [(2 * s, s % 3) for s in some], 64 ** -0.5)
    close("out", out, ref["out"], bound["out"])
    close("lse", lse, ref["lse"], bound["lse"])
    # every row: no key, one key (out is its value), two keys (between the two values)
    none, lone = k_len == 0, k_len == 1
    assert (out[none] == 0).all() and (lse.t()[none] == -torch.inf).all()
    two = v.view(n, 2, Hkv, 64)
    # p is 1 exactly, so is l
    assert torch.equal(out[lone], two[lone][:, 0])
    pair = two[k_len == 2].float()
    mid, half = (pair[:, 0] + pair[:, 1]) / 2, (pair[:, 0] - pair[:, 1]).abs() / 2
    slack = 2.0 ** -6 * pair.abs().amax(1)  # two roundings of p, one of the result, one of the sum
    assert ((out[k_len == 2].float() - mid).abs() <= half + slack).all()
