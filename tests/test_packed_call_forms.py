"""What the binding hands to the library, without a GPU: the call is recorded in
place of being made."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(bd, "_call", lambda fn, dev, *args: made.append(args))
    return made


def attention():
    x = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    return x, torch.tensor([0, 4, 8], dtype=torch.int32), torch.tensor([1, 1], dtype=torch.int32)


def test_keys_of_their_own_table_keep_their_lengths(calls):
    """q_len stands for the keys too where no k_off is given; with a k_off, the same tensor or an equal one, it does not."""
    x, off, one = attention()
    out, lse = x.clone(), torch.zeros(2, 8)
    for k_off in (off, off.clone()):
        bd.packed_forward(x, x, x, off, k_off, q_len=one)
        bd.packed_backward(x, x, x, out, lse, x, off, k_off, q_len=one)
        f, b = calls[-2:]
        assert f[4] == off.data_ptr() and f[5] == k_off.data_ptr() and f[6] == one.data_ptr() and f[7] is None
        assert b[7] == off.data_ptr() and b[8] == k_off.data_ptr() and b[9] == one.data_ptr() and b[10] is None
    bd.packed_forward(x, x, x, off, q_len=one)
    bd.packed_backward(x, x, x, out, lse, x, off, q_len=one)
    f, b = calls[-2:]
    assert f[5] == f[4] and f[7] == one.data_ptr() and b[8] == b[7] and b[10] == one.data_ptr()
