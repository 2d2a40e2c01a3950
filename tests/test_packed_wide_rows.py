"""Rows whose offsets in elements pass 2^31 and 2^32, in tokens and in heads."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make as make_delta
from tests.test_packed import make, off_of

BUFFER = (1 << 32) + (1 << 27)  # bf16 elements, 8.9 GB


@pytest.fixture(scope="module")
def buffer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.empty(BUFFER, dtype=torch.bfloat16, device="cuda")
    yield x
    del x
    torch.cuda.empty_cache()


def far(buffer, x, by_heads, first):
    """x's values in a view whose tokens (or heads) lie as far apart as the buffer allows."""
    T, H = x.shape[:2]
    d = x.shape[2] if x.dim() == 3 else 1
    wide, narrow = (BUFFER - (1 << 26)) // ((H if by_heads else T) - 1) // 2048 * 2048, 2048
    st, sh = (narrow, wide) if by_heads else (wide, narrow)
    y = buffer.as_strided((T, H, d), (st, sh, 1), first)
    y = y if x.dim() == 3 else y[..., 0]
    y.copy_(x)
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("by_heads", [False, True])
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_TC, bd.INFINI_PATH_SPLIT])
def test_attention(cuda_ok, buffer, path, by_heads):
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, H, d = 40, 3, 64
    off = off_of([9, 31])
    q, k, v, do = (make(T, H, d, torch.bfloat16, gen) for _ in range(4))
    want = list(bd.packed_forward(q, k, v, off, path=path))
    wide = [far(buffer, t, by_heads, 128 * i) for i, t in enumerate((q, k, v, do, torch.zeros_like(q)))]
    got = list(bd.packed_forward(*wide[:3], off, out=wide[4], path=path))
    if path != bd.INFINI_PATH_SPLIT:
        want += bd.packed_backward(q, k, v, *want, do, off, path=path)
        g = [far(buffer, torch.zeros_like(q), by_heads, 128 * (5 + i)) for i in range(3)]
        got += bd.packed_backward(*wide[:3], *got, wide[3], off, dq=g[0], dk=g[1], dv=g[2], path=path)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK


@pytest.mark.gpu
@pytest.mark.parametrize("by_heads", [False, True])
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_TC])
def test_delta(cuda_ok, buffer, path, by_heads):
    T, H, d = 80, 3, 64
    off = off_of([9, 71])
    x, randn = make_delta(T, H, H, d, torch.bfloat16, 5)
    do, S0 = randn(T, H, d).bfloat16(), 0.3 * randn(2, H, d, d)
    want = [*bd.delta_forward(*x.values(), off, S_in=S0, path=path), *bd.delta_backward(*x.values(), off, do, S_in=S0, path=path)]
    last = S0.new_zeros(T, H, d, d)
    want.append(bd.delta_step(*x.values(), last.clone()))
    y = [far(buffer, t, by_heads, 128 * i) for i, t in enumerate((*x.values(), do))]
    z = [far(buffer, torch.zeros_like(t), by_heads, 128 * (6 + i)) for i, t in enumerate((x["v"], *x.values()))]
    got = [*bd.delta_forward(*y[:5], off, S_in=S0, out=z[0], path=path)]
    got[0] = got[0].clone()
    got += bd.delta_backward(*y[:5], off, y[5], S_in=S0, dq=z[1], dk=z[2], dv=z[3], dg=z[4], dbeta=z[5], path=path)
    got.append(bd.delta_step(*y[:5], last, out=z[0]))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
