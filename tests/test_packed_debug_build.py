"""The packed operators in the debug build (INFINI_DEBUG): every row that their
kernels address through a tensor's strides is checked against the tensor. Odd
shapes on every path leave the status clean and give the regular build's bits."""
import ctypes

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from compressive_memory_segment_b200 import build as b
from tests.test_delta import make as make_delta
from tests.test_packed import make, off_of


@pytest.fixture
def debug(monkeypatch):
    """Switches the binding to the debug build and back; reads its status word."""
    typed = bd.open_library(b.build(debug=True))
    lean = ctypes.CDLL(b.DEBUG_LIB)
    for name in [n for n in vars(bd._lean) if n.startswith("infini_attn_")]:
        regular, fn = getattr(bd._lean, name), getattr(lean, name)
        fn.argtypes, fn.restype = regular.argtypes, regular.restype

    def run(fn):
        with monkeypatch.context() as m:
            m.setattr(bd, "_lean", lean)
            res = fn()
        torch.cuda.synchronize()
        assert typed.infini_attn_device_status(torch.cuda.current_stream().cuda_stream) == bd.INFINI_OK
        return res
    return run


def same(a, b):
    return all(torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0)) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.float32, bd.INFINI_PATH_SPLIT),
                                        (torch.bfloat16, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SPLIT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
@pytest.mark.parametrize("lens_q,lens_k", [([1], [1]), ([129, 0, 5], [129, 0, 5]), ([3, 70, 1], [300, 20, 0]),
                                           ([i % 5 for i in range(40)], [i % 7 for i in range(40)])])
def test_attention(cuda_ok, debug, lens_q, lens_k, dtype, path, d):
    gen = torch.Generator(device="cuda").manual_seed(d)
    q_off, k_off = off_of(lens_q), off_of(lens_k)
    q, do = (make(sum(lens_q), 6, d, dtype, gen) for _ in range(2))
    k, v = (make(sum(lens_k), 2, d, dtype, gen) for _ in range(2))

    def run():
        r = list(bd.packed_forward(q, k, v, q_off, k_off, path=path))
        return r if path == bd.INFINI_PATH_SPLIT else r + list(bd.packed_backward(q, k, v, *r, do, q_off, k_off, path=path))
    assert same(run(), debug(run))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
@pytest.mark.parametrize("lens", [[1], [70, 0, 5], [130], [i % 9 for i in range(40)]])
def test_delta(cuda_ok, debug, lens, dtype, path, d):
    x, randn = make_delta(sum(lens), 2, 4, d, dtype, d)
    off, do, S0 = off_of(lens), randn(sum(lens), 4, d).to(dtype), 0.3 * randn(len(lens), 4, d, d)

    def run():
        r = [*bd.delta_forward(*x.values(), off, S_in=S0, max_len=max(lens), path=path)]
        r += bd.delta_backward(*x.values(), off, do, S_in=S0, dS_out=S0, path=path)
        one = [t[:1] for t in x.values()]
        return r + [bd.delta_step(*one, S0[:1].clone())]
    assert same(run(), debug(run))
