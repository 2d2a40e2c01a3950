"""The polynomial exponential of the packed attention gradients, in the steps and
the fp32 roundings of the kernel, with the constants that stand in its source."""
import os
import re

import numpy as np

from compressive_memory_segment_b200 import build as b

f32, f64 = np.float32, np.float64


def constants():
    with open(os.path.join(b.CSRC, "packed_tc_bwd_kernels.cuh")) as f:
        body = f.read().split("void exp2_poly(")[1].split("\n}\n")[0]
    return [f32(x) for x in re.findall(r"f32x2\((0\.\d+)f, \1f\)", body)]


def fma(a, x, y):
    return (a.astype(f64) * x.astype(f64) + np.asarray(y, f64)).astype(f32)  # the product is exact in 64 bits


def exp2(x, c):
    x = np.where(np.isnan(x), x, np.maximum(x, f32(-125))).astype(f32)
    r = (x + f32(12582912)).astype(f32)
    n = (r - f32(12582912)).astype(f32)
    f = fma(n, np.full_like(x, -1), x)
    p = np.full_like(x, c[0])
    for k in c[1:]:
        p = fma(p, f, k)
    scale = ((r.view(np.uint32) << np.uint32(23)) + np.uint32(0x3F800000)).view(f32)
    with np.errstate(invalid="ignore"):
        return p * scale


def test_error_and_ends():
    c = constants()
    assert len(c) == 5
    x = np.concatenate([np.linspace(-126, 1, 400001), np.arange(-125, 2) + 0.5, np.arange(-125, 2) - 0.5]).astype(f32)
    want = np.exp2(np.maximum(x, -125).astype(f64))
    err = np.abs(exp2(x, c).astype(f64) / want - 1)
    # the polynomial's own error, in 64 bits, and a rounding of 2^-24 for each of its five steps
    f = np.linspace(-0.5, 0.5, 200001)
    own = np.abs(np.polyval([float(k) for k in c], f) / np.exp2(f) - 1).max()
    assert own < 2.7e-6 and err.max() < own + 5 * 2.0 ** -24, (own, err.max())
    assert exp2(f32([0.0, -1.0, -125.0, -200.0, -np.inf]), c).tolist()[2:] == [exp2(f32([-125.0]), c)[0]] * 3
    assert np.isnan(exp2(f32([np.nan]), c)).all()
