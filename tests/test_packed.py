"""Causal attention over packed sequences with grouped heads, against the
definition in 64 bits.

Bounds are elementwise and come from the roundings: u = half a step of the row
type (2^-8 bf16, 2^-24 fp32), E = 1e-5 for fp32 sums, exponentials and their
arguments (up to a few thousand terms of rounding 2^-24, random in sign). With
A_i = sum_j p_ij |v_j|, every bf16 result is off by at most u for its own
rounding, p by u before its products, D_i by sum_c |dout| (the error of out).
"""
import math

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 1e-5


def off_of(lens, device="cuda", gap=0, first=0):
    o = [first]
    for n in lens:
        o.append(o[-1] + n + gap)
    return torch.tensor(o, dtype=torch.int32, device=device)


def reference(q, k, v, qs, ks, scale, dout=None):
    """qs, ks: (first row, length) of each sequence. Values and bounds in 64 bits; rows of no sequence are NaN."""
    u = U[q.dtype]
    q, k, v = q.double(), k.double(), v.double()
    Hq, Hkv = q.shape[1], k.shape[1]
    G = Hq // Hkv
    nan = lambda x: torch.full_like(x, math.nan)  # noqa: E731
    r = {"out": nan(q), "lse": torch.full((Hq, q.shape[0]), math.nan, dtype=torch.float64, device=q.device)}
    b = {"out": nan(q), "lse": r["lse"].clone()}
    if dout is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            r[n], b[n] = nan(x), nan(x)
    for (a, nq), (c, nk) in zip(qs, ks):
        if dout is not None:
            for n in ("dk", "dv"):
                r[n][c:c + nk] = 0
                b[n][c:c + nk] = 0
        for h in range(Hq):
            Q, K, V = q[a:a + nq, h], k[c:c + nk, h // G], v[c:c + nk, h // G]
            i = torch.arange(nq, device=q.device)[:, None]
            seen = torch.arange(nk, device=q.device)[None, :] <= i + nk - nq
            x = (scale * Q @ K.T).masked_fill(~seen, -math.inf)
            mag = scale * Q.abs() @ K.abs().T
            lse = torch.logsumexp(x, -1) if nk else torch.full((nq,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.where(seen, torch.exp(x - lse.unsqueeze(-1)), 0.0)
            o, A = p @ V, p @ V.abs()
            ex = E * (1 + mag)  # relative error of p
            r["out"][a:a + nq, h], r["lse"][h, a:a + nq] = o, lse
            bo = u * o.abs() + u * A + (p * ex) @ V.abs() + E * A
            b["out"][a:a + nq, h] = bo
            b["lse"][h, a:a + nq] = torch.where(seen, ex, 0.0).amax(-1) + E * lse.abs().clamp(max=1e30) if nk else 0.0
            if dout is None:
                continue
            dO = dout[a:a + nq, h].double()
            D, eD = (dO * o).sum(-1, keepdim=True), (dO.abs() * bo).sum(-1, keepdim=True)
            dp, dpm = dO @ V.T, dO.abs() @ V.abs().T
            ds = scale * p * (dp - D)
            e_ds = u * ds.abs() + scale * p * (eD + E * (dpm + D.abs())) + ex * ds.abs()
            g = {"dq": ds @ K, "dk": ds.T @ Q, "dv": p.T @ dO}
            e = {"dq": e_ds @ K.abs() + E * ds.abs() @ K.abs(), "dk": (e_ds + E * ds.abs()).T @ Q.abs(),
                 "dv": ((u + E + ex) * p).T @ dO.abs()}
            r["dq"][a:a + nq, h], b["dq"][a:a + nq, h] = g["dq"], e["dq"] + u * g["dq"].abs()
            for n in ("dk", "dv"):
                r[n][c:c + nk, h // G] += g[n]
                b[n][c:c + nk, h // G] += e[n]
    if dout is not None:
        for n in ("dk", "dv"):
            b[n] += u * r[n].abs()
    return r, b


def close(name, got, ref, bound):
    got = got.double()
    own = ~torch.isnan(ref)
    g, w, e = got[own], ref[own], bound[own]
    inf = torch.isinf(w)
    assert torch.equal(g[inf], w[inf]), name + ": infinities"
    g, w, e = g[~inf], w[~inf], e[~inf]
    bad = ~((g - w).abs() <= e + 1e-30)
    assert not bad.any(), "%s: %d of %d off, worst %.2f of its bound" % (
        name, int(bad.sum()), bad.numel(), float(((g - w).abs() / (e + 1e-30)).nan_to_num(1e9).max()))


def make(T, H, d, dtype, gen):
    return torch.randn(T, H, d, generator=gen, device="cuda").to(dtype)


def run_case(lens_q, lens_k, Hq, Hkv, d, dtype, path, backward=True, gap=0, scale=None, seed=0, max_q=None, max_k=None,
             fused=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    scale = d ** -0.5 if scale is None else scale
    q_off, k_off = off_of(lens_q, gap=gap, first=gap), off_of(lens_k, gap=gap, first=gap)
    Tq, Tk = int(q_off[-1]) + gap, int(k_off[-1]) + gap
    if fused:
        x = make(Tq, Hq + 2 * Hkv, d, dtype, gen)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = make(Tq, Hq, d, dtype, gen), make(Tk, Hkv, d, dtype, gen), make(Tk, Hkv, d, dtype, gen)
    dout = make(Tq, Hq, d, dtype, gen)
    q_len = k_len = None
    if gap:  # what lies behind a sequence is not read
        q_len, k_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens_q, lens_k))
        for t, off, lens in ((q, q_off, lens_q), (dout, q_off, lens_q), (k, k_off, lens_k), (v, k_off, lens_k)):
            keep = torch.zeros(t.shape[0], dtype=torch.bool, device="cuda")
            for a, n in zip(off.tolist(), lens):
                keep[a:a + n] = True
            t[~keep] = math.nan
    out, lse = torch.full_like(dout, 7.0), torch.full((Hq, Tq), 7.0, device="cuda")
    bd.packed_forward(q, k, v, q_off, k_off, q_len, k_len, max_q, max_k, scale, out, lse, path=path)
    grads = ()
    if backward:
        grads = tuple(torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for x in (q, k, v))
        bd.packed_backward(q, k, v, out, lse, dout, q_off, k_off, q_len, k_len, max_q, max_k, scale, *grads,
                           path=bd.INFINI_PATH_AUTO if path == bd.INFINI_PATH_SPLIT else path)
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
    ref, bound = reference(q, k, v, list(zip(q_off.tolist(), lens_q)), list(zip(k_off.tolist(), lens_k)), scale,
                           dout if backward else None)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        close(name, x, ref[name], bound[name])
        assert (x[torch.isnan(ref[name])] == 7.0).all(), name + ": a row of no sequence was written"


LENS = [
    ([1], [1]),
    ([5], [5]),
    ([128], [128]),
    ([129], [129]),
    ([257, 1, 0, 63, 64, 65], [257, 1, 0, 63, 64, 65]),
    ([3, 40, 1, 200], [130, 40, 77, 500]),        # queries at the end of longer keys
    ([70, 9, 300, 4], [20, 0, 290, 4]),           # more queries than keys: rows that see nothing
    ([0, 0, 384], [0, 17, 384]),
]
TYPES = [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_AUTO)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("lens_q,lens_k", LENS)
def test_lengths(cuda_ok, lens_q, lens_k, dtype, path, d):
    run_case(lens_q, lens_k, 4, 2, d, dtype, path, seed=len(lens_q) + d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 8), (6, 2), (16, 1)])
@pytest.mark.parametrize("dtype,path", TYPES)
def test_groups_and_fused_rows(cuda_ok, Hq, Hkv, dtype, path):
    run_case([100, 33], [100, 33], Hq, Hkv, 64, dtype, path, fused=True, seed=Hq)
    run_case([150], [150], Hq, Hkv, 128, dtype, path, fused=True, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_behind_sequences(cuda_ok, dtype, path, d):
    """Gaps (NaN) between, before and behind the sequences: not read, not written."""
    run_case([100, 5, 0, 190], [130, 5, 60, 260], 4, 2, d, dtype, path, gap=29, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (128, 16, 1), (64, 24, 2)])
@pytest.mark.parametrize("lens_q,lens_k", [([1, 1, 1], [1, 700, 0]), ([1] * 5, [3000, 64, 65, 1, 2047]),
                                           ([4, 2, 0, 3], [600, 1, 9, 5000])])
def test_split(cuda_ok, lens_q, lens_k, d, Hq, Hkv, dtype):
    """Few queries against many keys, with the hints right, absent and too small."""
    for mq, mk in ((max(lens_q), max(lens_k)), (None, None), (1, 100)):
        run_case(lens_q, lens_k, Hq, Hkv, d, dtype, bd.INFINI_PATH_SPLIT, backward=False, max_q=mq, max_k=mk, seed=d)
    run_case(lens_q, lens_k, Hq, Hkv, d, dtype, bd.INFINI_PATH_AUTO, backward=False, max_q=max(lens_q),
             max_k=max(lens_k), seed=d, gap=7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
def test_large_scores(cuda_ok, dtype, path):
    """Scores far from zero in both directions: the running maximum carries them."""
    run_case([200], [200], 2, 1, 64, dtype, path, scale=3.0, seed=8)


@pytest.mark.gpu
def test_many_sequences(cuda_ok):
    """More sequences than one round of the slot search covers."""
    lens = [(i * 37) % 50 for i in range(1500)]
    for dtype in (torch.float32, torch.bfloat16):
        run_case(lens, lens, 2, 1, 64, dtype, bd.INFINI_PATH_AUTO, seed=4)


@pytest.mark.gpu
def test_head_major_rows_and_another_stream(cuda_ok):
    """[H, T, d] buffers passed transposed, on a side stream, captured and replayed on new inputs."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, H, d = 300, 4, 128
    off = off_of([100, 200])
    q, k, v, do = (make(H, T, d, torch.bfloat16, gen).transpose(0, 1) for _ in range(4))
    out = torch.empty(H, T, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.empty(H, T, device="cuda")
    g = [torch.empty_like(out) for _ in range(3)]
    ws = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()

    def step():
        bd.packed_forward(q, k, v, off, out=out, lse=lse, workspace=ws[0])
        bd.packed_backward(q, k, v, out, lse, do, off, dq=g[0], dk=g[1], dv=g[2], workspace=ws[1])

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for x in (q, k, v, do):
        x.copy_(make(T, H, d, torch.bfloat16, gen))
    graph.replay()
    torch.cuda.synchronize()
    seqs = [(0, 100), (100, 200)]
    ref, bound = reference(q, k, v, seqs, seqs, d ** -0.5, do)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        close(name, x, ref[name], bound[name])
    again = [x.clone() for x in (out, lse, *g)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, (out, lse, *g)))


@pytest.mark.gpu
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_AUTO])
def test_gradient_against_differences(cuda_ok, path):
    """fp32: the gradients against central differences of the library's own forward. The difference of the
    loss in 64 bits over steps of 2^-6 is off by the third derivative (below 2^-12 / 6 of values near one) and
    by the forward's rounding, 2^-24 times sqrt(n) over the step: 5e-3 of the gradient's size covers both."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    off = off_of([37, 20])
    x = [make(57, h, 64, torch.float32, gen) for h in (4, 2, 2)]
    do = make(57, 4, 64, torch.float32, gen)
    out, lse = bd.packed_forward(*x, off, path=path)
    grads = bd.packed_backward(*x, out, lse, do, off, path=path)
    h = 2.0 ** -6
    for i in range(3):
        way = make(*x[i].shape, torch.float32, gen)
        way /= way.norm()
        loss = []
        for s in (h, -h):
            y = list(x)
            y[i] = x[i] + s * way
            loss.append((bd.packed_forward(*y, off, path=path)[0].double() * do.double()).sum())
        want, got = float(loss[0] - loss[1]) / (2 * h), float((grads[i].double() * way.double()).sum())
        assert abs(want - got) <= 5e-3 * float(grads[i].norm()), (i, want, got)


@pytest.mark.gpu
def test_bad_offsets_are_reported(cuda_ok):
    """Offsets out of range or decreasing: no access out of range, the other sequences right, the status says so."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (make(64, 2, 64, torch.bfloat16, gen) for _ in range(3))
    for offs in ([0, 30, 99], [0, 40, 20], [-5, 30, 64], [0, 1 << 30, 64]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        for path in (bd.INFINI_PATH_SIMT, bd.INFINI_PATH_SPLIT, bd.INFINI_PATH_AUTO):
            bd.packed_forward(q, k, v, off, path=path)
            assert bd.infini_attn_device_status(None) == bd.INFINI_ERR_OFFSETS
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK


# ------------------------------------------------------------------ refusals
def shape(**kw):
    a = dict(n_seq=2, Tq=8, Tk=8, Hq=4, Hkv=2, d=64, max_q=8, max_k=8, dtype=bd.INFINI_BF16, scale=0.125)
    a.update(kw)
    return bd.infini_packed_shape(*(a[n] for n, _ in bd.infini_packed_shape._fields_))


def raw_forward(s, **kw):
    """The C call on made-up pointers that the checks refuse."""
    row = lambda p, H: bd.infini_rows(p, H * s.d, s.d)  # noqa: E731
    a = dict(q=row(0x10000000, 4), k=row(0x20000000, 2), v=row(0x30000000, 2), q_off=0x40000000, k_off=0x40001000,
             out=row(0x50000000, 4), lse=0x60000000, ws=0x70000000, nbytes=1 << 30, path=0)
    a.update(kw)
    return bd._lib.infini_attn_packed_forward(s, a["q"], a["k"], a["v"], a["q_off"], a["k_off"], None, None, a["out"],
                                              a["lse"], a["ws"], a["nbytes"], a["path"], None)


@pytest.mark.parametrize("change,code", [
    (dict(Hq=3), bd.INFINI_ERR_SHAPE), (dict(Hkv=0), bd.INFINI_ERR_SHAPE), (dict(Tq=-1), bd.INFINI_ERR_SHAPE),
    (dict(n_seq=-1), bd.INFINI_ERR_SHAPE), (dict(d=96), bd.INFINI_ERR_UNSUPPORTED),
    (dict(dtype=2), bd.INFINI_ERR_UNSUPPORTED), (dict(scale=0.0), bd.INFINI_ERR_UNSUPPORTED),
    (dict(scale=math.nan), bd.INFINI_ERR_UNSUPPORTED), (dict(scale=math.inf), bd.INFINI_ERR_UNSUPPORTED),
    (dict(Tk=1 << 30), bd.INFINI_ERR_SIZE), (dict(Hq=1 << 17), bd.INFINI_ERR_SIZE),
])
def test_shape_refusals(change, code):
    s = shape(**change)
    assert raw_forward(s) == code
    assert bd._lib.infini_attn_packed_workspace_size(s, 0) == 0


def test_argument_refusals():
    s, R = shape(), bd.infini_rows
    cases = [
        (dict(q=R(None, 256, 64)), bd.INFINI_ERR_NULL), (dict(q_off=None), bd.INFINI_ERR_NULL),
        (dict(ws=None, path=bd.INFINI_PATH_SPLIT), bd.INFINI_ERR_NULL), (dict(ws=0x70000010), bd.INFINI_ERR_ALIGN),
        (dict(nbytes=16), bd.INFINI_ERR_WORKSPACE), (dict(q=R(0x10000002, 256, 64)), bd.INFINI_ERR_ALIGN),
        (dict(k=R(0x20000000, 132, 64)), bd.INFINI_ERR_ALIGN), (dict(k=R(0x20000000, 0, 64)), bd.INFINI_ERR_SHAPE),
        (dict(out=R(0x10000000, 256, 64)), bd.INFINI_ERR_ALIAS), (dict(out=R(0x50000000, 128, 64)), bd.INFINI_ERR_ALIAS),
        (dict(lse=0x50000000), bd.INFINI_ERR_ALIAS), (dict(path=9), bd.INFINI_ERR_UNSUPPORTED),
        (dict(ws=0x20000000), bd.INFINI_ERR_ALIAS),
        # out inside the gaps of q's rows is not an overlap with q, but this one is with k's
        (dict(q=R(0x10000000, 1024, 64), out=R(0x10000000 + 256 * 2, 1024, 64), k=R(0x10000000 + 512 * 2, 1024, 64),
              v=R(0x10000000 + 480 * 2, 1024, 64)), bd.INFINI_ERR_ALIAS),
    ]
    for kw, code in cases:
        assert raw_forward(s, **kw) == code, kw


def test_select_path():
    sel = bd._lib.infini_attn_packed_select_path
    assert sel(shape(dtype=bd.INFINI_F32, max_q=500, max_k=500)) == bd.INFINI_PATH_SIMT
    assert sel(shape(max_q=1, max_k=4000)) == bd.INFINI_PATH_SPLIT
    assert sel(shape(max_q=33, max_k=4000)) == bd.INFINI_PATH_TC    # 66 rows for a key head
    assert sel(shape(max_q=500, max_k=500, Tk=0)) == bd.INFINI_PATH_SIMT
    assert sel(shape(d=100)) == bd.INFINI_ERR_UNSUPPORTED


def test_any_longest_sequence():
    """The caller's figure may be far off: it chooses a path and a split, and neither overflows."""
    sel, size = bd._lib.infini_attn_packed_select_path, bd._lib.infini_attn_packed_workspace_size
    for huge in (1 << 33, (1 << 62) + 5, (1 << 63) - 1):
        assert sel(shape(max_q=huge, max_k=huge)) == bd.INFINI_PATH_TC
        for q, n_seq in ((1, 1), (1, 500), (huge, 500)):
            a, b = (size(shape(max_q=q, max_k=k, n_seq=n_seq), bd.INFINI_PATH_SPLIT) for k in (huge, 1 << 30))
            assert 0 < a == b


def test_binding_refusals():
    x = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 8], dtype=torch.int32)
    for bad, err in (((x.half(), x, x, off), TypeError), ((x, x[:, :3], x[:, :3], off.long()), TypeError),
                     ((x, x, x[:, :2], off), ValueError), ((x, x.float(), x, off), TypeError),
                     ((x[0], x, x, off), ValueError), ((x, x, x, off[None]), ValueError),
                     ((x, x, x, off, torch.zeros(3, dtype=torch.int32)), ValueError), ((x, x, x, off), ValueError)):
        with pytest.raises(err):
            bd.packed_forward(*bad)
    with pytest.raises(ValueError):
        bd.packed_forward(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2), off)


def test_small_workspaces_are_not_optional():
    """However small the call, a kernel that needs scratch memory is refused without it."""
    s = shape(Tq=1, Tk=1, Hq=1, Hkv=1, n_seq=1)
    need = bd._lib.infini_attn_packed_backward_workspace_size(s)
    assert need > 256 and bd._lib.infini_attn_packed_workspace_size(s, bd.INFINI_PATH_SPLIT) > 256
    assert bd._lib.infini_attn_packed_workspace_size(s, bd.INFINI_PATH_SIMT) == 256
    row = lambda p: bd.infini_rows(p << 28, 64, 64)  # noqa: E731
    for ws, nbytes, code in ((None, need, bd.INFINI_ERR_NULL), (0xF0000000, need - 1, bd.INFINI_ERR_WORKSPACE)):
        assert bd._lib.infini_attn_packed_backward(s, row(1), row(2), row(3), row(4), 5 << 28, row(6), 7 << 28, 7 << 28, None,
                                                   None, row(8), row(9), row(10), ws, nbytes, 0, None) == code


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_AUTO])
def test_nothing_on_one_side(cuda_ok, dtype, path):
    """No sequence, no query, no key: what exists is written (zeros, -inf), nothing else."""
    new = lambda *s: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    zero, some = off_of([0, 0]), off_of([3, 70])
    for q_off, k_off, Tq, Tk in ((zero, zero, 0, 0), (some, zero, 73, 0), (zero, some, 0, 73), (off_of([]), off_of([]), 5, 5)):
        q, k, v, do = new(Tq, 4, 64), new(Tk, 2, 64), new(Tk, 2, 64), new(Tq, 4, 64)
        out, lse = bd.packed_forward(q, k, v, q_off, k_off, out=new(Tq, 4, 64), lse=torch.full((4, Tq), 7.0, device="cuda"),
                                     path=path)
        g = bd.packed_backward(q, k, v, out, lse, do, q_off, k_off, dq=new(Tq, 4, 64), dk=new(Tk, 2, 64), dv=new(Tk, 2, 64),
                               path=path)
        assert bd.infini_attn_device_status(None) == bd.INFINI_OK
        left = q_off.shape[0] == 1  # no sequence: every row is left as it was
        assert all((x == (7.0 if left else 0.0)).all() for x in (out, *g))
        assert (lse == (7.0 if left else -math.inf)).all()


@pytest.mark.gpu
def test_fused_gradients_and_more_queries_than_hinted(cuda_ok):
    """dq, dk, dv as slices of one buffer; the split path with long queries (several row tiles) and wrong hints."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    lens, Hq, Hkv, d = [200, 57], 6, 2, 128
    off, T = off_of(lens), sum(lens)
    x = make(T, Hq + 2 * Hkv, d, torch.bfloat16, gen)
    dx = torch.full_like(x, 7.0)
    cut = lambda t: (t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:])  # noqa: E731
    do = make(T, Hq, d, torch.bfloat16, gen)
    out, lse = bd.packed_forward(*cut(x), off)
    dq, dk, dv = bd.packed_backward(*cut(x), out, lse, do, off, dq=cut(dx)[0], dk=cut(dx)[1], dv=cut(dx)[2])
    seqs = list(zip(off.tolist(), lens))
    ref, bound = reference(*cut(x), seqs, seqs, d ** -0.5, do)
    for name, y in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, dq, dk, dv)):
        close(name, y, ref[name], bound[name])
    for dtype in (torch.float32, torch.bfloat16):
        run_case([90, 5], [300, 700], 6, 2, 64, dtype, bd.INFINI_PATH_SPLIT, backward=False, max_q=1, max_k=1, seed=2)
        run_case([90, 5], [300, 700], 6, 2, 64, dtype, bd.INFINI_PATH_SPLIT, backward=False, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_odd_groups_long_rows(cuda_ok, d):
    """Several tiles of 128 on both sides with groups of 3 and 5 (heads shared unevenly by two CTAs) and of 1."""
    for Hq, Hkv in ((3, 1), (5, 1), (2, 2)):
        run_case([700, 300], [700, 420], Hq, Hkv, d, torch.bfloat16, bd.INFINI_PATH_TC, seed=d + Hq)


@pytest.mark.gpu
def test_two_streams_at_once(cuda_ok):
    """Calls in flight on two streams (a workspace each) do not disturb each other."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    off = off_of([1000, 500])
    sets = [tuple(make(1500, h, 128, torch.bfloat16, gen) for h in (8, 2, 2, 8)) for _ in range(2)]

    def step(x):
        out, lse = bd.packed_forward(*x[:3], off)
        return (out, lse, *bd.packed_backward(*x[:3], out, lse, x[3], off))

    want = [step(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(sets[i])
    torch.cuda.synchronize()
    # the argument instead of the context, as a stream and as a raw handle
    for st in (streams[0], streams[0].cuda_stream):
        out, lse = bd.packed_forward(*sets[0][:3], off, stream=st)
        g = bd.packed_backward(*sets[0][:3], out, lse, sets[0][3], off, stream=st)
        streams[0].synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want[0], (out, lse, *g)))
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
