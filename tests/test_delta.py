"""The gated delta rule over packed sequences, against its definition token by
token in 64 bits.

Bounds are elementwise. The reference runs the recurrence and its reverse twice:
once on the values, once on their magnitudes (every product and sum with positive
terms), which gives for each result the size `mag` of what is summed into it. A
rounding of one factor to the row type is off by at most u = 2^-8 (bf16) of the
terms it enters; fp32 factors, sums and exponentials are covered by E = 1e-5 of
them. The chunked form rounds at most N = 4 factors on the way to a bf16 result
(a state, a pseudo-value, a score, a gradient of one of these) besides the
result itself. On the way to a state or a state's gradient a factor is the sum of
two bf16, the second the rounded rest of the first: off by at most u^2 = 2^-16.
There are five such errors to a term (the earlier state where it meets k; the
inverse and the pseudo-values it is applied to, and their product of second
parts, which is left out; the result where it meets k again), so P = 5 u^2.
"""
import math

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_packed import close, off_of

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E, N, P = 1e-5, 4, 5 * 2.0 ** -16


def recur(q, k, v, a, b, S, scale, sign):
    """One sequence and head in 64 bits; sign -1: the recurrence, +1: its magnitudes. Returns out, S, per-token states."""
    out, kept = torch.zeros_like(v), []
    for t in range(q.shape[0]):
        Sd = S * a[t]
        err = v[t] + sign * (k[t] @ Sd)
        S = Sd + torch.outer(k[t], b[t] * err)
        out[t] = scale * (q[t] @ S)
        kept.append((Sd, err, S))
    return out, S, kept


def reverse(q, k, v, a, b, do, dS, scale, kept, sign):
    g = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", a), ("dbeta", b))}
    for t in reversed(range(q.shape[0])):
        Sd, err, S = kept[t]
        g["dq"][t] = scale * (S @ do[t])
        X = dS + scale * torch.outer(q[t], do[t])
        du = k[t] @ X
        g["dbeta"][t] = du @ err
        g["dv"][t] = b[t] * du
        g["dk"][t] = X @ (b[t] * err) + sign * (Sd @ (b[t] * du))
        X = X + sign * torch.outer(k[t], b[t] * du)
        g["dg"][t] = (X * Sd).sum()
        dS = X * a[t]
    g["dS"] = dS
    return g


def reference(x, seqs, S0, scale, do=None, dS1=None):
    dtype, u = x["q"].dtype, U[x["q"].dtype]
    x = {n: t.double().cpu() for n, t in x.items()}
    T, Hv = x["v"].shape[:2]
    d, G = x["q"].shape[2], Hv // x["q"].shape[1]
    n_seq = len(seqs)
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    r = {"out": nan(T, Hv, d), "S": torch.zeros(n_seq, Hv, d, d, dtype=torch.float64)}
    if do is not None:
        r.update(dq=nan(*x["q"].shape), dk=nan(*x["q"].shape), dv=nan(T, Hv, d), dg=nan(T, Hv), dbeta=nan(T, Hv),
                 dS=torch.zeros(n_seq, Hv, d, d, dtype=torch.float64))
    mag = {n: t.clone() for n, t in r.items()}
    for s, (first, n) in enumerate(seqs):
        w = slice(first, first + n)
        if do is not None:
            for m in (r, mag):
                m["dq"][w] = 0
                m["dk"][w] = 0
        for h in range(Hv):
            one = [x["q"][w, h // G], x["k"][w, h // G], x["v"][w, h], x["g"][w, h].clamp(min=-200).exp(), x["beta"][w, h]]
            S = torch.zeros(d, d, dtype=torch.float64) if S0 is None else S0[s, h].double().cpu()
            for m, sign, args, St in ((r, -1, one, S), (mag, 1, [t.abs() for t in one], S.abs())):
                c = scale if sign < 0 else abs(scale)
                o, Sn, kept = recur(*args, St, c, sign)
                m["out"][w, h], m["S"][s, h] = o, Sn
                if do is not None:
                    dO, dS = do[w, h].double().cpu(), torch.zeros(d, d, dtype=torch.float64)
                    if dS1 is not None:
                        dS = dS1[s, h].double().cpu()
                    g = reverse(*args, dO if sign < 0 else dO.abs(), dS if sign < 0 else dS.abs(), c, kept, sign)
                    m["dq"][w, h // G] += g["dq"]
                    m["dk"][w, h // G] += g["dk"]
                    m["dv"][w, h], m["dg"][w, h], m["dbeta"][w, h], m["dS"][s, h] = (g["dv"], g["dg"], g["dbeta"], g["dS"])
    few, two = (N * u, P) if dtype == torch.bfloat16 else (0.0, 0.0)
    bound = {n: ((two + E) * mag[n] if n in ("S", "dS") else u * r[n].abs() + (few + E) * mag[n]) for n in r}
    return r, bound


def make(T, Hk, Hv, d, dtype, seed, strong=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = torch.nn.functional.normalize
    x = {"q": unit(randn(T, Hk, d), dim=-1), "k": unit(randn(T, Hk, d), dim=-1), "v": randn(T, Hv, d),
         "g": -torch.exp(randn(T, Hv) * (2.0 if strong else 1.0) - (1.0 if strong else 3.0)),
         "beta": torch.sigmoid(2 * randn(T, Hv))}
    return {n: t.to(dtype) for n, t in x.items()}, randn


def run_case(lens, Hk, Hv, d, dtype, path, seed=0, state=True, backward=True, gap=0, scale=None, edit=None, strong=False):
    off = off_of(lens, gap=gap, first=gap)
    T, n = int(off[-1]) + gap, len(lens)
    scale = d ** -0.5 if scale is None else scale
    x, randn = make(T, Hk, Hv, d, dtype, seed, strong)
    if edit:
        edit(x)
    seq_len = None
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    do = randn(T, Hv, d).to(dtype)
    if gap:
        seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        keep[:] = False
        for a, m in zip(off.tolist(), lens):
            keep[a:a + m] = True
        for t in (*x.values(), do):
            t[~keep] = math.nan
    S0 = 0.3 * randn(n, Hv, d, d) if state else None
    dS1 = 0.1 * randn(n, Hv, d, d) if state else None
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], off)
    out, S = bd.delta_forward(*args, seq_len, S0, scale, max(lens, default=0), out=torch.full_like(x["v"], 7.0), path=path)
    got = {"out": out, "S": S}
    if backward:
        new = {m: torch.full_like(x[m[1:]], 7.0) for m in ("dq", "dk", "dv", "dg", "dbeta")}
        g = bd.delta_backward(*args, do, seq_len, S0, dS1, scale, max(lens, default=0), **new, path=path)
        got.update(zip(("dq", "dk", "dv", "dg", "dbeta", "dS"), g))
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
    ref, bound = reference(x, list(zip(off.tolist(), lens)), S0, scale, do if backward else None, dS1)
    for name, y in got.items():
        close(name, y.cpu(), ref[name], bound[name])
        assert (y.cpu()[torch.isnan(ref[name])] == 7.0).all(), name + ": a row of no sequence was written"


TYPES = [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_AUTO)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("lens", [[1], [2, 0, 1], [63, 65], [64], [130, 32, 31, 33], [0], [200]])
def test_lengths(cuda_ok, lens, dtype, path, d):
    run_case(lens, 1, 2, d, dtype, path, seed=sum(lens) + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", TYPES)
def test_short_and_long_sequences_together(cuda_ok, dtype, path, d):
    """Token by token and in chunks in one launch, at both sides of the length that parts them."""
    run_case([48, 49, 1, 97, 0, 47], 2, 4, d, dtype, path, seed=d, gap=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 2), (1, 3), (2, 8)])
def test_heads(cuda_ok, Hk, Hv, dtype, path):
    run_case([40, 70], Hk, Hv, 64, dtype, path, seed=Hv)
    run_case([67], Hk, Hv, 128, dtype, path, seed=Hv, state=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
def test_rows_behind_sequences(cuda_ok, dtype, path):
    run_case([70, 0, 5, 64], 1, 2, 64, dtype, path, gap=13, seed=9)
    run_case([70, 3], 1, 1, 128, dtype, path, gap=70, seed=9)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
def test_gates_at_their_ends(cuda_ok, dtype, path):
    """No decay, decays to nothing (a reset) and just short of it, writes of strength 0 and 1."""
    def edit(x):
        x["g"][3::7] = -math.inf
        x["g"][5::11] = 0.0
        x["g"][8::13] = -90.0
        x["g"][20:24] = -300.0
        x["beta"][2::5] = 0.0
        x["beta"][4::9] = 1.0

    run_case([150, 70], 1, 2, 64, dtype, path, seed=21, edit=edit, strong=True)
    run_case([130], 1, 1, 128, dtype, path, seed=22, edit=edit, strong=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
@pytest.mark.parametrize("at", range(8))
def test_gradient_of_a_strong_decay(cuda_ok, dtype, path, at):
    """What passes such a decay is tiny beside what follows it: its gradient keeps its own digits, at each place of a tile."""
    def edit(x):  # all tokens share one key: the terms are as large as their magnitudes
        x["q"][:] = x["k"][:] = x["k"].shape[-1] ** -0.5
        x["v"].abs_()
        x["beta"][:] = 0.125
        x["g"][at::8] = -18.0

    run_case([140, 3], 1, 2, 64, dtype, path, seed=30 + at, edit=edit, state=False)


@pytest.mark.gpu
def test_negative_scale(cuda_ok):
    run_case([70, 3], 1, 2, 64, torch.bfloat16, bd.INFINI_PATH_AUTO, seed=5, scale=-0.5)
    run_case([3, 5], 1, 2, 64, torch.float32, bd.INFINI_PATH_AUTO, seed=5, scale=-0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
def test_one_key_again_and_again(cuda_ok, dtype, path):
    """The same index written many times: every write replaces the last, the solve in a chunk is at its hardest."""
    def edit(x):
        x["k"][:] = x["k"][:1]
        x["g"][:] = 0.0

    run_case([100], 1, 1, 64, dtype, path, seed=23, edit=edit)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES)
def test_pieces_equal_the_whole(cuda_ok, dtype, path):
    """A sequence in two calls, the state updated in place, equals one call: out within two roundings of each
    other (u each, and the states' E), S within twice E of its size."""
    x, randn = make(173, 1, 2, 64, dtype, 31)
    off = off_of([173])
    out, S = bd.delta_forward(*x.values(), off, path=path)
    St, outs = torch.zeros(1, 2, 64, 64, device="cuda"), []
    for a, b in ((0, 100), (100, 173)):
        o, _ = bd.delta_forward(*(t[a:b] for t in x.values()), off_of([b - a]), S_in=St, S_out=St, path=path)
        outs.append(o)
    ref, bound = reference(x, [(0, 173)], None, 64 ** -0.5)
    close("out", torch.cat(outs).cpu(), ref["out"], bound["out"])
    close("S", St.cpu(), ref["S"], bound["S"])
    close("S whole", S.cpu(), ref["S"], bound["S"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,Hk,Hv,d", [(1, 1, 1, 64), (5, 2, 6, 128), (3, 4, 4, 64)])
def test_step(cuda_ok, B, Hk, Hv, d, dtype):
    """One token against the reference, in place and not, and a run of steps against the sequence form."""
    x, randn = make(B, Hk, Hv, d, dtype, 40 + B)
    S = 0.3 * randn(B, Hv, d, d)
    ref, bound = reference(x, [(b, 1) for b in range(B)], S, d ** -0.5)
    S2 = torch.empty_like(S)
    for to in (S2, None):
        out = bd.delta_step(*x.values(), S, S_out=to)
        close("out", out.cpu(), ref["out"], bound["out"])
        close("S", (S if to is None else S2).cpu(), ref["S"], bound["S"])
    T = 70
    x, randn = make(T, Hk, Hv, d, dtype, 50 + B)
    S = torch.zeros(1, Hv, d, d, device="cuda")
    outs = torch.cat([bd.delta_step(*(t[i:i + 1] for t in x.values()), S) for i in range(T)])
    ref, bound = reference(x, [(0, T)], None, d ** -0.5)
    close("outs", outs.cpu(), ref["out"], bound["out"])
    close("S", S.cpu(), ref["S"], bound["S"])


@pytest.mark.gpu
def test_attention_and_memory_together(cuda_ok):
    """The two operators as a hybrid block runs them: packed attention and the delta rule on the same packed
    rows with one offsets tensor, then one more token for each sequence against the cache and the states."""
    d, H, lens = 64, 2, [90, 33, 128]
    x, randn = make(sum(lens) + 3, H, H, d, torch.bfloat16, 60)
    off = off_of(lens)
    T = sum(lens)
    head = {n: t[:T] for n, t in x.items()}
    from tests.test_packed import reference as attention
    out, lse = bd.packed_forward(head["q"], head["k"], head["v"], off, max_q=max(lens), max_k=max(lens))
    mem, S = bd.delta_forward(*head.values(), off)
    seqs = list(zip(off.tolist(), lens))
    r, b = attention(head["q"], head["k"], head["v"], seqs, seqs, d ** -0.5)
    close("out", out, r["out"], b["out"])
    r, b = reference(head, seqs, None, d ** -0.5)
    close("memory", mem.cpu(), r["out"], b["out"])
    cap = 160
    kc, vc = (torch.full((3 * cap, H, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for s, (a, n) in enumerate(seqs):
        for c, t in ((kc, x["k"]), (vc, x["v"])):
            c[s * cap:s * cap + n], c[s * cap + n] = t[a:a + n], t[T + s]
    new = {n: t[T:] for n, t in x.items()}
    one = off_of([1, 1, 1])
    k_len = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")
    out, _ = bd.packed_forward(new["q"], kc, vc, one, one * cap, None, k_len, 1, cap)
    r, b = attention(new["q"], kc, vc, [(s, 1) for s in range(3)], [(s * cap, n + 1) for s, n in enumerate(lens)], d ** -0.5)
    close("step", out, r["out"], b["out"])
    long = {n: torch.cat([torch.cat([t[a:a + m], t[T + s:T + s + 1]]) for s, (a, m) in enumerate(seqs)]) for n, t in x.items()}
    r, b = reference(long, [(a + s, m + 1) for s, (a, m) in enumerate(seqs)], None, d ** -0.5)
    got = bd.delta_step(*new.values(), S)
    last = [a + s + m for s, (a, m) in enumerate(seqs)]
    close("memory step", got.cpu(), r["out"][last], b["out"][last])
    close("S", S.cpu(), r["S"], b["S"])
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK


@pytest.mark.gpu
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_AUTO])
def test_gradient_against_differences(cuda_ok, path):
    """fp32 gradients against central differences of the library's forward along random directions: steps of
    2^-6 and the loss summed in 64 bits leave 5e-3 of the gradient's size (third derivatives and the forward's
    fp32 rounding over the step)."""
    x, randn = make(75, 1, 2, 64, torch.float32, 70)
    off, S0 = off_of([40, 35]), 0.3 * randn(2, 2, 64, 64)
    do, dS1 = randn(75, 2, 64), 0.1 * randn(2, 2, 64, 64)

    def loss(y, S):
        o, Sn = bd.delta_forward(*y.values(), off, S_in=S, path=path)
        return float((o.double() * do.double()).sum() + (Sn.double() * dS1.double()).sum())

    g = bd.delta_backward(*x.values(), off, do, S_in=S0, dS_out=dS1, path=path)
    h = 2.0 ** -6
    for i, name in enumerate(list(x) + ["S"]):
        t = S0 if name == "S" else x[name]
        way = randn(*t.shape)
        way /= way.norm()
        side = []
        for s in (h, -h):
            y = dict(x)
            if name != "S":
                y[name] = t + s * way
            side.append(loss(y, S0 + s * way if name == "S" else S0))
        want, got = (side[0] - side[1]) / (2 * h), float((g[i].double() * way.double()).sum())
        assert abs(want - got) <= 5e-3 * float(g[i].norm()), (name, want, got)


@pytest.mark.gpu
def test_captured_and_repeated(cuda_ok):
    """Forward, backward and step captured on a side stream; replays on new inputs are right and bit for bit the same."""
    x, randn = make(150, 1, 2, 128, torch.bfloat16, 80)
    off, do, S0 = off_of([100, 50]), randn(150, 2, 128).bfloat16(), 0.3 * randn(2, 2, 128, 128)
    shp = bd.delta_shape(x["q"], x["v"], 2)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        bd._lib.infini_attn_delta_workspace_size(shp, 0), bd._lib.infini_attn_delta_backward_workspace_size(shp, 0))]
    res = {}

    def step():
        res["f"] = bd.delta_forward(*x.values(), off, S_in=S0, workspace=ws[0])
        res["b"] = bd.delta_backward(*x.values(), off, do, S_in=S0, workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    y, _ = make(150, 1, 2, 128, torch.bfloat16, 81)
    for n in x:
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    ref, bound = reference(x, [(0, 100), (100, 50)], S0, 128 ** -0.5, do)
    got = dict(zip(("out", "S", "dq", "dk", "dv", "dg", "dbeta", "dS"), (*res["f"], *res["b"])))
    for name, t in got.items():
        close(name, t.cpu(), ref[name], bound[name])
    first = {n: t.clone() for n, t in got.items()}
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], got[n]) for n in got)


# ------------------------------------------------------------------ refusals
def shape(**kw):
    a = dict(n_seq=2, T=8, Hk=2, Hv=4, d=64, max_len=64, dtype=bd.INFINI_BF16, scale=0.125)
    a.update(kw)
    return bd.infini_delta_shape(*(a[n] for n, _ in bd.infini_delta_shape._fields_))


def raw(s, **kw):
    row = lambda p, H, d=64: bd.infini_rows(p, H * d, d)  # noqa: E731
    a = dict(q=row(0x10000000, 2), k=row(0x11000000, 2), v=row(0x12000000, 4), g=row(0x13000000, 4, 1),
             beta=row(0x14000000, 4, 1), off=0x15000000, S_in=0x16000000, out=row(0x17000000, 4), S_out=0x18000000,
             ws=0x20000000, nbytes=1 << 30, path=0)
    a.update(kw)
    return bd._lib.infini_attn_delta_forward(s, a["q"], a["k"], a["v"], a["g"], a["beta"], a["off"], None, a["S_in"],
                                             a["out"], a["S_out"], a["ws"], a["nbytes"], a["path"], None)


@pytest.mark.parametrize("change,code", [
    (dict(Hv=3), bd.INFINI_ERR_SHAPE), (dict(Hk=0), bd.INFINI_ERR_SHAPE), (dict(T=-1), bd.INFINI_ERR_SHAPE),
    (dict(d=32), bd.INFINI_ERR_UNSUPPORTED), (dict(dtype=5), bd.INFINI_ERR_UNSUPPORTED),
    (dict(scale=math.nan), bd.INFINI_ERR_UNSUPPORTED), (dict(T=1 << 30), bd.INFINI_ERR_SIZE),
    (dict(n_seq=1 << 17), bd.INFINI_ERR_SIZE),
])
def test_shape_refusals(change, code):
    s = shape(**change)
    assert raw(s) == code
    assert bd._lib.infini_attn_delta_workspace_size(s, 0) == 0
    assert bd._lib.infini_attn_delta_backward_workspace_size(s, 0) == 0


def test_argument_refusals():
    s, R = shape(), bd.infini_rows
    for kw, code in [
        (dict(q=R(None, 128, 64)), bd.INFINI_ERR_NULL), (dict(off=None), bd.INFINI_ERR_NULL),
        (dict(ws=None), bd.INFINI_ERR_NULL), (dict(nbytes=1), bd.INFINI_ERR_WORKSPACE),
        (dict(v=R(0x12000008, 256, 64)), bd.INFINI_ERR_ALIGN), (dict(g=R(0x13000001, 4, 1)), bd.INFINI_ERR_ALIGN),
        (dict(S_in=0x16000004), bd.INFINI_ERR_ALIGN), (dict(out=R(0x12000000, 256, 64)), bd.INFINI_ERR_ALIAS),
        (dict(S_out=0x16000100), bd.INFINI_ERR_ALIAS), (dict(path=bd.INFINI_PATH_SPLIT), bd.INFINI_ERR_UNSUPPORTED),
        (dict(beta=R(0x14000000, 0, 1)), bd.INFINI_ERR_SHAPE),
    ]:
        assert raw(s, **kw) == code, kw


def test_step_refusals():
    s, R = shape(), bd.infini_rows
    rows = [R(0x10000000, 128, 64), R(0x11000000, 128, 64), R(0x12000000, 256, 64), R(0x13000000, 4, 1), R(0x14000000, 4, 1)]
    step = lambda S, out, S_out: bd._lib.infini_attn_delta_step(s, *rows, S, out, S_out, None)  # noqa: E731
    out = R(0x17000000, 256, 64)
    assert step(None, out, 0x18000000) == bd.INFINI_ERR_NULL
    assert step(0x18000000, out, None) == bd.INFINI_ERR_NULL
    assert step(0x18000000, out, 0x18000100) == bd.INFINI_ERR_ALIAS
    assert step(0x18000000, R(0x12000000, 256, 64), 0x18000000) == bd.INFINI_ERR_ALIAS


def test_binding_refusals():
    q, v, g = (torch.zeros(8, *s, dtype=torch.bfloat16) for s in ((2, 64), (4, 64), (4,)))
    off = torch.tensor([0, 8], dtype=torch.int32)
    for args, err in (((q, q, v, g, g, off.long()), TypeError), ((q, q, v, g.float(), g, off), TypeError),
                      ((q, q, v, g[:, :2], g, off), ValueError), ((q, q, v[:4], g, g, off), ValueError),
                      ((q, q, v, g, g, off), ValueError)):
        with pytest.raises(err):
            bd.delta_forward(*args)
    with pytest.raises(ValueError):
        bd.delta_step(q, q, v, g, g, torch.zeros(8, 4, 64, 32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", TYPES + [(torch.bfloat16, bd.INFINI_PATH_TC)])
def test_many_and_short_sequences(cuda_ok, dtype, path):
    """More sequences than one round of the slot search covers, most of a few tokens (the recurrence's side of
    the choice of path, and the chunked form forced)."""
    run_case([(i * 7) % 9 for i in range(70)], 1, 2, 64, dtype, path, seed=90)
    run_case([8, 3, 1], 2, 4, 128, dtype, path, seed=91, backward=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing(cuda_ok, dtype):
    """No tokens: states are handed through; no sequences: nothing is written."""
    x = {n: torch.zeros(s, dtype=dtype, device="cuda") for n, s in
         (("q", (0, 1, 64)), ("k", (0, 1, 64)), ("v", (0, 2, 64)), ("g", (0, 2)), ("beta", (0, 2)))}
    S = torch.randn(2, 2, 64, 64, device="cuda")
    out, So = bd.delta_forward(*x.values(), off_of([0, 0]), S_in=S)
    assert torch.equal(S, So)
    g = bd.delta_backward(*x.values(), off_of([0, 0]), x["v"], S_in=S, dS_out=S)
    assert torch.equal(g[5], S)
    y, _ = make(5, 1, 2, 64, dtype, 1)
    out = torch.full_like(y["v"], 7.0)
    bd.delta_forward(*y.values(), off_of([]), out=out)
    assert (out == 7.0).all() and bd.infini_attn_device_status(None) == bd.INFINI_OK


@pytest.mark.gpu
@pytest.mark.parametrize("path", [bd.INFINI_PATH_SIMT, bd.INFINI_PATH_AUTO])
def test_strided_rows_and_states_in_place(cuda_ok, path):
    """Slices of fused buffers (v, g and beta beside each other), the gradient of the state in place."""
    T, d = 150, 64
    y, randn = make(T, 1, 2, d, torch.bfloat16, 95)
    qkv = torch.cat([y["q"], y["k"], y["v"]], 1)
    gb = torch.cat([y["g"], y["beta"]], 1)
    x = {"q": qkv[:, :1], "k": qkv[:, 1:2], "v": qkv[:, 2:], "g": gb[:, :2], "beta": gb[:, 2:]}
    off, do, S0, dS = off_of([100, 50]), randn(T, 2, d).bfloat16(), 0.3 * randn(2, 2, d, d), 0.1 * randn(2, 2, d, d)
    ref, bound = reference(x, [(0, 100), (100, 50)], S0, d ** -0.5, do, dS)
    g = bd.delta_backward(*x.values(), off, do, S_in=S0, dS_out=dS, dS_in=dS, path=path)
    out, S = bd.delta_forward(*x.values(), off, S_in=S0, S_out=S0, path=path)
    for name, t in zip(("out", "S", "dq", "dk", "dv", "dg", "dbeta", "dS"), (out, S, *g)):
        close(name, t.cpu(), ref[name], bound[name])


@pytest.mark.gpu
def test_bad_offsets_are_reported(cuda_ok):
    x, randn = make(64, 1, 2, 64, torch.bfloat16, 96)
    for offs in ([0, 30, 99], [0, 40, 20], [-5, 30, 64], [0, 1 << 30, 64]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        for path in (bd.INFINI_PATH_SIMT, bd.INFINI_PATH_TC):
            bd.delta_forward(*x.values(), off, path=path)
            assert bd.infini_attn_device_status(None) == bd.INFINI_ERR_OFFSETS
            bd.delta_backward(*x.values(), off, x["v"], path=path)
            assert bd.infini_attn_device_status(None) == bd.INFINI_ERR_OFFSETS
