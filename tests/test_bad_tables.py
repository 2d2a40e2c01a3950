"""Offsets and lengths that are out of range: their own sequences are left as
they were, the others are computed as ever, and the status says so."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make as make_delta
from tests.test_packed import make, off_of

FAR = 1 << 30
TABLES = [  # rows, offsets
    (1024, [0, FAR, 64, 192]),
    (1024, [FAR, 0, 700, 1024]),
    (1024, [0, 640, -5, 700, 1024]),
    (1024, [0, -5, 64, 192, 300, FAR, 400, 512, -1]),
    (700, [i * 10 if i % 7 else (-3, FAR, 701)[i % 3] for i in range(71)]),          # every seventh of 70
    (700, [FAR if 20 <= i < 45 else i * 10 for i in range(71)]),                      # many side by side
    (700, [-1] * 40 + [i * 20 for i in range(36)]),
    (2100, [FAR if i in (0, 37, 1050) else i for i in range(2101)]),                  # two rounds of the search
]


def valid(T, offs):
    return [(s, a, b) for s, (a, b) in enumerate(zip(offs, offs[1:])) if 0 <= a <= b <= T]


def table(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows_of(T, seqs):
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    for _, a, b in seqs:
        keep[a:b] = True
    return keep


def check_status():
    assert bd.infini_attn_device_status(None) == bd.INFINI_ERR_OFFSETS
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(len(TABLES)))
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC), (torch.float32, bd.INFINI_PATH_SPLIT),
                                        (torch.bfloat16, bd.INFINI_PATH_SPLIT)])
def test_attention_beside_bad_offsets(cuda_ok, dtype, path, which):
    T, offs = TABLES[which]
    gen = torch.Generator(device="cuda").manual_seed(which)
    q, k, v, do = (make(T, h, 64, dtype, gen) for h in (2, 1, 1, 2))
    seqs = valid(T, offs)
    # the same sequences in a table without bad entries: gaps are the room behind short sequences
    starts, lens = [a for _, a, _ in seqs], [b - a for _, a, b in seqs]
    good, n_len = table(starts + [T]), table(lens)
    new = lambda x: torch.full_like(x, 7.0)  # noqa: E731
    keep = rows_of(T, seqs)
    res = []
    for off, ln in ((good, n_len), (table(offs), None)):
        out, lse = new(q), torch.full((2, T), 7.0, device="cuda")
        bd.packed_forward(q, k, v, off, q_len=ln, out=out, lse=lse, max_q=T, max_k=T, path=path)
        if ln is None:
            check_status()
        r = [out, lse.t()]
        if path != bd.INFINI_PATH_SPLIT:
            r += bd.packed_backward(q, k, v, res[0][0] if res else out, res[0][1].t() if res else lse, do, off, q_len=ln,
                                    dq=new(q), dk=new(k), dv=new(v), path=path)
            if ln is None:
                check_status()
        res.append(r)
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
    for i, (a, b) in enumerate(zip(*res)):
        assert (b[~keep] == 7.0).all(), i
        if path == bd.INFINI_PATH_SPLIT:
            # Its chunks of keys depend on the number of sequences: two roundings of p and two of the result (u each,
            # |v| < 6), or fp32 sums and arguments of exponentials (1e-5 of 1 and of scores below 16) on each side.
            assert (b[keep] - a[keep]).abs().max() <= (4e-4 if dtype == torch.float32 else 4 * 2.0 ** -8 * 6), i
        else:
            assert torch.equal(a[keep], b[keep]), i


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(len(TABLES)))
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
def test_delta_beside_bad_offsets(cuda_ok, dtype, path, which):
    T, offs = TABLES[which]
    n, d = len(offs) - 1, 64
    x, randn = make_delta(T, 1, 2, d, dtype, which)
    do, S0, dS1 = randn(T, 2, d).to(dtype), 0.3 * randn(n, 2, d, d), 0.1 * randn(n, 2, d, d)
    seqs = valid(T, offs)
    at = torch.tensor([s for s, _, _ in seqs], device="cuda")
    good, n_len = table([a for _, a, _ in seqs] + [T]), table([b - a for _, a, b in seqs])
    new = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    keep = rows_of(T, seqs)
    res = []
    for off, ln, S, dS in ((good, n_len, S0[at], dS1[at]), (table(offs), None, S0, dS1)):
        # workspaces full of NaN: what a kernel did not write must not be read
        ws = [torch.full((bd._lib.infini_attn_delta_workspace_size(bd.delta_shape(x["q"], x["v"], off.shape[0] - 1, T), path),),
                         255, dtype=torch.uint8, device="cuda"),
              torch.full((bd._lib.infini_attn_delta_backward_workspace_size(
                  bd.delta_shape(x["q"], x["v"], off.shape[0] - 1, T), path),), 255, dtype=torch.uint8, device="cuda")]
        out, S1 = bd.delta_forward(*x.values(), off, ln, S, max_len=T, out=new(x["v"]), workspace=ws[0], path=path)
        if ln is None:
            check_status()
        g = bd.delta_backward(*x.values(), off, do, ln, S, dS, max_len=T, workspace=ws[1], path=path,
                              **{"d" + m: new(t) for m, t in x.items()})
        if ln is None:
            check_status()
        res.append([out, *g[:5], S1, g[5]])
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK
    for i, (a, b) in enumerate(zip(*res)):
        if i < 6:
            assert torch.equal(a[keep], b[keep]) and (b[~keep] == 7.0).all(), i
        else:
            assert torch.equal(a, b[at]), i
            rest = torch.ones(n, dtype=torch.bool, device="cuda")
            rest[at] = False
            assert torch.equal(b[rest], (S0 if i == 6 else dS1)[rest]), i  # handed through


MIXED = [(i * 37) % 70 * 10 for i in range(70)]
DECREASING = [  # offsets, lengths; the sequences with tokens do not overlap
    ([100, 200, 0, 50], [100, 0, 50]),
    ([0, 100, 50, 200, 260], [50, 0, 150, 60]),
    ([512, 640, 256, 300, 0, 128], [128, 0, 44, 0, 128]),
    (MIXED, [10 if b > a else 0 for a, b in zip(MIXED, MIXED[1:])]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
@pytest.mark.parametrize("offs,lens", DECREASING)
def test_decreasing_offsets(cuda_ok, dtype, path, offs, lens):
    """Each sequence is right or left as it was (its state handed through)."""
    T, d = 1024, 64
    x, randn = make_delta(T, 1, 2, d, dtype, 5)
    n = len(lens)
    S0, ln = 0.3 * randn(n, 2, d, d), table(lens)
    q, k, v = x["q"], x["k"], x["q"]
    ws = torch.full((bd._lib.infini_attn_delta_workspace_size(bd.delta_shape(x["q"], x["v"], n, T), path),), 255,
                    dtype=torch.uint8, device="cuda")
    out, S1 = bd.delta_forward(*x.values(), table(offs), ln, S0, max_len=T, out=torch.full_like(x["v"], 7.0), workspace=ws,
                               path=path)
    check_status()
    o2, lse = torch.full_like(q, 7.0), torch.full((1, T), 7.0, device="cuda")
    bd.packed_forward(q, k, v, table(offs), q_len=ln, out=o2, lse=lse, path=path)
    check_status()
    for s, (a, m) in enumerate(zip(offs, lens)):
        if m == 0:
            continue
        alone, S = bd.delta_forward(*(t[a:a + m] for t in x.values()), off_of([m]), S_in=S0[s:s + 1], max_len=T, path=path)
        w = slice(a, a + m)
        right = torch.equal(out[w], alone) and torch.equal(S1[s], S[0])
        left = (out[w] == 7.0).all() and torch.equal(S1[s], S0[s])
        assert right or left, s
        alone, _ = bd.packed_forward(q[w], k[w], v[w], off_of([m]), path=path)
        assert (((o2[w] == alone) | (o2[w] == 7.0)).all()), s
    assert bd.infini_attn_device_status(None) == bd.INFINI_OK


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 31, 33, 500])
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_TC),
                                        (torch.bfloat16, bd.INFINI_PATH_SPLIT)])
def test_every_bad_entry_is_reported(cuda_ok, dtype, path, n):
    """One bad length or offset, of queries or keys, also in a sequence without rows on the other side."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    T = 4 * n
    q, k, v, do = (make(T, h, 64, dtype, gen) for h in (2, 1, 1, 2))
    off = [4 * i for i in range(n + 1)]
    for s in {0, 1, n // 2, n - 1}:
        for change in ("q_len", "k_len", "q_off", "k_off"):
            for other in (4, 0):  # rows of the sequence on the other side
                t = {"q_off": list(off), "k_off": list(off), "q_len": [4] * n, "k_len": [4] * n}
                t["k_len" if change[0] == "q" else "q_len"][s] = other
                t[change][s] = 5 if change.endswith("len") else FAR
                t = {m: table(y) for m, y in t.items()}
                out, lse = torch.full_like(q, 7.0), torch.full((2, T), 7.0, device="cuda")
                bd.packed_forward(q, k, v, out=out, lse=lse, path=path, **t)
                check_status()
                assert (out[4 * s:4 * s + 4] == 7.0).all() and (lse[:, 4 * s:4 * s + 4] == 7.0).all(), (s, change)
                if path != bd.INFINI_PATH_SPLIT:
                    g = [torch.full_like(y, 7.0) for y in (q, k, v)]
                    bd.packed_backward(q, k, v, out, lse, do, path=path, dq=g[0], dk=g[1], dv=g[2], **t)
                    check_status()
                    assert all((y[4 * s:4 * s + 4] == 7.0).all() for y in g), (s, change)


@pytest.mark.gpu
@pytest.mark.parametrize("change", ["q_len", "k_len", "q_off", "k_off"])
def test_bad_entries_beside_many_keys(cuda_ok, change):
    """So many rows of keys that the tensor-core forward searches for few sequences too."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T = 220000  # 113 MB of keys and values
    q, do = make(300, 2, 128, torch.bfloat16, gen), make(300, 2, 128, torch.bfloat16, gen)
    k = torch.zeros(T, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[:300] = make(300, 1, 128, torch.bfloat16, gen)
    for s in range(3):
        t = {"q_off": [0, 100, 200, 300], "k_off": [0, 100, 200, T], "q_len": [50] * 3, "k_len": [60] * 3}
        t["k_len" if change[0] == "q" else "q_len"][s] = 0
        t[change][s] = 1 << 20
        t = {m: table(y) for m, y in t.items()}
        out, lse = torch.full_like(q, 7.0), torch.full((2, 300), 7.0, device="cuda")
        bd.packed_forward(q, k, k, out=out, lse=lse, max_k=300, path=bd.INFINI_PATH_TC, **t)
        check_status()
        assert (out[100 * s:100 * s + 100] == 7.0).all()
        bd.packed_backward(q, k, k, out, lse, do, path=bd.INFINI_PATH_TC, **t)
        check_status()
