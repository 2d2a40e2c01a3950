"""The gated delta rule over many chunks, by norms.

The elementwise bounds of test_delta.py follow magnitudes through the recurrence,
which grow from token to token where the values do not, so that they say little
behind a few dozen tokens. Here the error's norm over a head is held against the
norm of the true result. The recurrence does not enlarge an error (keys of norm
1, 0 <= beta <= 1, decays of at most 1: each token's map of the state has norm 1 or
less), so what is committed in a chunk stays as large as it was:
 * a result in bf16 takes up to N = 4 roundings of factors and its own, u = 2^-8 of
   the terms each; terms and results have comparable norms: 5 u;
 * a state or its gradient takes five errors of 2^-16 of its terms in each chunk,
   random in sign, and a state remembers the last few chunks only at these decays:
   5 times 2^-16 twice over, 1.6e-4;
 * fp32: 1e-5 for the sums, as everywhere, twice over.
`test_the_bounds_can_fail` shows that these bounds notice what could go wrong
between chunks."""
import pytest
import torch

from compressive_memory_segment_b200 import binding as bd
from tests.test_delta import make, recur, reverse
from tests.test_packed import off_of

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS")


def bound(name, dtype):
    if dtype == torch.float32:
        return 2e-5
    return 10 * 2.0 ** -16 if name in ("S", "dS") else 5 * U[dtype]


def truth(x, seqs, S0, dS1, do, scale, forget=0, cut=0):
    """The definition in 64 bits. For the test of the bounds: `forget` starts the state anew every so many tokens,
    `cut` does so with its gradient."""
    x = {n: t.double().cpu() for n, t in x.items()}
    S0, dS1, do = S0.double().cpu(), dS1.double().cpu(), do.double().cpu()
    Hv, G = x["v"].shape[1], x["v"].shape[1] // x["q"].shape[1]
    r = {"out": torch.zeros_like(x["v"]), "S": S0.clone(), "dS": dS1.clone(),
         **{"d" + n: torch.zeros_like(t) for n, t in x.items()}}
    for s, (first, n) in enumerate(seqs):
        for h in range(Hv):
            S, kept = S0[s, h], []
            part = lambda a, b: [t[first + a:first + b, i] for t, i in (  # noqa: E731
                (x["q"], h // G), (x["k"], h // G), (x["v"], h), (x["g"].exp(), h), (x["beta"], h))]
            step = forget or cut or n
            for a in range(0, n, step):
                o, S, k = recur(*part(a, min(n, a + step)), torch.zeros_like(S) if forget and a else S, scale, -1)
                r["out"][first + a:first + a + o.shape[0], h] = o
                kept.append(k)
            r["S"][s, h], dS = S, dS1[s, h]
            for a in reversed(range(0, n, step)):
                w = slice(first + a, first + min(n, a + step))
                g = reverse(*part(a, min(n, a + step)), do[w, h], dS, scale, kept.pop(), -1)
                dS = torch.zeros_like(dS) if cut else g["dS"]
                r["dq"][w, h // G] += g["dq"]
                r["dk"][w, h // G] += g["dk"]
                for m in ("dv", "dg", "dbeta"):
                    r[m][w, h] = g[m]
            r["dS"][s, h] = dS
    return r


def errors(got, want):
    """Largest ratio of norms over the heads."""
    r = {}
    for n, y in want.items():
        x = got[n].double().cpu().transpose(0, 1).flatten(1)
        y = y.transpose(0, 1).flatten(1)
        r[n] = float(((x - y).norm(dim=1) / y.norm(dim=1)).max())
    return r


def inputs(lens, Hk, Hv, d, dtype, seed, device):
    if device == "cuda":
        x, randn = make(sum(lens), Hk, Hv, d, dtype, seed)
    else:
        gen = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        unit, T = torch.nn.functional.normalize, sum(lens)
        x = {"q": unit(randn(T, Hk, d), dim=-1), "k": unit(randn(T, Hk, d), dim=-1), "v": randn(T, Hv, d),
             "g": -torch.exp(randn(T, Hv) - 3.0), "beta": torch.sigmoid(2 * randn(T, Hv))}
        x = {n: t.to(dtype) for n, t in x.items()}
    return x, 0.3 * randn(len(lens), Hv, d, d), 0.1 * randn(len(lens), Hv, d, d), randn(sum(lens), Hv, d).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,path", [(torch.float32, bd.INFINI_PATH_SIMT), (torch.bfloat16, bd.INFINI_PATH_SIMT),
                                        (torch.bfloat16, bd.INFINI_PATH_TC)])
@pytest.mark.parametrize("lens,Hk,Hv,d", [([200], 1, 2, 64), ([130, 33, 193], 1, 2, 64), ([300, 64], 1, 1, 128),
                                          ([700], 2, 2, 64)])
def test_norms(cuda_ok, lens, Hk, Hv, d, dtype, path):
    x, S0, dS1, do = inputs(lens, Hk, Hv, d, dtype, sum(lens), "cuda")
    off = off_of(lens)
    out, S = bd.delta_forward(*x.values(), off, S_in=S0, path=path)
    g = bd.delta_backward(*x.values(), off, do, S_in=S0, dS_out=dS1, path=path)
    got = dict(zip(NAMES, g), out=out, S=S)
    err = errors(got, truth(x, list(zip(off.tolist(), lens)), S0, dS1, do, d ** -0.5))
    assert all(e <= bound(n, dtype) for n, e in err.items()), err


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_bounds_can_fail(dtype):
    """What a broken hand-over between chunks would give, and zeros, lie several times beyond the bounds."""
    lens, d = [130, 200], 32
    x, S0, dS1, do = inputs(lens, 1, 2, d, dtype, 7, "cpu")
    seqs = [(0, 130), (130, 200)]
    want = truth(x, seqs, S0, dS1, do, d ** -0.5)
    for n, e in errors({n: torch.zeros_like(t) for n, t in want.items()}, want).items():
        assert e > 10 * bound(n, dtype), n
    chunk = 64 if dtype == torch.bfloat16 else 32
    e = errors(truth(x, seqs, S0, dS1, do, d ** -0.5, forget=chunk), want)
    assert all(e[n] > 4 * bound(n, dtype) for n in ("out", "S", "dq", "dk", "dg", "dbeta")), e
    e = errors(truth(x, seqs, S0, dS1, do, d ** -0.5, cut=chunk), want)
    assert all(e[n] > 4 * bound(n, dtype) for n in ("dk", "dv", "dg", "dbeta", "dS")), e
    # one term of a gradient left out, and the gates' rows off by one
    assert float((want["dk"] - 0.9 * want["dk"]).norm() / want["dk"].norm()) > bound("dk", dtype)
    late = {**want, "dg": want["dg"].roll(1, 0)}
    assert errors(late, want)["dg"] > 10 * bound("dg", dtype)
