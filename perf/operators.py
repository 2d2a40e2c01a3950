"""Workloads of the packed-sequence operators: causal softmax attention over
packed sequences with grouped heads (a whole prompt, a training step, one new
token against a cache) and the gated delta rule over the same packed sequences
(a whole prompt, a training step, one token against a state).

`run` makes one pass: with `own` false in plain torch operations, with `own`
true through the library's entry points. `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def _prompt(name, op, n_seq, lo, hi, Hq, Hkv, d, dtype, spread, fused=False, capacity=0):
    c = dict(op=op, n_seq=n_seq, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, spread=spread, fused=fused,
             capacity=capacity)
    return dict(c, name=name) if name else c


def _delta(name, op, n_seq, lo, hi, Hk, Hv, d, dtype, spread):
    c = dict(op=op, n_seq=n_seq, lo=lo, hi=hi, Hk=Hk, Hv=Hv, d=d, dtype=dtype, spread=spread)
    return dict(c, name=name) if name else c


def listed():
    return [
        # A handful of short questions that arrive together: latency.
        _prompt("prompt_small", "prompt", 3, 1, 96, 8, 2, 64, "bf16", 1),
        # A batch of prompts of very different lengths, q, k, v in one projection's output.
        _prompt("prompt_ragged", "prompt", 16, 64, 2048, 16, 16, 128, "bf16", 2, fused=True),
        # One long document, an 8B-like layer's heads with grouped keys.
        _prompt("prompt_long", "prompt", 1, 8192, 8192, 32, 8, 128, "bf16", 3),
        # The fp32 path, as numerical checks of a layer use it.
        _prompt("prompt_f32", "prompt", 4, 100, 700, 8, 4, 64, "f32", 4),
        # A training micro-batch of packed documents, forward and backward.
        _prompt("prompt_train", "prompt_train", 6, 200, 2048, 16, 4, 128, "bf16", 5),
        # The same at the small end, with the small head dimension.
        _prompt("prompt_train_small", "prompt_train", 5, 1, 300, 4, 4, 64, "bf16", 6),
        # A serving step: one new token per sequence against caches of different fill.
        _prompt("cache_step", "cache_step", 48, 300, 8192, 32, 8, 128, "bf16", 7, capacity=8192),
        # Short prompts through the delta-rule memory: latency.
        _delta("delta_small", "delta", 4, 1, 150, 4, 8, 64, "bf16", 8),
        # Two long documents through the delta-rule memory, incoming state given.
        _delta("delta_long", "delta", 2, 6000, 8192, 16, 32, 128, "bf16", 9),
        # A training micro-batch through the delta-rule memory, forward and backward.
        _delta("delta_train", "delta_train", 8, 128, 2048, 8, 16, 128, "bf16", 10),
        # The fp32 training path at a check's size.
        _delta("delta_train_f32", "delta_train", 2, 30, 200, 4, 4, 64, "f32", 11),
        # A serving step: one token per sequence, every state read and written.
        _delta("delta_step", "delta_step", 64, 1, 1, 16, 32, 128, "bf16", 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt_train", "cache_step", "delta", "delta", "delta_train", "delta_step"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    spread = rng.randrange(1 << 30)
    group = rng.choice([1, 2, 3, 4, 8])
    if op.startswith("delta"):
        Hk = rng.choice([1, 2, 4, 8])
        Hv = Hk * rng.choice([1, 2, 3])
        if op == "delta_step":
            return _delta(None, op, _log_int(rng, 1, 80), 1, 1, Hk, Hv, d, dtype, spread)
        n = _log_int(rng, 1, 8)
        hi = _log_int(rng, 1, 4000 if op == "delta" else 1500)
        if dtype == "f32":
            hi = min(hi, 400)
        return _delta(None, op, n, max(1, hi // rng.choice([1, 2, 16])), hi, Hk, Hv, d, dtype, spread)
    Hkv = rng.choice([1, 2, 4])
    Hq = Hkv * group
    if op == "cache_step":
        cap = _log_int(rng, 64, 8192)
        return _prompt(None, op, _log_int(rng, 1, 48), max(1, cap // 20), cap, Hq, Hkv, d, dtype, spread, capacity=cap)
    n = _log_int(rng, 1, 12)
    # A training row with a single key has a zero gradient for its query: batches of such rows alone are left out.
    hi = _log_int(rng, 1, 3000) if op == "prompt" else _log_int(rng, 24, 1500)
    if dtype == "f32":
        hi = min(hi, 700)
    return _prompt(None, op, n, max(1, hi // rng.choice([1, 3, 20])), hi, Hq, Hkv, d, dtype, spread,
                   fused=rng.random() < 0.5)


def _lengths(case):
    r = random.Random(case["spread"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    lens[r.randrange(len(lens))] = case["hi"]
    return lens


def work(case):
    lens, d = _lengths(case), case["d"]
    T, e = sum(lens), 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("delta"):
        Hk, Hv = case["Hk"], case["Hv"]
        tok = T * d * e * (2 * Hk + Hv) + 2 * T * Hv * e
        state = case["n_seq"] * Hv * d * d * 4
        bytes_, flops = tok + T * Hv * d * e + 2 * state, 6.0 * T * Hv * d * d
        if case["op"] == "delta_train":
            # out, dout, the gradients of every token input, the state's gradient in and out
            bytes_, flops = bytes_ + T * Hv * d * e + tok + 2 * state, 3 * flops
        return {"bytes": float(bytes_), "flops": flops}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "cache_step":
        n = case["n_seq"]
        return {"bytes": float(2 * T * Hkv * d * e + 2 * n * Hq * d * e + 4 * n * Hq), "flops": 4.0 * T * Hq * d}
    pairs = sum(n * (n + 1) // 2 for n in lens)
    bytes_ = T * d * e * (2 * Hq + 2 * Hkv) + 4 * T * Hq
    flops = 4.0 * pairs * Hq * d
    if case["op"] == "prompt_train":
        bytes_, flops = bytes_ + T * d * e * (2 * Hq + 2 * Hkv), 3.5 * flops
    return {"bytes": float(bytes_), "flops": flops}


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev, dt, d = "cuda", DTYPES[case["dtype"]], case["d"]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    lens, n = _lengths(case), case["n_seq"]
    s = dict(op=case["op"], longest=max(lens), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    s["off"], T = torch.tensor(starts, dtype=torch.int32, device=dev), starts[-1]
    if case["op"].startswith("delta"):
        Hk, Hv = case["Hk"], case["Hv"]
        unit = torch.nn.functional.normalize
        s["q"], s["k"] = (unit(randn(T, Hk, d), dim=-1).to(dt) for _ in range(2))
        s["v"] = randn(T, Hv, d).to(dt)
        # log decays between about -0.6 and -0.002, write strengths around one half
        s["g"] = (-torch.exp(1.5 * randn(T, Hv) - 3.5).clamp(0.002, 0.6)).to(dt)
        s["beta"] = torch.sigmoid(randn(T, Hv)).to(dt)
        s["S"] = 0.3 * randn(n, Hv, d, d)
        s["scale"] = 1.0 / math.sqrt(d)
        if case["op"] == "delta_train":
            s["dout"], s["dS"] = randn(T, Hv, d).to(dt), 0.1 * randn(n, Hv, d, d)
        return s
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "cache_step":
        cap = case["capacity"]
        s["q"] = randn(n, Hq, d).to(dt)
        s["k"], s["v"] = (randn(n * cap, Hkv, d).to(dt) for _ in range(2))
        s["q_off"] = torch.arange(n + 1, dtype=torch.int32, device=dev)
        s["k_off"] = s["q_off"] * cap
        s["q_len"], s["k_len"] = torch.ones(n, dtype=torch.int32, device=dev), s["lens"]
        s["max_q"], s["max_k"] = 1, s["longest"]
        return s
    if case["fused"]:
        qkv = randn(T, Hq + 2 * Hkv, d).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = randn(T, Hq, d).to(dt), randn(T, Hkv, d).to(dt), randn(T, Hkv, d).to(dt)
    s["q_off"] = s["k_off"] = s["off"]
    s["q_len"] = s["k_len"] = s["lens"]
    s["max_q"] = s["max_k"] = s["longest"]
    if case["op"] == "prompt_train":
        s["dout"] = randn(T, Hq, d).to(dt)
    return s


# ---------------------------------------------------------------- plain forms
def _rows(off, lens, longest):
    """Row numbers [n_seq, longest] of the padded sequences, and which are theirs."""
    t = torch.arange(longest, device=off.device)
    ok = t[None, :] < lens[:, None]
    return torch.where(ok, off[:-1, None] + t[None, :], 0).long(), ok


def _plain_attention(q, k, v, s):
    """Softmax attention in 32 bits on padded sequences; (out, lse) packed."""
    Tq, Hq, d = q.shape
    iq, okq = _rows(s["q_off"], s["q_len"], s["max_q"])
    ik, okk = _rows(s["k_off"], s["k_len"], s["max_k"])
    n, Hkv = iq.shape[0], k.shape[1]
    qp = q[iq].view(n, -1, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    kp, vp = (x[ik].permute(0, 2, 1, 3).unsqueeze(2) for x in (k, v))
    i = torch.arange(s["max_q"], device=q.device)[None, :, None] + (s["k_len"] - s["q_len"])[:, None, None]
    seen = (torch.arange(s["max_k"], device=q.device)[None, None, :] <= i) & okk[:, None, :]
    x = torch.matmul(qp, kp.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True).detach().clamp_min(-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vp) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(n, -1, Hq, d)[okq], lse.permute(0, 3, 1, 2).reshape(n, -1, Hq)[okq].t()


def _plain_delta(q, k, v, g, beta, S, s):
    """The gated delta rule in 32 bits over chunks of 64 tokens (log decays summed in 64); (out packed, S)."""
    C = 64
    m = -(-s["longest"] // C)
    idx, ok = _rows(s["off"], s["lens"], m * C)
    n, rep = idx.shape[0], v.shape[1] // q.shape[1]

    def chunks(x):
        x = torch.where(ok.view(n, m * C, *[1] * (x.dim() - 1)), x[idx], 0)
        return x.view(n, m, C, *x.shape[2:]).transpose(2, 3)  # [n, chunk, head, token, ...]

    qc, kc = (chunks(x).repeat_interleave(rep, dim=2) for x in (q, k))
    vc, bc = chunks(v), chunks(beta).unsqueeze(-1)
    G = chunks(g).double().cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~low, float("-inf"))).float()
    into, rest, whole = torch.exp(G).float().unsqueeze(-1), torch.exp(G[..., -1:] - G).float().unsqueeze(-1), \
        torch.exp(G[..., -1]).float()[..., None, None]
    A = (bc * torch.matmul(kc, kc.transpose(-1, -2)) * D).tril(-1) + torch.eye(C, device=q.device)
    both = torch.linalg.solve_triangular(A, torch.cat([bc * vc, bc * into * kc], -1), upper=False, unitriangular=True)
    u0, w = both.split([vc.shape[-1], kc.shape[-1]], -1)
    P = s["scale"] * torch.matmul(qc, kc.transpose(-1, -2)) * D
    qs, kr, outs = s["scale"] * into * qc, (rest * kc).transpose(-1, -2), []
    for c in range(m):
        u = u0[:, c] - torch.matmul(w[:, c], S)
        outs.append(torch.matmul(qs[:, c], S) + torch.matmul(P[:, c], u))
        S = whole[:, c] * S + torch.matmul(kr[:, c], u)
    o = torch.stack(outs, 1).transpose(2, 3).reshape(n, m * C, v.shape[1], -1)
    return o[ok], S


def _plain(s):
    f = {x: s[x].float() for x in ("q", "k", "v", "g", "beta", "dout") if x in s}
    dt = s["q"].dtype
    if s["op"] in ("prompt", "cache_step"):
        out, lse = _plain_attention(f["q"], f["k"], f["v"], s)
        return {"out": out.to(dt), "lse": lse}
    if s["op"] == "prompt_train":
        x = [f[a].detach().requires_grad_() for a in ("q", "k", "v")]
        out, lse = _plain_attention(*x, s)
        grads = torch.autograd.grad(out, x, f["dout"])
        return {"out": out.detach().to(dt), "lse": lse.detach(),
                **{"d" + a: y.to(dt) for a, y in zip(("q", "k", "v"), grads)}}
    if s["op"] == "delta":
        out, S = _plain_delta(f["q"], f["k"], f["v"], f["g"], f["beta"], s["S"], s)
        return {"out": out.to(dt), "S": S}
    if s["op"] == "delta_train":
        x = [f[a].detach().requires_grad_() for a in ("q", "k", "v", "g", "beta")] + [s["S"].clone().requires_grad_()]
        out, S = _plain_delta(*x, s)
        grads = torch.autograd.grad([out, S], x, [f["dout"], s["dS"]])
        return {"out": out.detach().to(dt), "S": S.detach(), "dS": grads[5],
                **{"d" + a: y.to(dt) for a, y in zip(("q", "k", "v", "g", "beta"), grads)}}
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (f[a].repeat_interleave(rep, dim=1).unsqueeze(-2) for a in ("q", "k"))
    S = s["S"].mul_(torch.exp(f["g"])[..., None, None])
    u = f["beta"][..., None] * (f["v"] - torch.matmul(k, S).squeeze(-2))
    S.add_(k.transpose(-1, -2) * u.unsqueeze(-2))
    return {"out": (s["scale"] * torch.matmul(q, S).squeeze(-2)).to(dt), "S": S}


# ------------------------------------------------------------- the operators
def _own(s):
    from compressive_memory_segment_b200 import binding as bd

    if s["op"] == "cache_step":
        out, lse = bd.packed_forward(s["q"], s["k"], s["v"], s["q_off"], s["k_off"], k_len=s["k_len"], max_q=1,
                                     max_k=s["max_k"])
        return {"out": out, "lse": lse}
    if s["op"] in ("prompt", "prompt_train"):
        out, lse = bd.packed_forward(s["q"], s["k"], s["v"], s["q_off"], max_q=s["max_q"], max_k=s["max_k"])
        r = {"out": out, "lse": lse}
        if s["op"] == "prompt_train":
            r["dq"], r["dk"], r["dv"] = bd.packed_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["q_off"],
                                                           max_q=s["max_q"], max_k=s["max_k"])
        return r
    x = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if s["op"] == "delta_step":
        return {"out": bd.delta_step(*x, s["S"], scale=s["scale"]), "S": s["S"]}
    out, S = bd.delta_forward(*x, s["off"], S_in=s["S"], scale=s["scale"], max_len=s["longest"])
    r = {"out": out, "S": S}
    if s["op"] == "delta_train":
        g = bd.delta_backward(*x, s["off"], s["dout"], S_in=s["S"], dS_out=s["dS"], scale=s["scale"],
                              max_len=s["longest"])
        r.update(zip(("dq", "dk", "dv", "dg", "dbeta", "dS"), g))
    return r


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- exact
def _exact_attention(s):
    """Sequence by sequence and key head by key head, from the definition."""
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    train = "dout" in s
    do = s["dout"].double() if train else None
    Hkv, d = k.shape[1], q.shape[2]
    G = q.shape[1] // Hkv
    r = {"out": torch.zeros_like(q), "lse": torch.full((q.shape[1], q.shape[0]), -math.inf, device=q.device,
                                                       dtype=torch.float64)}
    if train:
        r.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    at = list(zip(*(s[x].tolist() for x in ("q_len", "k_len")), s["q_off"].tolist(), s["k_off"].tolist()))
    for nq, nk, a, b in at:
        hidden = torch.ones(nq, nk, dtype=torch.bool, device=q.device).triu(nk - nq + 1)
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            Q, K, V = q[a:a + nq, hs].transpose(0, 1), k[b:b + nk, h], v[b:b + nk, h]
            z = (Q @ K.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(z, -1)
            p = z.sub_(lse.unsqueeze(-1)).exp_()
            o = p @ V
            r["out"][a:a + nq, hs], r["lse"][hs, a:a + nq] = o.transpose(0, 1), lse
            if train:
                dO = do[a:a + nq, hs].transpose(0, 1)
                r["dv"][b:b + nk, h] = (p.transpose(1, 2) @ dO).sum(0)
                ds = p * (dO @ V.T - (dO * o).sum(-1, keepdim=True)) / math.sqrt(d)
                r["dq"][a:a + nq, hs] = (ds @ K).transpose(0, 1)
                r["dk"][b:b + nk, h] = (ds.transpose(1, 2) @ Q).sum(0)
    return r


def _exact_delta(s):
    """Token by token over all sequences and heads at once, in both directions."""
    lens = [1] * s["v"].shape[0] if s["op"] == "delta_step" else s["lens"].tolist()
    n, Hv, d = len(lens), s["v"].shape[1], s["v"].shape[2]
    rep, T = Hv // s["q"].shape[1], s["v"].shape[0]
    first = [0]
    for x in lens:
        first.append(first[-1] + x)
    first = torch.tensor(first[:-1], device=s["v"].device)
    left = torch.tensor(lens, device=first.device)
    q, k = (s[x].double().repeat_interleave(rep, dim=1) for x in ("q", "k"))
    v, b, a = s["v"].double(), s["beta"].double(), s["g"].double().exp()
    S, out, kept = s["S"].double(), torch.zeros_like(v), []
    train = s["op"] == "delta_train"
    for t in range(max(lens)):
        live = (t < left).nonzero().squeeze(1)
        at = first[live] + t
        Sd = S[live] * a[at][..., None, None]
        u = b[at][..., None] * (v[at] - torch.einsum("nhkv,nhk->nhv", Sd, k[at]))
        Sn = Sd + k[at].unsqueeze(-1) * u.unsqueeze(-2)
        out[at] = s["scale"] * torch.einsum("nhkv,nhk->nhv", Sn, q[at])
        if train:
            kept.append((live, at, Sd))
        S = S.index_copy(0, live, Sn)
    r = {"out": out, "S": S}
    if not train:
        return r
    do, dS = s["dout"].double(), s["dS"].double().clone()
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(b)
    while kept:
        live, at, Sd = kept.pop()
        kt, bt = k[at], b[at][..., None]
        err = v[at] - torch.einsum("nhkv,nhk->nhv", Sd, kt)
        Sn = Sd + kt.unsqueeze(-1) * (bt * err).unsqueeze(-2)
        dq[at] = s["scale"] * torch.einsum("nhkv,nhv->nhk", Sn, do[at])
        X = dS[live] + s["scale"] * q[at].unsqueeze(-1) * do[at].unsqueeze(-2)
        du = torch.einsum("nhkv,nhk->nhv", X, kt)
        db[at] = (du * err).sum(-1)
        dv[at] = bt * du
        dk[at] = torch.einsum("nhkv,nhv->nhk", X, bt * err) - torch.einsum("nhkv,nhv->nhk", Sd, bt * du)
        X = X - kt.unsqueeze(-1) * (bt * du).unsqueeze(-2)
        dg[at] = (X * Sd).sum((-1, -2))
        dS[live] = X * a[at][..., None, None]
    heads = lambda x: x.view(T, -1, rep, d).sum(2)  # noqa: E731
    r.update(dq=heads(dq), dk=heads(dk), dv=dv, dg=dg, dbeta=db, dS=dS)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("delta"):
        return _exact_attention(s)
    # The reverse recurrence keeps one state for each token.
    if case["op"] == "delta_train" and case["n_seq"] * case["hi"] * case["Hv"] * case["d"] ** 2 * 8 > 80e9:
        return None
    return _exact_delta(s)
