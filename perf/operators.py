"""Cases of the router's balance loss and of the microscaled 4-bit (MXFP4) quantisation and products.

A case is a dict of plain values.  `prepare` makes its inputs on the GPU from a seed, `run` makes one
pass: in elementary torch operations where `own` is false, through the package's entry points where
it is true.  `exact` gives the same outputs from the definitions in 64 bits.

Definitions
  balance   per sequence q of n_q tokens, counts_qe = (token, slot) pairs of q that chose expert e,
            f_qe = counts_qe E / (k n_q), p_te = s_te / sum_j s_tj;
            loss = coef / S' sum_q sum_e f_qe mean_{t in q} p_te over the S' sequences with tokens,
            and its gradient in s (the choice, and with it f, is constant).  Tokens outside every
            sequence take no part (gradient 0).
  MXFP4     32 values along K share a scale 2^X, X = floor(log2 max|v|) - 2 clamped to [-127, 127];
            each value is held as v 2^-X rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to
            the even code), saturating at 6.
  product   C = A B^T of MXFP4 operands, sums in fp32; grouped: the rows of expert e times expert e's
            matrix; swiglu: columns in groups of 64 gate and 64 linear values, C = silu(gate) linear.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_MAX_GROUPED = 262144 * 1024 * 2048   # rows x N x K of the largest grouped case
_MAX_WEIGHTS = 896 * 1024 * 2048      # E x N x K of its weights
_MAX_DENSE = 16384 * 8192 * 7168


def listed():
    return [
        # a short last micro-batch of one sequence at a small expert count: launch latency
        dict(name="balance_short", op="balance", T=37, E=64, k=4, seqs=1, ragged=False),
        # the replica's batch, four sequences of 2048 tokens, 256 experts choose 6
        dict(name="balance_replica", op="balance", T=8192, E=256, k=6, seqs=4, ragged=False),
        # the wide layer's batch packed from seven documents of uneven lengths, padding behind the last
        dict(name="balance_wide", op="balance", T=16384, E=896, k=16, seqs=7, ragged=True),
        # one token's backbone row, as a serving step quantises it
        dict(name="quant_token", op="quant", rows=1, K=7168, dtype="bf16"),
        # fp32 rows whose length is not a multiple of 128
        dict(name="quant_odd", op="quant", rows=2047, K=1056, dtype="f32"),
        # the wide layer's batch of backbone rows
        dict(name="quant_wide", op="quant", rows=16384, K=7168, dtype="bf16"),
        # the up-projection of a single token: the weights' stream
        dict(name="gemm_token", op="gemm", M=1, N=7168, K=2048, swiglu=False, out="bf16"),
        # sizes that fill no tile, fp32 results
        dict(name="gemm_odd", op="gemm", M=333, N=1000, K=992, swiglu=False, out="f32"),
        # the shared expert's gate and linear projections at the wide layer
        dict(name="gemm_wide", op="gemm", M=16384, N=8192, K=7168, swiglu=True, out="bf16"),
        # one token's 16 experts of 896: gate and linear projections of a decoding step
        dict(name="experts_token", op="grouped", T=1, E=896, k=16, N=1024, K=2048, swiglu=True, out="bf16"),
        # the replica's down-projections, 256 experts choose 6
        dict(name="experts_replica", op="grouped", T=8192, E=256, k=6, N=256, K=256, swiglu=False, out="bf16"),
        # the wide layer's gate and linear projections, 896 experts choose 16
        dict(name="experts_wide", op="grouped", T=16384, E=896, k=16, N=1024, K=2048, swiglu=True, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "quant", "gemm", "grouped"])
    if op == "balance":
        E = rng.choice([8, 33, 64, 100, 128, 160, 256, 384, 512, 896, 1024])
        T = _log_int(rng, 1, min(65536, 16384 * 896 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), seqs=rng.randint(1, min(T, 24)),
                    ragged=rng.random() < 0.5)
    if op == "quant":
        rows, K = _log_int(rng, 1, 16384), 32 * _log_int(rng, 1, 224)
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "f32"]) if rows * K <= 8192 * 7168 else "bf16")
    swiglu = rng.random() < 0.4
    out = "bf16" if swiglu or rng.random() < 0.6 else "f32"
    if op == "gemm":
        while True:
            M, K = _log_int(rng, 1, 16384), 32 * _log_int(rng, 1, 224)
            N = 128 * _log_int(rng, 1, 64) if swiglu else _log_int(rng, 8, 8192)
            if M * N * K <= _MAX_DENSE // 2:
                return dict(op=op, M=M, N=N, K=K, swiglu=swiglu, out=out)
    while True:
        T, E = _log_int(rng, 1, 16384), rng.choice([8, 17, 32, 64, 96, 128, 256, 512, 896])
        k, K = rng.randint(1, min(E, 16)), 32 * _log_int(rng, 2, 64)
        N = 128 * _log_int(rng, 1, 16) if swiglu else _log_int(rng, 32, 2048)
        if T * k * N * K <= _MAX_GROUPED // 2 and E * N * K <= _MAX_WEIGHTS // 2:
            return dict(op=op, T=T, E=E, k=k, N=N, K=K, swiglu=swiglu, out=out)


# --------------------------------------------------------------------------- inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(shape, g, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else
                        torch.bfloat16) * scale).to(dtype)


def _rows(shape, g, dtype):
    """Activations: normal, with a size of its own for each row and a few columns ten times larger."""
    v = _randn(shape, g, dtype=dtype)
    v *= torch.exp2(torch.randint(-3, 4, (shape[0], 1), generator=g, device="cuda").float()).to(dtype)
    v[:, torch.randint(0, shape[1], (max(1, shape[1] // 128),), generator=g, device="cuda")] *= 10
    return v


def _cuts(T, seqs, ragged, seed):
    """Sequence bounds: equal lengths, or uneven ones with padding tokens behind the last."""
    if not ragged:
        return [q * T // seqs for q in range(seqs + 1)]
    r = np.random.default_rng([seed, T, seqs])
    last = T - T // 50
    return [0] + sorted(int(v) for v in r.integers(0, last + 1, seqs - 1)) + [last]


def _offsets(T, E, k, g):
    """First row of each expert and the end, for T tokens that choose k of E experts, some liked more."""
    liking = torch.randn(E, generator=g, device="cuda") * 0.5
    idx = (torch.randn((T, E), generator=g, device="cuda") + liking).topk(k, dim=1).indices
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(idx.flatten(), minlength=E).cumsum(0).int()
    return off


def _operands(case, g):
    """Offsets (grouped), rows and weights of a product, bf16."""
    N, K = case["N"], case["K"]
    off, rows, E = None, case.get("M"), 1
    if case["op"] == "grouped":
        rows, E = case["T"] * case["k"], case["E"]
        off = _offsets(case["T"], E, case["k"], g)
    x = _rows((rows, K), g, torch.bfloat16)
    return off, x, _randn((E, N, K), g, 1 / math.sqrt(K))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn((T, E), generator=g, device="cuda")
        logits += 0.7 * torch.randn(E, generator=g, device="cuda")
        scores = torch.sigmoid(logits)
        idx = scores.topk(k, dim=1).indices.int()
        cu = torch.tensor(_cuts(T, case["seqs"], case["ragged"], seed), dtype=torch.int32, device="cuda")
        return dict(op=op, scores=scores, idx=idx, cu=cu, coef=1e-2, k=k)
    if op == "quant":
        return dict(op=op, x=_rows((case["rows"], case["K"]), g, _type(case["dtype"])))
    off, x, w = _operands(case, g)
    N, K = case["N"], case["K"]
    s = dict(op=op, x=x, off=off, swiglu=case["swiglu"], out=_type(case["out"]))
    if off is not None:
        s["bounds"] = off.tolist()
    # weights are laid out once: 4-bit operands, or the values these stand for (bf16 holds them exactly)
    if own:
        import latent_routing_quantile_b200 as lq
        if case["swiglu"]:
            v = w.view(w.shape[0], N // 128, 2, 64, K)
            w1, w3 = (v[:, :, i].reshape(-1, N // 2, K).contiguous() for i in range(2))
            s["w"] = lq.mx4_quant_w13(w1, w3) if op == "grouped" else lq.mx4_quant_w13(w1[0], w3[0])
        else:
            s["w"] = lq.mx4_quant(w if op == "grouped" else w[0])
    else:
        s["w"] = torch.empty_like(w)
        for e in range(w.shape[0]):
            s["w"][e] = _mx4_values(w[e])
    return s


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# --------------------------------------------------------------------------- plain forms
def _mx4_values(x):
    """The values that x [rows, K] stands for in MXFP4, in fp32."""
    v = x.float().view(x.shape[0], -1, 32)
    amax = v.abs().amax(dim=2, keepdim=True)
    # the exponent field of an fp32 number is floor(log2) + 127
    X = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp(-127, 127)
    u = torch.ldexp(v, -X)
    a = u.abs()
    # halfway points between neighbouring codes; a tie goes to the even one
    q = 0.5 * (a > 0.25).float()
    q += 0.5 * (a >= 0.75).float()
    q += 0.5 * (a > 1.25).float()
    q += 0.5 * (a >= 1.75).float()
    q += (a > 2.5).float()
    q += (a >= 3.5).float()
    q += 2.0 * (a > 5.0).float()
    return torch.ldexp(torch.copysign(q, u), X).view(x.shape)


def _swiglu(c):
    v = c.view(c.shape[0], -1, 2, 64)
    gate, lin = v[:, :, 0], v[:, :, 1]
    return (gate / (1 + torch.exp(-gate)) * lin).reshape(c.shape[0], -1)


def _plain_balance(s):
    scores, cu, k = s["scores"], s["cu"].long(), s["k"]
    T, E = scores.shape
    S = cu.numel() - 1
    t = torch.arange(T, device=scores.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    inside = (seq >= 0) & (seq < S)
    seq = torch.where(inside, seq, S)
    n = torch.zeros(S + 1, device=scores.device).index_add(0, seq, torch.ones(T, device=scores.device))
    pair = (seq[:, None] * E + s["idx"].long()).flatten()
    counts = torch.bincount(pair, minlength=(S + 1) * E).view(S + 1, E)
    f = counts.float() * (E / k) / n.clamp(min=1)[:, None]
    weight = inside.float() * s["coef"] / ((n[:S] > 0).sum() * n[seq].clamp(min=1))
    total = scores.sum(dim=1, keepdim=True)
    p = scores / total
    ft = f[seq]
    dot = (p * ft).sum(dim=1)
    loss = (weight.double() * dot.double()).sum().float()
    dscores = weight[:, None] * (ft - dot[:, None]) / total
    return dict(loss=loss.view(1), counts=counts[:S].int(), dscores=dscores)


def _plain_product(s):
    a = _mx4_values(s["x"])
    if s["off"] is None:
        c = a @ s["w"][0].float().t()
    else:
        c = torch.empty((a.shape[0], s["w"].shape[1]), device=a.device)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                c[lo:hi] = a[lo:hi] @ s["w"][e].float().t()
    return (_swiglu(c) if s["swiglu"] else c).to(s["out"])


def run(state):
    s = state
    if own:
        import latent_routing_quantile_b200 as lq
        if s["op"] == "balance":
            return lq.balance_loss(s["scores"], s["idx"], s["coef"], cu_seqlens=s["cu"])
        if s["op"] == "quant":
            return lq.mx4_dequant(lq.mx4_quant(s["x"]), dtype=s["x"].dtype)
        return lq.mx4_gemm(lq.mx4_quant(s["x"], offsets=s["off"]), s["w"], swiglu=s["swiglu"], dtype=s["out"])
    if s["op"] == "balance":
        return _plain_balance(s)
    if s["op"] == "quant":
        return _mx4_values(s["x"]).to(s["x"].dtype)
    return _plain_product(s)


def work(case):
    """Inputs read once and outputs written once; 4-bit weights take 17/32 byte an element."""
    op = case["op"]
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        return {"bytes": 8 * T * E + 4 * T * k + 4 * S * E, "flops": 6 * T * E}
    if op == "quant":
        n, es = case["rows"] * case["K"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * es * n + n * 17 / 32, "flops": 4 * n}
    N, K = case["N"], case["K"]
    es = 4 if case["out"] == "f32" else 2
    if op == "gemm":
        M, mats = case["M"], 1
    else:
        M, mats = case["T"] * case["k"], min(case["E"], case["T"] * case["k"])
    return {"bytes": 2 * M * K + mats * N * K * 17 / 32 + es * M * (N // 2 if case["swiglu"] else N),
            "flops": 2 * M * N * K}


# --------------------------------------------------------------------------- definitions in 64 bits
def _exact_mx4(x):
    v = x.double().reshape(-1, 32)
    amax = v.abs().amax(dim=1)
    _, e = torch.frexp(torch.where(amax > 0, amax, torch.ones_like(amax)))
    X = torch.where(amax > 0, e.double() - 1 - 2, torch.full_like(amax, -127)).clamp(-127, 127)[:, None]
    u = v / torch.exp2(X)
    # spacing of the grid at |u|: 1/2 below 2, then 1, then 2 (torch.round takes a tie to the even multiple)
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0))
    q = (torch.round(u / step) * step).clamp(-6, 6)
    return (q * torch.exp2(X)).reshape(x.shape)


def exact(case, seed):
    op = case["op"]
    if op in ("gemm", "grouped"):
        return _exact_product(case, seed)
    s = prepare(case, seed)
    if op == "quant":
        return _exact_mx4(s["x"])
    sc, idx, cu = s["scores"].double(), s["idx"].long(), s["cu"].tolist()
    T, E = sc.shape
    counts = torch.zeros((case["seqs"], E), dtype=torch.int32, device="cuda")
    grad = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    filled = sum(hi > lo for lo, hi in zip(cu, cu[1:]))
    for q, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi == lo:
            continue
        chosen = torch.zeros((hi - lo, E), dtype=torch.float64, device="cuda").scatter_(1, idx[lo:hi], 1.0)
        counts[q] = chosen.sum(0).int()
        f = chosen.mean(0) * E / case["k"]
        R = sc[lo:hi].sum(1, keepdim=True)
        loss += s["coef"] / filled * (f * (sc[lo:hi] / R).mean(0)).sum()
        # d(s_e / R) / ds_j = (delta_ej - s_e / R) / R
        grad[lo:hi] = s["coef"] / filled / (hi - lo) * (f / R - (sc[lo:hi] @ f)[:, None] / R ** 2)
    return dict(loss=loss, counts=counts, dscores=grad)


def _exact_product(case, seed):
    off, x, w = _operands(case, _gen(seed))
    N = case["N"]
    bounds = [0, case["M"]] if off is None else off.tolist()
    out = torch.empty((x.shape[0], N // 2 if case["swiglu"] else N), dtype=torch.float64, device="cuda")
    for e, (first, end) in enumerate(zip(bounds, bounds[1:])):
        if end == first:
            continue
        wt = _exact_mx4(w[e]).t()
        for lo in range(first, end, 4096):
            hi = min(lo + 4096, end)
            c = _exact_mx4(x[lo:hi]) @ wt
            if case["swiglu"]:
                c = c.view(hi - lo, N // 128, 128)
                c = (c[..., :64] * torch.sigmoid(c[..., :64]) * c[..., 64:]).reshape(hi - lo, -1)
            out[lo:hi] = c
    return out
