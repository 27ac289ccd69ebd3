"""Cases of the operators beside the quantized linear: low-rank adapters of
many requests (forward and backward), layer norm (forward and backward) and
layer norm fused with the row-wise activation quantizer.

`own = False` computes an operator in its plain form (elementary torch
operations in f32, rounded once at the end); `own = True` calls the package.

Operators (bf16 tensors unless stated; m: token, k: in-feature, n: out-feature,
j: rank index, l = l(m): the adapter of the request that token m belongs to,
-1 for none; rank_l <= R entries of an adapter's rank axis are in use):
  adapters          u[m, j]   = scale_l sum_k x[m, k] a[l, j, k]          (f32)
                    out[m, n] = base[m, n] + sum_j u[m, j] b[l, n, j]
  adapters_backward g[m, j]   = scale_l sum_n dy[m, n] b[l, n, j]
                    dx[m, k]  = base[m, k] + sum_j g[m, j] a[l, j, k]
                    da[l, j, k] = sum_{m of l} g[m, j] x[m, k]            (f32)
                    db[l, n, j] = sum_{m of l} dy[m, n] u[m, j]           (f32)
  norm              y = (x - mean) rstd weight + bias, mean and rstd f32
  norm_backward     dx, dweight (f32), dbias (f32)
  norm_quant        e4m3 codes and row scales of the normalised rows
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one request generating one token beside a small projection: latency
        dict(name="adapters, one token", op="adapters", M=1, K=1024, N=1024, R=16, L=4, S=1, cut=0),
        # a decode step of 48 requests, each with an adapter of its own choice
        dict(name="adapters, decode 48", op="adapters", M=48, K=4096, N=4096, R=16, L=32, S=48, cut=1),
        # prompts of nine requests of uneven lengths, one empty and one without an adapter, ranks differ
        dict(name="adapters, prompts", op="adapters", M=1531, K=2048, N=5120, R=32, L=6, S=9, cut=2),
        # a training step's forward beside the widest projection of this repository's workloads
        dict(name="adapters, training", op="adapters", M=8192, K=4096, N=12288, R=64, L=1, S=1, cut=3),
        # the backward pass of seven uneven sequences that train four adapters
        dict(name="adapters backward, four", op="adapters_backward", M=2039, K=4096, N=1024, R=16, L=4, S=7, cut=4),
        # the backward pass of one adapter over a training batch
        dict(name="adapters backward, training", op="adapters_backward", M=8192, K=4096, N=4096, R=32, L=1, S=1, cut=5),
        # the norm in front of a decode step's projections
        dict(name="norm, decode 16", op="norm", M=16, K=4096, dtype="bf16", affine=True),
        # a diffusion transformer's norm: its scale and shift come later, so no weights
        dict(name="norm, training", op="norm", M=4608, K=5120, dtype="bf16", affine=False),
        # an odd width, in f32
        dict(name="norm backward, odd", op="norm_backward", M=333, K=1001, dtype="f32", affine=True),
        # a training step's backward
        dict(name="norm backward, training", op="norm_backward", M=8192, K=4096, dtype="bf16", affine=True),
        # the norm and quantizer in front of a decode step's 8-bit projections
        dict(name="norm to codes, decode 7", op="norm_quant", M=7, K=1280, dtype="bf16", affine=True),
        # the same over a prompt or a training batch
        dict(name="norm to codes, training", op="norm_quant", M=8192, K=4096, dtype="bf16", affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_backward", "norm", "norm_backward", "norm_quant"])
    if op.startswith("adapters"):
        K, N = 8 * _log_int(rng, 32, 768), 8 * _log_int(rng, 32, 768)
        R, L = rng.choice([8, 16, 24, 32, 64, 128]), rng.randint(1, 16)
        # no more than the largest listed case, whose plain form multiplies by every adapter there is
        most = 2 * 8192 * (4096 + 12288) * 64 // ((2 if op == "adapters" else 4) * (K + N) * R * L)
        M = _log_int(rng, 1, min(8192, most))
        return dict(op=op, M=M, K=K, N=N, R=R, L=L, S=min(_log_int(rng, 1, 64), M), cut=rng.randrange(1 << 20))
    dtype, affine = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7
    M = _log_int(rng, 1, 8192 if dtype == "bf16" else 4096)
    if op == "norm_quant":
        K = 16 * _log_int(rng, 16, 384)
    else:
        K = _log_int(rng, 64, 6144)
        K = K if rng.random() < 0.3 else 8 * ((K + 7) // 8)
    return dict(op=op, M=M, K=K, dtype=dtype, affine=affine)


def _requests(case):
    """(lengths, adapters, ranks) of a case: S requests of M tokens in all.
    One token each where M == S; else cut at random, the third (of more than
    four) empty; of more than seven requests every eighth has no adapter."""
    rng = random.Random(case["cut"])
    M, S, L, R = case["M"], case["S"], case["L"], case["R"]
    if S == M or S == 1:
        lengths = [M // S] * S
    else:
        at = sorted(rng.randint(0, M) for _ in range(S - 1))
        if S > 4:
            at[2] = at[1]
        lengths = [b - a for a, b in zip([0] + at, at + [M])]
    adapters = [i % L if S <= L else rng.randrange(L) for i in range(S)]
    if S > 7:
        adapters[7::8] = [-1] * len(adapters[7::8])
    ranks = [R] * L
    if L > 4:
        ranks = [max(1, R >> rng.randint(0, 2)) for _ in range(L)]
    return lengths, adapters, ranks


# ------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, M, K, dtype=torch.bfloat16):
    """Normal activations with 8 outlier channels and an offset."""
    x = torch.randn((M, K), generator=g, device="cuda") + 0.1
    x[:, torch.randperm(K, generator=g, device="cuda")[:8]] *= 6.0
    return x.to(dtype)


def prepare(case, seed):
    g = _rng(seed)
    M, K = case["M"], case["K"]
    if not case["op"].startswith("adapters"):
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s = dict(op=case["op"], x=_activations(g, M, K, dt), w=None, b=None)
        if case["affine"]:
            s["w"] = (torch.randn(K, generator=g, device="cuda") * 0.2 + 1.0).to(dt)
            s["b"] = _normal(g, (K,), 0.1, dt)
        if case["op"] == "norm_backward":
            s["dy"] = _normal(g, (M, K), 1e-3, dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        return s

    N, R, L = case["N"], case["R"], case["L"]
    lengths, adapters, ranks = _requests(case)
    token = torch.repeat_interleave(torch.tensor(adapters), torch.tensor(lengths)).cuda()
    s = dict(op=case["op"], token=token, ranks=torch.tensor(ranks, dtype=torch.int32).cuda(),
             x=_activations(g, M, K),
             a=_normal(g, (L, R, K), K ** -0.5), b=_normal(g, (L, N, R), 0.05),
             scale=torch.rand(L, generator=g, device="cuda") + 0.5)
    if case["op"] == "adapters":
        s["base"] = _normal(g, (M, N), 1.0)
    else:
        s["dy"] = _normal(g, (M, N), 1e-3)
        s["base"] = _normal(g, (M, K), 1e-3)
        s["u"] = _down(s["x"].float(), s["a"].float(), s)[0]
    if own:
        import w8a8_quantized_linear_quant_amd as w8
        s["plan"] = w8.lora_plan(lengths, adapters, L)
    return s


# -------------------------------------------------------------- plain forms
def _in_use(s):
    """[M, L, R]: whether token m uses rank entry j of adapter l."""
    L, R = s["a"].shape[:2]
    l = torch.arange(L, device="cuda")
    j = torch.arange(R, device="cuda")
    return (s["token"][:, None] == l)[:, :, None] & (j < s["ranks"][:, None])[None]


def _down(x, w, s):
    """(u [M, R], its spread over the adapters [M, L * R]): scale x w^T, w [L, R, K]."""
    L, R, K = w.shape
    full = (x @ w.reshape(L * R, K).T).reshape(-1, L, R) * s["scale"][:, None]
    full = torch.where(_in_use(s), full, 0.0)
    return full.sum(1), full.reshape(-1, L * R)


def _spread(u, s):
    """u [M, R] -> [M, L * R]: zero but at the token's own adapter."""
    return torch.where(_in_use(s), u[:, None, :], 0.0).reshape(u.shape[0], -1)


def _plain_adapters(s):
    a, b = s["a"].float(), s["b"].float()
    u, full = _down(s["x"].float(), a, s)
    out = s["base"].float() + full @ b.transpose(1, 2).reshape(full.shape[1], -1)
    return out.to(torch.bfloat16), u


def _plain_adapters_backward(s):
    x, dy, a, b = s["x"].float(), s["dy"].float(), s["a"].float(), s["b"].float()
    L, R, K = a.shape
    _, full = _down(dy, b.transpose(1, 2).contiguous(), s)
    dx = (s["base"].float() + full @ a.reshape(L * R, K)).to(torch.bfloat16)
    da = (full.T @ x).reshape(L, R, K)
    db = (_spread(s["u"], s).T @ dy).reshape(L, R, -1).transpose(1, 2).contiguous()
    return dx, da, db


def _normalised(s):
    x = s["x"].float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
    y = d * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"].float() + s["b"].float()
    return y, mean, rstd


def _plain_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    K = x.shape[1]
    h = (x - s["mean"][:, None]) * s["rstd"][:, None]
    wdy = dy * s["w"].float() if s["w"] is not None else dy
    c1 = wdy.sum(1, keepdim=True) / K
    c2 = (wdy * h).sum(1, keepdim=True) / K
    dx = ((wdy - c1 - h * c2) * s["rstd"][:, None]).to(s["x"].dtype)
    if s["w"] is None:
        return dx, None, None
    return dx, (dy * h).sum(0), dy.sum(0)


def _plain(s):
    op = s["op"]
    if op == "adapters":
        return _plain_adapters(s)
    if op == "adapters_backward":
        return _plain_adapters_backward(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    y, mean, rstd = _normalised(s)
    if op == "norm":
        return y.to(s["x"].dtype), mean, rstd
    top = y.abs().amax(1)
    scale = torch.where(top < 1e-10, 1e-10, top / E4M3_MAX)
    return (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def run(s):
    if not own:
        return _plain(s)
    import w8a8_quantized_linear_quant_amd as w8

    op = s["op"]
    if op == "adapters":
        return w8.lora_forward(s["x"], s["a"], s["b"], s["plan"], scale=s["scale"], ranks=s["ranks"], base=s["base"])
    if op == "adapters_backward":
        return w8.lora_backward(s["dy"], s["x"], s["u"], s["a"], s["b"], s["plan"], scale=s["scale"],
                                ranks=s["ranks"], base=s["base"])
    if op == "norm":
        return w8.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_backward":
        return w8.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    return w8.w8a8_quant_act_rowwise_layer_norm(s["x"], s["w"], s["b"], eps=EPS, qtype=w8.FP8_E4M3)


# -------------------------------------------------------------------- work
def work(case):
    M, K = case["M"], case["K"]
    if case["op"].startswith("adapters"):
        N, R, L = case["N"], case["R"], case["L"]
        lengths, adapters, ranks = _requests(case)
        used = sorted({l for n, l in zip(lengths, adapters) if n and l >= 0})
        rows = sum(n for n, l in zip(lengths, adapters) if l >= 0)
        rank_rows = sum(n * ranks[l] for n, l in zip(lengths, adapters) if l >= 0)
        weights = 2 * (K + N) * sum(ranks[l] for l in used)
        if case["op"] == "adapters":
            return {"bytes": 2 * rows * K + 4 * M * N + 4 * M * R + weights, "flops": 2 * rank_rows * (K + N)}
        return {"bytes": 2 * rows * (K + N) + 4 * M * K + 4 * M * R + weights + 4 * L * R * (K + N),
                "flops": 4 * rank_rows * (K + N)}
    e = 4 if case["dtype"] == "f32" else 2
    w = 2 * e * K if case["affine"] else 0
    if case["op"] == "norm":
        return {"bytes": 2 * e * M * K + 8 * M + w, "flops": 8 * M * K}
    if case["op"] == "norm_backward":
        return {"bytes": 3 * e * M * K + 8 * M + (w // 2 + 8 * K if w else 0), "flops": 14 * M * K}
    return {"bytes": (e + 1) * M * K + 4 * M + w, "flops": 11 * M * K}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The definition, request by request and in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"].startswith("adapters"):
        lengths, adapters, ranks = _requests(case)
        x, a, b, base = (s[k].to(f64) for k in ("x", "a", "b", "base"))
        ends = np.cumsum(lengths)
        spans = [(slice(int(e) - n, int(e)), l) for e, n, l in zip(ends, lengths, adapters) if n and l >= 0]
        if case["op"] == "adapters":
            u = torch.zeros(case["M"], case["R"], dtype=f64, device="cuda")
            out = base.clone()
            for rows, l in spans:
                r = ranks[l]
                u[rows, :r] = float(s["scale"][l]) * torch.mm(x[rows], a[l, :r].t())
                out[rows] += torch.mm(u[rows, :r], b[l, :, :r].t())
            return out, u
        dy, u = s["dy"].to(f64), s["u"].to(f64)
        dx, da, db = base.clone(), torch.zeros_like(a), torch.zeros_like(b)
        for rows, l in spans:
            r = ranks[l]
            g = float(s["scale"][l]) * torch.mm(dy[rows], b[l, :, :r])
            dx[rows] += torch.mm(g, a[l, :r])
            da[l, :r] += torch.mm(g.t(), x[rows])
            db[l, :, :r] += torch.mm(dy[rows].t(), u[rows, :r])
        return dx, da, db
    x = s["x"].to(f64)
    weight = s["w"].to(f64) if s["w"] is not None else torch.ones(case["K"], dtype=f64, device="cuda")
    shift = s["b"].to(f64) if s["b"] is not None else torch.zeros(case["K"], dtype=f64, device="cuda")
    if case["op"] == "norm_backward":
        # with t = dy weight and h the normalised row: dx = (t - <t> - h <t h>) / sigma
        dy, mu, inv = s["dy"].to(f64), s["mean"].to(f64).unsqueeze(1), s["rstd"].to(f64).unsqueeze(1)
        h = torch.mul(torch.sub(x, mu), inv)
        t = torch.mul(dy, weight)
        dx = inv * (t - t.mean(1, keepdim=True) - h * torch.mul(t, h).mean(1, keepdim=True))
        if s["w"] is None:
            return dx, None, None
        return dx, torch.mul(dy, h).sum(0), dy.sum(0)
    var, mu = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    inv = torch.rsqrt(var + EPS)
    y = torch.addcmul(shift, (x - mu) * inv, weight)
    if case["op"] == "norm":
        return y, mu.squeeze(1), inv.squeeze(1)
    step = y.abs().amax(1).clamp(min=1e-10 * E4M3_MAX) / E4M3_MAX
    return torch.div(y, step.unsqueeze(1)).clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn).to(f64), step
