"""Cases of the microscaled 4-bit format (quantizer, dequantizer, product) and
of products whose rows fall into groups with a weight each (the experts of a
mixture), in 8 bits and in the 4-bit format, with their input gradients.

`own = False` computes an operator in its plain form (elementary torch
operations in f32, rounded once at the end); `own = True` calls the package.

The format: a block of 32 values along a row shares a scale 2^e, e held as one
byte e + 127; a value is one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it.
  quantize   e = max(floor(log2(absmax of the block)) - 2, -127); values
             x / 2^e rounded to the nearest (ties to the even code), at most 6.
  Codes lie two a byte, the first of a pair in the low half; a row's scales
  are padded to a multiple of 16 bytes with 127 (the scale 1).

Products (p: row of the output, k: in-feature, n: out-feature, t = rows[p] the
row of x that it takes, g = g(p) the group with offsets[g] <= p < offsets[g+1]):
  mx_linear   y[p, n] = sum_k x[p, k] w[n, k] + bias[n]                  (bf16)
  experts     y[p, n] = sx[t] sw[g] sum_k x[t, k] w[g, n, k] + bias[g, n]
  mx_experts  y[p, n] = sum_k x[t, k] w[g, n, k] + bias[g, n]
  The input gradient is the same product of the quantized dy with the weight's
  transpose: rows = 0 .. M - 1 and no bias.
"""
import math
import random

import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the activations of a decode step, quantized and expanded again: latency
        dict(name="mx round trip, decode 8", op="mx_round_trip", M=8, K=4096, dtype="bf16", transposed=False),
        # a projection's weight as the forward and the backward pass of a training run with 4-bit weights see it
        dict(name="mx round trip, weight and transpose", op="mx_round_trip", M=5120, K=4096, dtype="bf16",
             transposed=True),
        # one token through a small projection: latency
        dict(name="mx linear, one token", op="mx_linear", M=1, N=1024, K=1024, bias=True),
        # a decode step of 48 requests through a wide projection
        dict(name="mx linear, decode 48", op="mx_linear", M=48, N=12288, K=4096, bias=True),
        # a prompt of odd length, an odd width and a reduction that ends inside a tile
        dict(name="mx linear, odd prompt", op="mx_linear", M=1531, N=5121, K=2080, bias=False),
        # a training step's forward through the widest projection of this repository's workloads
        dict(name="mx linear, training", op="mx_linear", M=8192, N=12288, K=4096, bias=True),
        # a decode step of 16 tokens, two of 32 experts each
        dict(name="experts int8, decode 16", op="experts", qtype="int8", X=16, top=2, E=32, N=2048, K=4096,
             channels=False, bias=False, cut=0),
        # a prompt of odd length, four of 16 experts a token, a scale for each output channel
        dict(name="experts e4m3, odd prompt", op="experts", qtype="e4m3", X=1531, top=4, E=16, N=2048, K=4096,
             channels=True, bias=True, cut=1),
        # a training step's forward, two of eight experts a token
        dict(name="experts int8, training", op="experts", qtype="int8", X=8192, top=2, E=8, N=5120, K=4096,
             channels=False, bias=False, cut=2),
        # its backward: the gradient through the experts' second projection, from 4096 columns to 1280
        dict(name="experts e4m3, backward", op="experts", qtype="e4m3", X=16384, top=0, E=8, N=1280, K=4096,
             channels=False, bias=False, cut=3),
        # a decode step of 64 tokens, four of 64 experts each, 4-bit weights
        dict(name="mx experts, decode 64", op="mx_experts", X=64, top=4, E=64, N=2048, K=4096, bias=False, cut=4),
        # a training step's forward with 4-bit experts
        dict(name="mx experts, training", op="mx_experts", X=8192, top=2, E=8, N=5120, K=4096, bias=True, cut=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mx_round_trip", "mx_linear", "mx_linear", "experts", "experts", "experts", "mx_experts",
                     "mx_experts"])
    if op == "mx_round_trip":
        return dict(op=op, M=_log_int(rng, 1, 5120), K=_log_int(rng, 64, 4096), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    transposed=rng.random() < 0.3)
    K = 32 * _log_int(rng, 8, 160)
    N = _log_int(rng, 128, 6144)
    N = N if rng.random() < 0.2 else 16 * ((N + 15) // 16)
    if op == "mx_linear":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=N, K=K, bias=rng.random() < 0.5)
    E = _log_int(rng, 1, 64)
    E = max(1, min(E, 8 * 5120 * 4096 // (N * K)))        # no more weights than the largest listed case
    top = rng.choice([0, 1, 2, 4])
    most = 16384 // max(top, 1)
    case = dict(op=op, X=_log_int(rng, 1, most), top=top, E=E, N=N, K=K, bias=rng.random() < 0.5,
                cut=rng.randrange(1 << 20))
    if op == "experts":
        case.update(qtype=rng.choice(["int8", "e4m3"]), channels=rng.random() < 0.3)
    return case


def _lengths(case):
    """Rows of each group: M = X * top slots (X where top is 0: rows that lie
    in the groups' order already) fall to the groups with uneven chances; of
    more than four groups the third has none."""
    rng = random.Random(case["cut"])
    M, E = case["X"] * max(case["top"], 1), case["E"]
    chance = [rng.uniform(0.25, 1.0) for _ in range(E)]
    if E > 4:
        chance[2] = 0.0
    lengths = [0] * E
    for g in rng.choices(range(E), chance, k=M):
        lengths[g] += 1
    return lengths


# ------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, M, K):
    """Normal activations with 8 outlier channels."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[:8]] *= 6.0
    return x


def _codes8(x, qtype, dims):
    """(codes, scales over `dims`): absmax scaling to int8 or e4m3."""
    top = 127.0 if qtype == "int8" else 448.0
    scale = (x.abs().amax(dims, keepdim=True) / top).clamp(min=1e-10)
    q = (x / scale).clamp(-top, top)
    q = q.round().to(torch.int8) if qtype == "int8" else q.to(torch.float8_e4m3fn)
    return q, scale


def _codes4(x):
    """(packed codes [..., K / 2], padded scale bytes) of x [..., K]."""
    values, e = _to_mx(x)
    y = torch.ldexp(values, -e).reshape(x.shape)
    a = y.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)) + torch.where(y < 0, 8.0, 0.0)
    code = code.to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), _scale_bytes(e)


def prepare(case, seed):
    g = _rng(seed)
    op, K = case["op"], case["K"]
    if op == "mx_round_trip":
        x = _activations(g, case["M"], K)
        return dict(op=op, x=x if case["dtype"] == "f32" else x.to(torch.bfloat16), transposed=case["transposed"])
    N = case["N"]
    if op == "mx_linear":
        xq, xs = _codes4(_activations(g, case["M"], K))
        wq, ws = _codes4(torch.randn((N, K), generator=g, device="cuda") * 0.02)
        bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if case["bias"] else None
        return dict(op=op, xq=xq, xs=xs, wq=wq, ws=ws, bias=bias)

    X, E, lengths = case["X"], case["E"], _lengths(case)
    M = sum(lengths)
    ends = torch.tensor([0] + lengths).cumsum(0)
    s = dict(op=op, offsets=ends.to(torch.int32).cuda(), longest=max(lengths), rows=None, bias=None)
    if case["top"]:
        s["rows"] = (torch.randperm(M, generator=g, device="cuda") % X).to(torch.int32)
    if case["bias"]:
        s["bias"] = torch.randn((E, N), generator=g, device="cuda").to(torch.bfloat16)
    x = _activations(g, X, K)
    w = torch.randn((E, N, K), generator=g, device="cuda") * 0.02
    if op == "experts":
        s["xq"], sx = _codes8(x, case["qtype"], 1)
        s["wq"], sw = _codes8(w, case["qtype"], 2 if case["channels"] else (1, 2))
        s["xs"], s["ws"] = sx.flatten(), sw.reshape((E, N) if case["channels"] else (E,)).contiguous()
    else:
        s["xq"], s["xs"] = _codes4(x)
        s["wq"], s["ws"] = _codes4(w)
    return s


# -------------------------------------------------------------- plain forms
def _to_mx(x):
    """(the values that x [..., K] is rounded to, in blocks [..., K' / 32, 32],
    and e of each block [..., K' / 32, 1]), K' = K rounded up to whole blocks."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    y = torch.ldexp(x, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.ldexp((torch.round(y / step) * step).clamp(-6.0, 6.0), e), e


def _scale_bytes(e):
    """e [..., blocks, 1] as bytes, rows padded to a multiple of 16."""
    b = (e.squeeze(-1) + 127).to(torch.uint8)
    return torch.nn.functional.pad(b, (0, -b.shape[-1] % 16), value=127)


def _plain_round_trip(x):
    values, e = _to_mx(x)
    return values.flatten(-2)[..., :x.shape[-1]].to(x.dtype), _scale_bytes(e).view(torch.float8_e8m0fnu)


def _expand(codes, scales):
    """The f32 values [..., K] of packed codes [..., K / 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    half, mantissa = (c >> 1) & 3, 1.0 + 0.5 * (c & 1)
    a = torch.where(half > 0, torch.ldexp(mantissa, half.int() - 1), 0.5 * (c & 1))
    a = torch.where(c > 7, -a, a).unflatten(-1, (-1, BLOCK))
    e = scales[..., :a.shape[-2]].int() - 127
    return torch.ldexp(a, e[..., None]).flatten(-2)


def _plain_groups(s):
    """Every group's rows padded to the longest group, one batched product."""
    if s["op"] == "experts":
        x, w = s["xq"].float() * s["xs"][:, None], s["wq"].float()
        w = w * (s["ws"][:, None, None] if s["ws"].dim() == 1 else s["ws"][:, :, None])
    else:
        x, w = _expand(s["xq"], s["xs"]), _expand(s["wq"], s["ws"])
    first, M = s["offsets"].long(), (s["rows"] if s["rows"] is not None else x).shape[0]
    p = torch.arange(M, device="cuda")
    group = torch.searchsorted(first, p, right=True) - 1
    slot = group * s["longest"] + p - first[group]
    padded = torch.zeros((w.shape[0] * s["longest"], x.shape[1]), device="cuda")
    padded[slot] = x if s["rows"] is None else x[s["rows"].long()]
    y = torch.bmm(padded.view(w.shape[0], s["longest"], -1), w.transpose(1, 2).contiguous())
    y = y.view(-1, w.shape[1])[slot]
    if s["bias"] is not None:
        y = y + s["bias"].float()[group]
    return y.to(torch.bfloat16)


def _plain(s):
    if s["op"] == "mx_round_trip":
        there = _plain_round_trip(s["x"])
        return (*there, *_plain_round_trip(s["x"].T)) if s["transposed"] else there
    if s["op"] == "mx_linear":
        y = _expand(s["xq"], s["xs"]) @ _expand(s["wq"], s["ws"]).T
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    return _plain_groups(s)


def run(s):
    if not own:
        return _plain(s)
    import w8a8_quantized_linear_quant_amd as w8

    op = s["op"]
    if op == "mx_round_trip":
        x = s["x"]
        xq, xs = w8.mxfp4_quantize(x)
        there = w8.mxfp4_dequantize(xq, xs, x.shape[1], dtype=x.dtype), xs.view(torch.float8_e8m0fnu)
        if not s["transposed"]:
            return there
        tq, ts = w8.mxfp4_quantize_transposed(x)
        return (*there, w8.mxfp4_dequantize(tq, ts, x.shape[0], dtype=x.dtype), ts.view(torch.float8_e8m0fnu))
    if op == "mx_linear":
        return w8.mxfp4_linear(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"])
    if op == "experts":
        return w8.w8a8_linear_grouped(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], rows=s["rows"], bias=s["bias"])
    return w8.mxfp4_linear_grouped(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], rows=s["rows"], bias=s["bias"])


# -------------------------------------------------------------------- work
def _mx_bytes(rows, K):
    return rows * (-(-K // BLOCK) * BLOCK // 2 + -(-K // (16 * BLOCK)) * 16)


def work(case):
    op, K = case["op"], case["K"]
    if op == "mx_round_trip":
        M, e = case["M"], 4 if case["dtype"] == "f32" else 2
        # x read, codes and scales written and read again, values written
        there, back = 2 * e * M * K + 2 * _mx_bytes(M, K), e * M * K + 2 * _mx_bytes(K, M)
        return {"bytes": there + (back if case["transposed"] else 0), "flops": 8 * M * K * (2 if case["transposed"] else 1)}
    N = case["N"]
    if op == "mx_linear":
        M = case["M"]
        return {"bytes": _mx_bytes(M, K) + _mx_bytes(N, K) + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    lengths = _lengths(case)
    M, used = sum(lengths), sum(1 for n in lengths if n)
    if op == "experts":
        operands = case["X"] * (K + 4) + used * (N * K + (4 * N if case["channels"] else 4))
    else:
        operands = _mx_bytes(case["X"], K) + _mx_bytes(used * N, K)
    extra = (2 * used * N if case["bias"] else 0) + (4 * M if case["top"] else 0) + 4 * (case["E"] + 1)
    return {"bytes": operands + 2 * M * N + extra, "flops": 2 * M * N * K}


# ------------------------------------------------------------------- exact
_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _decoded(codes, scales):
    """Values in 64 bits by table, one code at a time of each pair."""
    table = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device="cuda")
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    out[..., 0::2], out[..., 1::2] = table[(codes & 15).long()], table[(codes // 16).long()]
    factor = torch.pow(2.0, scales.to(torch.float64) - 127.0)
    return out * factor.repeat_interleave(BLOCK, -1)[..., :out.shape[-1]]


def _nearest(x):
    """The round trip of rows x in 64 bits: the nearest table value by its
    borders, a border itself to the even code."""
    K = x.shape[1]
    blocks = -(-K // BLOCK)
    full = torch.zeros(x.shape[0], blocks * BLOCK, dtype=torch.float64, device="cuda")
    full[:, :K] = x.to(torch.float64)
    full = full.view(x.shape[0], blocks, BLOCK)
    e = torch.floor(torch.log2(full.abs().amax(2))) - 2
    scale = torch.pow(2.0, torch.clamp(e, min=-127.0))
    y = full / scale.unsqueeze(2)
    values = torch.tensor(_VALUES, dtype=torch.float64, device="cuda")
    borders = (values[1:] + values[:-1]) / 2
    low = torch.bucketize(y.abs(), borders, right=False)       # a border falls to the lower code
    at_border = (low < 7) & (y.abs() == borders[low.clamp(max=6)])
    code = torch.where(at_border & (low % 2 == 1), low + 1, low)
    out = (torch.sign(y) * values[code] * scale.unsqueeze(2)).view(x.shape[0], -1)[:, :K]
    padded = torch.ones(x.shape[0], -(-blocks // 16) * 16, dtype=torch.float64, device="cuda")
    padded[:, :blocks] = scale
    return out, padded


def exact(case, seed):
    """The definition, group by group and in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "mx_round_trip":
        there = _nearest(s["x"])
        return (*there, *_nearest(s["x"].t().contiguous())) if case["transposed"] else there
    f64 = torch.float64
    if case["op"] == "mx_linear":
        y = torch.mm(_decoded(s["xq"], s["xs"]), _decoded(s["wq"], s["ws"]).t())
        return y if s["bias"] is None else y.add_(s["bias"].to(f64))
    if case["op"] == "experts":
        x = torch.mul(s["xq"].to(f64), s["xs"].to(f64).unsqueeze(1))
    else:
        x = _decoded(s["xq"], s["xs"])
    if s["rows"] is not None:
        x = torch.index_select(x, 0, s["rows"].long())
    y = torch.empty(x.shape[0], case["N"], dtype=f64, device="cuda")
    at = 0
    for g, n in enumerate(_lengths(case)):
        if not n:
            continue
        if case["op"] == "experts":
            w = s["wq"][g].to(f64) * s["ws"][g].to(f64).reshape(-1, 1)
        else:
            w = _decoded(s["wq"][g], s["ws"][g])
        torch.mm(x[at:at + n], w.t(), out=y[at:at + n])
        if s["bias"] is not None:
            y[at:at + n] += s["bias"][g].to(f64)
        at += n
    return y
