"""Plain 64-bit definitions of the microscaled 4-bit format and of products of
groups of rows, for the tests of include/w8a8_experts.h."""
import torch

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2      # 2^-8, relative


def stride_of(K):
    return (K + 511) // 512 * 16


def quantize(x, ldq=None):
    """(codes 0..15 [M, ldq], scale bytes [M, stride]) of x [M, K], on the CPU."""
    x = x.detach().cpu().double()
    M, K = x.shape
    ldq = ldq or K + (-K) % 32
    full = torch.zeros(M, ldq, dtype=torch.float64)
    full[:, :K] = x
    blocks = full.view(M, ldq // 32, 32)
    top = blocks.abs().amax(2)
    bad = ~torch.isfinite(blocks).all(2)
    top = torch.where(bad, 1.0, top)
    e = torch.frexp(top).exponent - 1 - 2
    e = torch.where(top > 0, e, -127).clamp(min=-127)
    y = torch.where(bad[..., None], 0.0, blocks) * torch.pow(2.0, -e.double())[..., None]
    a = y.abs()
    dist = (a[..., None] - VALUES).abs()
    near = dist.argmin(-1)                                     # the first of two equal distances: the lower
    tie = (near < 7) & ((a - VALUES[near]) == (VALUES[(near + 1).clamp(max=7)] - a))
    near = torch.where(tie & (near % 2 == 1), near + 1, near)
    code = torch.where(torch.signbit(blocks) & ~bad[..., None], near + 8, near)
    scale = torch.full((M, stride_of(ldq)), 127, dtype=torch.uint8)
    scale[:, :ldq // 32] = torch.where(bad, 255, e + 127).to(torch.uint8)
    return code.view(M, ldq).to(torch.uint8), scale


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def values(packed, scale):
    """64-bit values of packed codes with their scales (any leading shape), on the codes' device."""
    code = unpack(packed).long()
    v = VALUES.to(packed.device)[code & 7] * torch.where(code > 7, -1.0, 1.0)
    s = scale[..., :code.shape[-1] // 32].double()
    f = torch.where(s == 255, float("nan"), torch.pow(2.0, s - 127))
    return v * f.repeat_interleave(32, -1)


def random_mx(g, shape, lo=120, hi=134):
    """Codes of every value and scale bytes in [lo, hi) (packed codes, scales), on the GPU."""
    K = shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, dtype=torch.uint8)
    scale = torch.randint(lo, hi, (*shape[:-1], stride_of(K)), generator=g, dtype=torch.uint8)
    return codes.cuda(), scale.cuda()


def groups_of(offsets, M):
    """[(group, first, end)] as the header defines them: offsets clamped to [0, M] and to the greatest before."""
    out, top = [], 0
    o = [int(v) for v in offsets]
    for g in range(len(o) - 1):
        first = max(top, min(max(o[g], 0), M))
        end = max(first, min(o[g + 1], M))
        top = end
        out.append((g, first, end))
    return out


def grouped(x, w, offsets, M, rows=None, bias=None):
    """(y, sum of |terms|, which rows are in a group) in 64 bits: x [X, K], w [E, N, K] dequantized."""
    y = torch.zeros(M, w.shape[1], dtype=torch.float64, device=x.device)
    mass = torch.zeros_like(y)
    inside = torch.zeros(M, dtype=torch.bool, device=x.device)
    if rows is None:
        src = x
    else:
        r = rows.long()
        ok = (r >= 0) & (r < x.shape[0])
        src = torch.where(ok[:, None], x[r.clamp(0, max(x.shape[0] - 1, 0))], 0.0)
    for g, a, b in groups_of(offsets, M):
        if b <= a:
            continue
        y[a:b] = src[a:b] @ w[g].T
        mass[a:b] = src[a:b].abs() @ w[g].abs().T
        if bias is not None:
            y[a:b] += bias[g].double()
            mass[a:b] += bias[g].double().abs()
        inside[a:b] = True
    return y, mass, inside


def peaks(x, w, offsets, M, rows=None):
    """The greatest |x[k] w[k]| of each sum of `grouped`, as float32."""
    out = torch.zeros(M, w.shape[1], device=x.device)
    src = (x if rows is None else x[rows.long().clamp(0, x.shape[0] - 1)]).abs().float()
    w = w.abs().float()
    step = max(1, (1 << 27) // (w.shape[1] * w.shape[2]))
    for g, a, b in groups_of(offsets, M):
        for i in range(a, b, step):
            j = min(b, i + step)
            out[i:j] = (src[i:j, None, :] * w[g][None]).amax(2)
    return out.double()


def assert_close(got, ref, mass, K, exact_sums=False, peak=None, what=""):
    """One bf16 rounding of a sum of K terms in f32: K additions, each off by at
    most a unit in the last place (2^-23) of a partial sum that is at most
    `mass`, 4 more roundings for the scales and the bias, then half a step of
    bf16.  exact_sums: the sum itself is exact (int32).

    peak: the greatest product of each sum, for e4m3.  The matrix unit lines the
    products of 16 of a row's e4m3 codes up with the one of the greatest
    exponent and cuts them off 13 bits below its leading bit: 2^16 and -2^16
    beside it leave 2^3 + 2^2 + 2^1 as 2^3, and nothing of what is below 2^3
    (whatever kernel issues the instruction; products of 4-bit values, whole
    multiples of 1/4 up to 36, fit).  Each of the K products is then off by
    less than 2^-13 of a product that is at most `peak`."""
    u = (4 if exact_sums else K + 4) * 2.0 ** -23
    low = u * mass
    if peak is not None:
        low = low + K * 2.0 ** -13 * peak
    bound = low + BF16_HALF_STEP * (ref.abs() + low)
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), float((off - bound).max()))


# (type, kernel of probe_grouped_kernel, M, E, N, K): every kernel, each with a K
# that fills its ring of stages (the last of a pair) and one that ends inside
KERNELS = []
for _kernel, _M, _E, _N, _K8, _K4 in (
        (0, 37, 3, 100, (160, 512), (160, 1024)), (1, 5, 9, 8200, (1056, 1024), (1056, 2048)),
        (2, 500, 3, 516, (160, 512), (160, 1024)), (3, 700, 9, 1000, (2080, 2048), (2080, 2048)),
        (4, 250, 9, 2000, (160, 512), ()), (4, 70, 3, 8200, (), (1056, 2048)),
        (4, 500, 1, 4100, (2080, 2048), (2080, 4096)), (5, 1400, 1, 4100, (1056, 1024), (2080, 2048)),
        (5, 100, 9, 4100, (160, 512), (160, 1024)), (6, 12000, 9, 2000, (1056,), (2048,)),
        (6, 6000, 1, 4100, (1056, 2048), (2080, 2048)), (7, 2000, 1, 8200, (2080, 2048), (2080, 2048)),
        (7, 12000, 3, 4100, (4128, 4096), (8224, 8192))):
    for _type in ("int8", "e4m3", "mx"):
        for _K in _K4 if _type == "mx" else _K8:
            KERNELS.append((_type, _kernel, _M, _E, _N, _K))


def uneven(M, E):
    """Lengths of E groups, M in all: one empty, one of a single row where there are enough."""
    out = [M // E] * E
    out[-1] += M - sum(out)
    if E > 2:
        out[0] += out[1]
        out[1] = 0
    if E > 4:
        out[2] += out[3] - 1
        out[3] = 1
    return out
