"""Every kernel of the products of groups (named by probe_grouped_kernel) with
what can go wrong in one and not in another: NaN and padding, a bias and
scales of every shape, indices and offsets that make no sense, graphs, streams.

Operands are whole numbers and powers of two, so that every result is known bit
by bit: codes -8 .. 8 (4-bit format: every code, scales 2 and 4) have products
that are whole multiples of 1 up to 64 (576), their sums over K <= 8224 stay
below 2^24 in any order (8224 * 576 = 4.7e6), scales 2^-3 .. 2^3 of rows and
weights only move the exponent, and one rounding to f32 (the multiply-add that
takes the bias) and one to bf16 remain: those of `want`."""
import random

import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu
KERNELS = ref.KERNELS
# one shape of each kernel that has several groups and a K that ends inside a stage
SEVERAL = [next(k for k in KERNELS if k[:2] == (kind, kernel) and k[3] > 2)
           for kind in ("int8", "e4m3", "mx") for kernel in range(8)]
MX = [k for k in KERNELS if k[0] == "mx"]
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as w8
    yield w8
    torch.cuda.empty_cache()


class Whole:
    """Operands of one product, X rows of x."""

    def __init__(self, kind, X, E, N, K, seed, channels=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.X, self.E, self.N, self.K = kind, X, E, N, K

        def integers(lo, hi, *shape):
            return torch.randint(lo, hi, shape, generator=g, device="cuda")

        if kind == "mx":
            self.xq, self.wq = integers(0, 256, X, K // 2).to(torch.uint8), integers(0, 256, E, N, K // 2).to(torch.uint8)
            self.xs = integers(128, 130, X, ref.stride_of(K)).to(torch.uint8)
            self.ws = integers(128, 130, E, N, ref.stride_of(K)).to(torch.uint8)
        else:
            code = torch.int8 if kind == "int8" else torch.float8_e4m3fn
            self.xq, self.wq = integers(-8, 9, X, K).to(torch.float32).to(code), integers(-8, 9, E, N, K).to(torch.float32).to(code)
            self.xs = torch.pow(2.0, integers(-3, 4, X).float())
            self.ws = torch.pow(2.0, integers(-3, 4, *((E, N) if channels else (E,))).float())
        self.bias = integers(-100, 101, E, N).bfloat16()

    def run(self, w8, offsets, rows=None, bias=None, out=None):
        f = w8.mxfp4_linear_grouped if self.kind == "mx" else w8.w8a8_linear_grouped
        return f(self.xq, self.xs, self.wq, self.ws, offsets, rows=rows, bias=bias, out=out)

    def weight(self, g):
        if self.kind == "mx":
            return ref.values(self.wq[g], self.ws[g])
        s = self.ws[g].double()
        return self.wq[g].double() * (s[:, None] if s.dim() else s)

    def want(self, offsets, M, rows=None, bias=None, rest=7.25):
        """(the result, `rest` in rows of no group) in 64 bits."""
        x = ref.values(self.xq, self.xs) if self.kind == "mx" else self.xq.double() * self.xs.double()[:, None]
        if rows is not None:
            r = rows.long()
            inside = (r >= 0) & (r < self.X)
            x = torch.where(inside[:, None], x[r.clamp(0, self.X - 1)], 0.0)
        y = torch.full((M, self.N), rest, dtype=torch.float64, device="cuda")
        for g, a, b in ref.groups_of(offsets, M):
            if b > a:
                y[a:b] = x[a:b] @ self.weight(g).T
                if bias is not None:
                    y[a:b] += bias[g].double()
        return y

    def check(self, w8, offsets, M, rows=None, bias=None):
        out = torch.full((M, self.N), 7.25, dtype=torch.bfloat16, device="cuda")
        y = self.run(w8, _device(offsets), rows, bias, out)
        assert torch.equal(y, _rounded(self.want(offsets, M, rows, bias))), (self.kind, offsets)
        return y


def _rounded(want):
    return want.float().bfloat16()


def _device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def _even(M, E):
    out = [0]
    for n in ref.uneven(M, E):
        out.append(out[-1] + n)
    return out


def _rows(M, X, seed):
    return torch.randint(0, X, (M,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


def _named(w8, kind, kernel, M, E, N, K):
    print(f"[kernels] {kind} {kernel}: {M} {E} {N} {K}", flush=True)
    assert w8.probe_grouped_kernel(kind, M, N, K, E) == kernel


@pytest.mark.parametrize("kind,kernel,M,E,N,K", KERNELS)
def test_bias_and_scales_bit_by_bit(w8, kind, kernel, M, E, N, K):
    """A bias alone, a bias beside scales of each output channel, in order and
    gathered."""
    _named(w8, kind, kernel, M, E, N, K)
    offsets = _even(M, E)
    c = Whole(kind, M, E, N, K, seed=kernel)
    c.check(w8, offsets, M, bias=c.bias)
    c = Whole(kind, M // 2 + 1, E, N, K, seed=kernel + 1, channels=kind != "mx")
    offsets[0], offsets[-1] = 1, M - 1
    c.check(w8, offsets, M, rows=_rows(M, c.X, K))
    c.check(w8, offsets, M, rows=_rows(M, c.X, K), bias=c.bias)


@pytest.mark.parametrize("kind,kernel,M,E,N,K", KERNELS)
def test_random_products_near_the_definition(w8, kind, kernel, M, E, N, K):
    """Relative Frobenius error 1e-3 against the definition rounded to bf16, this
    library's measure of a product.  A result differs from the rounded
    definition where a border between two bf16 values lies between the sums: by
    a step s (2^-7 of the value at most) with the probability d / s of a
    deviation d, so d may be 1e-6 of 2^-7, 1.3e-4 of the value.  f32 sums of 8224
    terms stay far below it (2^-24 a term, at random: 6e-6); e4m3: products of 8
    codes lose less than 2^-13 of the greatest of them each, evenly spread: 2^-13
    / sqrt(3) = 7e-5 times the greatest of 8 products of normal values in units
    of their root mean square, below 3, and of the products the half that lies
    below 2^-5 of the greatest (those above lose nothing): 1.5e-4 of the sum's
    own root mean square, an upper estimate."""
    _named(w8, kind, kernel, M, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(kernel)
    X = M // 2 + 1
    x = torch.randn((X, K), generator=g, device="cuda")
    w = torch.randn((E, N, K), generator=g, device="cuda") * 0.05
    bias = torch.randn((E, N), generator=g, device="cuda").bfloat16()
    c = Whole(kind, 1, 1, 1, 512, seed=0)
    c.X, c.E, c.N, c.K = X, E, N, K
    if kind == "mx":
        c.xq, c.xs = w8.mxfp4_quantize(x)
        c.wq, c.ws = w8.mxfp4_quantize(w)
    else:
        top, code = (127.0, torch.int8) if kind == "int8" else (448.0, torch.float8_e4m3fn)
        c.xs, c.ws = x.abs().amax(1) / top, w.abs().amax(2) / top
        c.xq, c.wq = x / c.xs[:, None], w / c.ws[..., None]
        if kind == "int8":
            c.xq, c.wq = c.xq.round(), c.wq.round()
        c.xq, c.wq = c.xq.clamp(-top, top).to(code), c.wq.clamp(-top, top).to(code)
    offsets, rows = _even(M, E), _rows(M, X, K)
    y = c.run(w8, _device(offsets), rows, bias)
    want = _rounded(c.want(offsets, M, rows, bias)).double()
    off = float((y.double() - want).norm() / want.norm())
    assert off <= 1e-3, off


@pytest.mark.parametrize("kind,kernel,M,E,N,K", MX)
def test_nan_scales_and_padding(w8, kind, kernel, M, E, N, K):
    """4-bit format: bytes past a row's scales may be NaN, a NaN scale in a row's
    last block (and its first) makes that row NaN, one of a weight's row that
    column of its group, and nothing else."""
    _named(w8, kind, kernel, M, E, N, K)
    offsets = _even(M, E)
    c = Whole(kind, M, E, N, K, seed=kernel + 2)
    clean = c.check(w8, offsets, M, bias=c.bias)
    blocks = K // 32
    c.xs[:, blocks:] = 255
    c.ws[..., blocks:] = 255
    off = _device(offsets)
    assert torch.equal(c.run(w8, off, bias=c.bias), clean), "padding"
    group = E - 1
    row, column = offsets[group] + (M - offsets[group]) // 2, N - 1
    c.xs[row, blocks - 1], c.xs[0, 0] = 255, 255
    c.ws[group, column, blocks - 1], c.ws[group, 0, 0] = 255, 255
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[row], nan[0] = True, True
    nan[offsets[group]:, column], nan[offsets[group]:, 0] = True, True
    calls = [lambda: c.run(w8, off, bias=c.bias)]
    if E == 1:
        calls.append(lambda: w8.mxfp4_linear(c.xq, c.xs, c.wq[0], c.ws[0], c.bias[0]))
    for call in calls:
        y = call()
        assert torch.equal(torch.isnan(y), nan)
        assert torch.equal(y[~nan], clean[~nan])
    # gathered, in another order
    rows = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    want = torch.isnan(c.want(offsets, M, rows, c.bias))
    assert torch.equal(torch.isnan(c.run(w8, off, rows=rows, bias=c.bias)), want)


@pytest.mark.parametrize("kind,kernel,M,E,N,K", [k for k in KERNELS if k[0] != "mx"])
def test_nan_scales_and_codes(w8, kind, kernel, M, E, N, K):
    """8 bits: a row's NaN scale, a channel's, an e4m3 NaN in the last code of a
    row or of a weight's row."""
    _named(w8, kind, kernel, M, E, N, K)
    offsets = _even(M, E)
    off = _device(offsets)
    c = Whole(kind, M, E, N, K, seed=kernel + 3, channels=True)
    clean = c.check(w8, offsets, M, bias=c.bias)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    group, row = E - 1, M - 1
    c.xs[row] = float("nan")
    c.ws[group, N - 1] = float("nan")
    nan[row], nan[offsets[group]:, N - 1] = True, True
    if kind == "e4m3":
        c.xq.view(torch.uint8)[1, K - 1] = 0x7F
        c.wq.view(torch.uint8)[group, 0, K - 1] = 0xFF
        nan[1], nan[offsets[group]:, 0] = True, True
    y = c.run(w8, off, bias=c.bias)
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y[~nan], clean[~nan])
    one = Whole(kind, M, E, N, K, seed=kernel + 4)
    clean = one.check(w8, offsets, M)
    one.ws[group] = float("nan")
    y = one.run(w8, off)
    assert bool(torch.isnan(y[offsets[group]:]).all()) and torch.equal(y[:offsets[group]], clean[:offsets[group]])


@pytest.mark.parametrize("kind,kernel,M,E,N,K", SEVERAL)
def test_integers_that_make_no_sense(w8, kind, kernel, M, E, N, K):
    """Row indices outside x give the bias alone, exactly; offsets that fall, lie
    outside [0, M] or overlap are what the header says of them; both at once."""
    _named(w8, kind, kernel, M, E, N, K)
    X = M // 3 + 2
    c = Whole(kind, X, E, N, K, seed=kernel + 5, channels=kind != "mx")
    rows = _rows(M, X, kernel)
    rng = random.Random(kernel)
    bad = [-1, X, BIG, -BIG, -BIG - 1, X + 1, -X, BIG - 255]
    at = rng.sample(range(M), min(M, max(8, M // 5)))
    rows[torch.tensor(at, device="cuda")] = torch.tensor([bad[i % len(bad)] for i in range(len(at))], dtype=torch.int32,
                                                         device="cuda")
    y = c.check(w8, _even(M, E), M, rows=rows, bias=c.bias)
    starts = _device(_even(M, E)).cummax(0).values
    group = torch.searchsorted(starts, torch.tensor(at, dtype=torch.int32, device="cuda"), right=True) - 1
    assert torch.equal(y[at], c.bias[group])
    middle = [0] + [M // 2] * (E - 1) + [M]
    for offsets in ([-5] * (E // 2) + [7, 3] + [3 * M] * (E - E // 2 - 1), [M] + [0] * E, [BIG] * (E + 1),
                    [-BIG] * (E + 1), [-BIG, BIG, -BIG] + [0] * (E - 3) + [M], [M - 3] + [-BIG - 1] * (E - 1) + [BIG],
                    middle):
        c.check(w8, offsets, M, rows=rows, bias=c.bias)
    rows.fill_(BIG)
    c.check(w8, middle, M, rows=rows, bias=c.bias)


@pytest.mark.parametrize("kind,kernel,M,E,N,K", SEVERAL)
def test_a_captured_gather_with_new_routing(w8, kind, kernel, M, E, N, K):
    """One graph, replayed with other rows and offsets, eager calls between."""
    _named(w8, kind, kernel, M, E, N, K)
    c = Whole(kind, M // 2 + 1, E, N, K, seed=kernel + 6, channels=kind != "mx")
    off, rows = _device(_even(M, E)), _rows(M, c.X, 1)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    c.run(w8, off, rows, c.bias, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(w8, off, rows, c.bias, out)
    rng = random.Random(2)
    for i in range(4):
        offsets = [0] + sorted(rng.randint(0, M) for _ in range(E - 1)) + [M - i]
        offsets[-2] = min(offsets[-2], M - i)
        off.copy_(_device(offsets))
        rows.copy_(_rows(M, c.X, 20 + i))
        out.fill_(7.25)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _rounded(c.want(offsets, M, rows, c.bias))), i
        assert torch.equal(out, c.run(w8, off, rows, c.bias, torch.full_like(out, 7.25))), i


@pytest.mark.parametrize("kind,kernel,M,E,N,K", SEVERAL)
def test_two_streams_at_once(w8, kind, kernel, M, E, N, K):
    """The same kernel on two streams with other operands and outputs."""
    _named(w8, kind, kernel, M, E, N, K)
    offsets = _even(M, E)
    off = _device(offsets)
    a, b = Whole(kind, M, E, N, K, seed=kernel + 7), Whole(kind, M // 2 + 1, E, N, K, seed=kernel + 8)
    rows = _rows(M, b.X, 3)
    want = _rounded(a.want(offsets, M)), _rounded(b.want(offsets, M, rows, b.bias))
    outs = [[torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)] for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(3):
        with torch.cuda.stream(side):
            a.run(w8, off, out=outs[0][i])
        b.run(w8, off, rows, b.bias, outs[1][i])
    torch.cuda.synchronize()
    for i in range(3):
        assert torch.equal(outs[0][i], want[0]) and torch.equal(outs[1][i], want[1]), i


@pytest.mark.parametrize("kind,kernel,M,E,N,K", SEVERAL)
def test_rows_of_an_x_that_has_none(w8, kind, kernel, M, E, N, K):
    """Every index is outside x, whose tensors have no storage: the bias alone."""
    _named(w8, kind, kernel, M, E, N, K)
    c = Whole(kind, 1, E, N, K, seed=kernel + 9)
    c.xq, c.xs = c.xq[:0].clone(), c.xs[:0].clone()
    offsets = _even(M, E)
    rows = torch.arange(-1, M - 1, dtype=torch.int32, device="cuda")
    y = c.run(w8, _device(offsets), rows, c.bias)
    group = torch.cat([torch.full((b - a,), g, device="cuda") for g, a, b in ref.groups_of(offsets, M)])
    assert torch.equal(y, c.bias[group])
