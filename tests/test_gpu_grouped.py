"""Products of groups of rows (experts) on the GPU, in 8 bits and in the 4-bit
format, against their definition in 64 bits."""
import random

import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu
TYPES = ["int8", "e4m3", "mx"]


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as w8
    return w8


class Case:
    """Operands of one product: codes, scales, their 64-bit values."""

    def __init__(self, kind, X, E, N, K, seed, channels=False, whole=False):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.X, self.E, self.N, self.K = kind, X, E, N, K
        if kind == "mx":
            lo, hi = (128, 130) if whole else (120, 134)
            self.xq, self.xs = ref.random_mx(g, (X, K), lo, hi)
            self.wq, self.ws = ref.random_mx(g, (E, N, K), lo, hi)
            self.x, self.w = ref.values(self.xq, self.xs), ref.values(self.wq, self.ws)
        else:
            if kind == "int8":
                self.xq = torch.randint(-128, 128, (X, K), generator=g, dtype=torch.int8).cuda()
                self.wq = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8).cuda()
            elif whole:
                self.xq = torch.randint(-8, 9, (X, K), generator=g).float().to(torch.float8_e4m3fn).cuda()
                self.wq = torch.randint(-8, 9, (E, N, K), generator=g).float().to(torch.float8_e4m3fn).cuda()
            else:
                self.xq = torch.randn(X, K, generator=g).mul(30).to(torch.float8_e4m3fn).cuda()
                self.wq = torch.randn(E, N, K, generator=g).mul(30).to(torch.float8_e4m3fn).cuda()
            shape = (E, N) if channels else (E,)
            if whole:
                self.xs = torch.pow(2.0, torch.randint(-3, 4, (X,), generator=g).float()).cuda()
                self.ws = torch.pow(2.0, torch.randint(-3, 4, shape, generator=g).float()).cuda()
            else:
                self.xs = (torch.rand(X, generator=g) + 0.1).cuda()
                self.ws = (torch.rand(shape, generator=g) + 0.1).cuda()
            s = self.ws.double()[..., None] if channels else self.ws.double()[:, None, None]
            self.x, self.w = self.xq.double() * self.xs.double()[:, None], self.wq.double() * s
        self.bias = torch.randn(E, N, generator=g).mul(3).bfloat16().cuda()

    def run(self, w8, offsets, rows=None, bias=None, out=None):
        f = w8.mxfp4_linear_grouped if self.kind == "mx" else w8.w8a8_linear_grouped
        return f(self.xq, self.xs, self.wq, self.ws, offsets, rows=rows, bias=bias, out=out)

    def check(self, w8, offsets, M, rows=None, bias=None, exact=False):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        out = torch.full((M, self.N), 7.25, dtype=torch.bfloat16, device="cuda")
        y = self.run(w8, off, rows, bias, out)
        assert y is out
        want, mass, inside = ref.grouped(self.x, self.w, offsets, M, rows, bias)
        assert bool((y[~inside] == 7.25).all()), "rows in no group"
        if exact:
            assert torch.equal(y[inside].float(), want[inside].float().bfloat16().float())
        else:
            peak = ref.peaks(self.x, self.w, offsets, M, rows)[inside] if self.kind == "e4m3" else None
            ref.assert_close(y[inside], want[inside], mass[inside], self.K, exact_sums=self.kind == "int8", peak=peak)
        return y


def _offsets(lengths, first=0):
    out = [first]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _rows(M, X, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, X, (M,), generator=g, dtype=torch.int32).cuda()


# lengths of the groups, N, K
GROUPS = [
    ([1], 1, 32), ([1], 1024, 1024), ([0, 1, 0], 15, 64), ([3, 0, 1, 5], 40, 96), ([16, 17, 15, 1, 0, 2], 257, 160),
    ([1] * 8, 520, 4096), ([33, 64, 65, 1], 130, 288), ([0, 0, 0], 64, 64), ([200, 0, 3], 100, 544),
    ([2, 300, 61], 264, 1056), ([129] * 3, 256, 256), ([513, 40, 0, 255], 300, 512), ([700], 520, 768),
    ([1500, 0, 700, 2001], 4100, 96), ([4200], 4104, 544), ([90, 8000], 2056, 256),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lengths,N,K", GROUPS)
def test_groups(w8, kind, lengths, N, K):
    print(f"[groups] {kind} {lengths} {N} {K}", flush=True)
    M = sum(lengths)
    c = Case(kind, max(M, 1), len(lengths), N, K, seed=N + K)
    offsets = _offsets(lengths)
    if M:
        c.check(w8, offsets, M)
        c.check(w8, offsets, M, bias=c.bias)
    # a shuffled subset of x, rows before and behind the groups, an odd number of rows of x
    c = Case(kind, M // 2 + 3, len(lengths), N, K, seed=N + K + 1, channels=kind != "mx")
    c.check(w8, _offsets(lengths, 2), M + 5, rows=_rows(M + 5, c.X, K), bias=c.bias)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lengths,N,K", GROUPS)
def test_whole_numbers_are_exact(w8, kind, lengths, N, K):
    """int8 sums are whole; e4m3 codes -8 .. 8 and 4-bit values at scales 2 and 4
    have whole products whose sums stay below 2^24 (4096 * 576 = 2.4e6):
    any order of addition gives the exact sum, powers of two scale it exactly.
    int8: 4096 * 2^14 = 2^26 is rounded once to f32 and once to bf16, as the
    reference is by way of float."""
    M = sum(lengths)
    if M == 0:
        pytest.skip("no rows")
    c = Case(kind, M, len(lengths), N, K, seed=3 * N + K, whole=True)
    c.check(w8, _offsets(lengths), M, exact=True)
    c.check(w8, _offsets(lengths), M, rows=_rows(M, M, N), exact=True)


@pytest.mark.parametrize("kind,kernel,M,E,N,K", ref.KERNELS)
def test_every_kernel(w8, kind, kernel, M, E, N, K):
    """Each kernel with whole numbers, exactly, and with random ones; rows in
    order and gathered, rows in no group, a bias, scales of both shapes."""
    print(f"[groups] {kind} kernel {kernel}: {M} {E} {N} {K}", flush=True)
    assert w8.probe_grouped_kernel(kind, M, N, K, E) == kernel
    offsets = _offsets(ref.uneven(M, E))
    c = Case(kind, M, E, N, K, seed=kernel, whole=True)
    c.check(w8, offsets, M, exact=True)
    offsets[0], offsets[-1] = 1, M - 1
    c.check(w8, offsets, M, rows=_rows(M, M, K), exact=True)
    c = Case(kind, M // 2 + 1, E, N, K, seed=kernel + 1, channels=kind != "mx")
    rows = _rows(M, c.X, K)
    rows[M // 3], rows[M // 2] = -1, c.X
    c.check(w8, offsets, M, rows=rows, bias=c.bias)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("E,M", [(64, 100), (65, 100), (130, 200), (1000, 700), (4096, 300)])
def test_many_groups(w8, kind, E, M):
    print(f"[groups] {kind} E={E}", flush=True)
    rng = random.Random(E)
    lengths = [0] * E
    for _ in range(M):
        lengths[rng.randrange(E)] += 1
    c = Case(kind, M, E, 24, 64, seed=E)
    c.check(w8, _offsets(lengths), M, bias=c.bias)
    # one group far back has nearly all
    lengths = [0] * E
    lengths[0], lengths[E - 2], lengths[E - 1] = 1, M - 2, 1
    c.check(w8, _offsets(lengths), M, rows=_rows(M, M, E))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("E,M,N,K", [(70, 3000, 1100, 160), (300, 20000, 260, 96), (200, 30000, 2100, 512)])
def test_many_groups_with_many_rows(w8, kind, E, M, N, K):
    """More groups than a wave's lanes, in the kernels whose workgroups walk
    from tile to tile: the window of groups moves on, and back where tiles that
    advance together lie on both sides of its edge."""
    assert w8.probe_grouped_kernel(kind, M, N, K, E) >= 4
    rng = random.Random(E)
    lengths = [0] * E
    for g in rng.choices(range(E), [rng.random() ** 3 for _ in range(E)], k=M):
        lengths[g] += 1
    c = Case(kind, M, E, N, K, seed=E, whole=True)
    c.check(w8, _offsets(lengths), M, exact=True)
    c.check(w8, _offsets(lengths), M, rows=_rows(M, M, E), exact=True)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N", [(60, 40), (700, 300)])
def test_integers_that_make_no_sense(w8, kind, M, N):
    """Offsets that fall, lie outside [0, M] or overlap, and row indices outside
    x: what the header says of them, and nothing out of range."""
    E, K = 5, 96
    c = Case(kind, M, E, N, K, seed=4)
    big = 2 ** 31 - 1
    for offsets in ([0, 10, 5, M - 20, M - 10, M], [-5, -1, 7, 7, 3 * M, 4 * M], [M, 0, 0, 0, 0, 0], [big] * 6,
                    [-big] * 6, [-big, big, -big, big, 0, M], [3, 2, 1, 0, -1, 50]):
        print(f"[groups] {kind} {offsets}", flush=True)
        c.check(w8, offsets, M, bias=c.bias)
    rows = _rows(M, M, 5)
    rows[3], rows[4], rows[11], rows[M - 1], rows[M // 2] = -1, M, big, -big, M + 1
    c.check(w8, [0, 10, 20, 20, M - 3, M], M, rows=rows, bias=c.bias)


def test_one_group_of_int8_is_the_linear(w8):
    for M, N, K in ((5, 40, 64), (300, 264, 512)):
        c = Case("int8", M, 1, N, K, seed=6)
        y = c.run(w8, torch.tensor([0, M], dtype=torch.int32, device="cuda"), bias=c.bias)
        assert torch.equal(y, w8.w8a8_linear(c.xq, c.xs, c.wq[0], c.ws, c.bias[0]))


def test_one_group_of_mx_is_the_linear(w8):
    for M, N, K in ((5, 40, 64), (300, 264, 512)):
        c = Case("mx", M, 1, N, K, seed=6)
        y = c.run(w8, torch.tensor([0, M], dtype=torch.int32, device="cuda"), bias=c.bias)
        assert torch.equal(y, w8.mxfp4_linear(c.xq, c.xs, c.wq[0], c.ws[0], c.bias[0]))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M", [40, 600])
def test_a_nan_stays_in_its_row(w8, kind, M):
    c = Case(kind, M, 3, 70, 160, seed=8)
    offsets = torch.tensor([0, 9, 9, M], dtype=torch.int32, device="cuda")
    clean = c.run(w8, offsets)
    c.xs.view(-1)[(c.xs.stride(0) if kind == "mx" else 1) * 5] = 255 if kind == "mx" else float("nan")
    y = c.run(w8, offsets)
    nan = torch.isnan(y)
    assert bool(nan[5].all()) and int(nan.sum()) == 70 and torch.equal(y[~nan], clean[~nan])


@pytest.mark.parametrize("qtype", [0, 1])
def test_weights_of_groups(w8, qtype):
    g = torch.Generator().manual_seed(3)
    w = torch.randn(3, 48, 64, generator=g).bfloat16().cuda()
    wq, wt, s = w8.w8a8_quant_weight_grouped(w, qtype, transposed=True)
    assert s.shape == (3,)
    for e in range(3):
        a, b, c = w8.w8a8_quant_weight_tensorwise(w[e], qtype, transposed=True)
        assert torch.equal(a.view(torch.uint8), wq[e].view(torch.uint8))
        assert torch.equal(b.view(torch.uint8), wt[e].view(torch.uint8)) and torch.equal(c, s[e:e + 1])


@pytest.mark.parametrize("kind", TYPES)
def test_backward_is_the_gradient(w8, kind):
    """dX against the transposed operands' values; and for int8, whose forward
    and backward weights are the same values, <dX, V> against the difference of
    the forward product along V (linear: exact but for roundings)."""
    lengths, N, K = [20, 0, 70, 3], 96, 128
    M, E = sum(lengths), len(lengths)
    offsets = _offsets(lengths)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(9)
    w = (torch.randn(E, N, K, generator=g) * 0.1).bfloat16().cuda()
    dy = torch.randn(M, N, generator=g).bfloat16().cuda()
    if kind == "mx":
        dq, ds = w8.mxfp4_quantize(dy)
        wt, ws = w8.mxfp4_quantize_transposed(w)
        dx = w8.mxfp4_linear_grouped_backward_dx(dq, ds, wt, ws, off)
        d, wv = ref.values(dq, ds), ref.values(wt, ws)
    else:
        qt = w8.INT8 if kind == "int8" else w8.FP8_E4M3
        wq, wt, ws = w8.w8a8_quant_weight_grouped(w, qt, transposed=True)
        dq, ds = w8.w8a8_quant_act_rowwise(dy, qt)
        dx = w8.w8a8_linear_grouped_backward_dx(dq, ds, wt, ws, off)
        d, wv = dq.double() * ds.double()[:, None], wt.double() * ws.double()[:, None, None]
    want, mass, _ = ref.grouped(d, wv, offsets, M)
    peak = ref.peaks(d, wv, offsets, M) if kind == "e4m3" else None
    ref.assert_close(dx, want, mass, N, exact_sums=kind == "int8", peak=peak)
    if kind != "int8":
        return
    x = torch.randint(-100, 100, (M, K), generator=g, dtype=torch.int8).cuda()
    v = torch.randint(-20, 21, (M, K), generator=g, dtype=torch.int8).cuda()
    one = torch.ones(M, device="cuda")
    up = w8.w8a8_linear_grouped(x + v, one, wq, ws, off).double()
    down = w8.w8a8_linear_grouped(x - v, one, wq, ws, off).double()
    lhs = (d * (up - down) / 2).sum()
    rhs = (dx.double() * v.double()).sum()
    half = ref.BF16_HALF_STEP
    room = half * ((d.abs() * (up.abs() + down.abs()) / 2).sum() + (dx.double().abs() * v.double().abs()).sum())
    assert float((lhs - rhs).abs()) <= 1.01 * float(room)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lengths", [[3, 1, 0, 2], [300, 0, 41, 200]])
def test_captured_with_new_routing(w8, kind, lengths):
    """A captured call replayed with other rows and offsets: the grid knows the
    sizes alone, what lies on the device decides."""
    M, E, N, K = sum(lengths), 4, 72, 160
    c = Case(kind, M, E, N, K, seed=11)
    off = torch.tensor(_offsets(lengths), dtype=torch.int32, device="cuda")
    rows = _rows(M, M, 1)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(w8, off, rows, c.bias, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(w8, off, rows, c.bias, out)
    rng = random.Random(2)
    for i in range(4):
        cuts = sorted(rng.randint(0, M) for _ in range(E - 1))
        off.copy_(torch.tensor([0] + cuts + [M], dtype=torch.int32))
        rows.copy_(_rows(M, M, 20 + i))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run(w8, off, rows, c.bias)), i


def _uneven_offsets(M, E):
    """What no estimate foresees: every row in the last group, in the first; a few rows; none; a range that runs
    backwards; rows in the middle alone."""
    return [[0] * E + [M], [0] + [M] * E, [0] + [37] * E, [5] * (E + 1), [0, M // 2, 3] + [M] * (E - 2),
            [M // 3] * E + [M // 3 + 300]]


@pytest.mark.parametrize("kernel", range(8))
@pytest.mark.parametrize("kind", TYPES)
def test_any_offsets_in_every_kernel(w8, kind, kernel):
    """The kernel is chosen by the sizes alone, so each has to take whatever lies in `offsets`: eager, and captured
    with other offsets."""
    M, E, N, K = next(k[2:] for k in ref.KERNELS if k[:2] == (kind, kernel) and k[3] > 2)
    c = Case(kind, M, E, N, K, seed=kernel, whole=True)
    off = torch.tensor(_offsets(ref.uneven(M, E)), dtype=torch.int32, device="cuda")
    out = torch.full((M, N), 7.25, dtype=torch.bfloat16, device="cuda")
    c.run(w8, off, None, None, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(w8, off, None, None, out)
    for offsets in _uneven_offsets(M, E):
        y = c.check(w8, offsets, M, exact=True)
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        out.fill_(7.25)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y), offsets


@pytest.mark.parametrize("kind", TYPES)
def test_two_calls_at_once(w8, kind):
    a, b = Case(kind, 90, 3, 200, 256, seed=1), Case(kind, 400, 2, 264, 512, seed=2)
    oa = torch.tensor([0, 30, 31, 90], dtype=torch.int32, device="cuda")
    ob = torch.tensor([0, 260, 400], dtype=torch.int32, device="cuda")
    ya, yb = a.run(w8, oa), b.run(w8, ob)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            za = a.run(w8, oa)
        zb = b.run(w8, ob)
        torch.cuda.synchronize()
        assert torch.equal(ya, za) and torch.equal(yb, zb)


def test_nothing_to_do(w8):
    c = Case("int8", 4, 2, 8, 32, seed=0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert c.run(w8, off, rows=none).shape == (0, 8)
    e = torch.zeros(0, 32, dtype=torch.int8, device="cuda")
    f = torch.zeros(0, device="cuda")
    assert w8.w8a8_linear_grouped(e, f, c.wq, c.ws, off).shape == (0, 8)
    # rows of an x that has none: every index is outside it
    y = w8.w8a8_linear_grouped(e, f, c.wq, c.ws, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"),
                               rows=torch.zeros(2, dtype=torch.int32, device="cuda"), bias=c.bias)
    assert torch.equal(y, c.bias)


def test_refusals(w8):
    c, m = Case("int8", 4, 2, 8, 32, seed=0), Case("mx", 4, 2, 8, 64, seed=0)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for k in (c, m):
        with pytest.raises(TypeError, match="int32"):
            k.run(w8, off.long())
        with pytest.raises(ValueError, match="offsets"):
            k.run(w8, off[:2])
        with pytest.raises(ValueError, match="bias"):
            k.run(w8, off, bias=k.bias[0])
        with pytest.raises(TypeError, match="rows"):
            k.run(w8, off, rows=off.long())
        with pytest.raises(ValueError, match="out"):
            k.run(w8, off, out=torch.zeros(4, 9, dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(ValueError, match="offsets"):
            k.run(w8, off.cpu())
    with pytest.raises(TypeError, match="codes"):
        w8.w8a8_linear_grouped(c.xq, c.xs, c.wq.to(torch.float8_e4m3fn), c.ws, off)
    with pytest.raises(ValueError, match="share K"):
        w8.w8a8_linear_grouped(c.xq[:, :16].contiguous(), c.xs, c.wq, c.ws, off)
    with pytest.raises(ValueError, match="w_scale"):
        w8.w8a8_linear_grouped(c.xq, c.xs, c.wq, c.ws[:1], off)
    with pytest.raises(ValueError, match="x_scale"):
        w8.w8a8_linear_grouped(c.xq, c.xs[:3], c.wq, c.ws, off)
    with pytest.raises(ValueError, match="3-D"):
        w8.w8a8_linear_grouped(c.xq, c.xs, c.wq[0], c.ws, off)
