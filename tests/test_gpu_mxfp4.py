"""The microscaled 4-bit format on the GPU against its definition in 64 bits."""
import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as w8
    return w8


def _same(got, want, what):
    codes, scale = want
    assert torch.equal(got[1].cpu(), scale), what + " scales"
    assert torch.equal(got[0].cpu(), ref.pack(codes)), what + " codes"


def _inputs(M, K, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, ::7] *= 40
    x[torch.rand(M, K, generator=g) < 0.05] = 0
    if M > 1:
        x[1] *= 2.0 ** -40
    return x.to(dtype)


SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (1, 100), (65, 128), (4, 511), (4, 512), (7, 513), (130, 1000), (9, 2080),
          (300, 64), (17, 4096)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize(w8, M, K, dtype):
    print(f"[mx] quantize {M}x{K} {dtype}", flush=True)
    x = _inputs(M, K, M + K, dtype)
    _same(w8.mxfp4_quantize(x.cuda()), ref.quantize(x), "plain")
    # more columns than K: codes 0, scales of whole blocks of zeros
    ldq = K + (-K) % 32 + 64
    _same(w8.mxfp4_quantize(x.cuda(), ldq=ldq), ref.quantize(x, ldq), "wide")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_a_view_with_odd_rows(w8, dtype):
    big = _inputs(37, 203, 5, dtype).cuda()
    _same(w8.mxfp4_quantize(big[:, :77]), ref.quantize(big[:, :77].contiguous()), "view")
    assert w8.mxfp4_quantize(big[:0, :77])[0].shape == (0, 48)
    # leading dimensions
    x = _inputs(24, 96, 6, dtype).cuda()
    q, s = w8.mxfp4_quantize(x.view(2, 3, 4, 96))
    assert q.shape == (2, 3, 4, 48) and s.shape == (2, 3, 4, 16)
    _same((q.view(24, 48), s.view(24, 16)), ref.quantize(x), "leading")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_border(w8, dtype):
    """Blocks whose first value fixes the scale, the others on, just below and
    just above each border between codes, of both signs, at scales from the
    smallest to the largest."""
    mags = [0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.5]
    eps = 2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -20
    row = [4.0]
    for m in mags:
        row += [m, m * (1 + eps), m * (1 - eps / 2)]
    row += [-v for v in row]
    rows = []
    for lead in (4.0, 5.0, 6.0, 7.0, 7.5):
        body = [v for v in row if abs(v) < 8]
        blocks = [[lead] + body[i:i + 31] for i in range(0, len(body), 31)]
        blocks[-1] += [0.0] * (32 - len(blocks[-1]))
        rows.append(sum(blocks, []))
    base = torch.tensor(rows, dtype=torch.float64)
    x = torch.cat([base * 2.0 ** k for k in (0, 1, -1, 30, -30, 100, -100, -124, 124, 125, -126, -130, -140, -149)])
    x = x.to(torch.float32).to(dtype)
    assert bool(torch.isfinite(x).all())
    _same(w8.mxfp4_quantize(x.cuda()), ref.quantize(x), "borders")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_and_nan_stay_in_their_block(w8, dtype):
    x = _inputs(6, 160, 9, dtype)
    x[0, 3], x[1, 33], x[2, 159] = float("inf"), float("-inf"), float("nan")
    x[3, 0:32] = 0
    x[4] = 0
    _same(w8.mxfp4_quantize(x.cuda()), ref.quantize(x), "non-finite")
    q, s = w8.mxfp4_quantize(x.cuda())
    back = w8.mxfp4_dequantize(q, s, dtype=dtype).float()
    nan = torch.isnan(back).view(6, 5, 32)
    assert bool(nan[0, 0].all()) and bool(nan[1, 1].all()) and bool(nan[2, 4].all()) and int(nan.sum()) == 96
    t, ts = w8.mxfp4_quantize_transposed(x.T.contiguous().cuda())
    assert torch.equal(t, q) and torch.equal(ts, s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(1, 1), (31, 5), (32, 64), (33, 65), (255, 130), (256, 64), (257, 63), (513, 200),
                                 (1000, 96), (700, 1001)])
def test_quantize_transposed(w8, N, K, dtype):
    print(f"[mx] transposed {N}x{K} {dtype}", flush=True)
    x = _inputs(N, K, N + K, dtype)
    _same(w8.mxfp4_quantize_transposed(x.cuda()), ref.quantize(x.T), "transposed")
    ldq = N + (-N) % 32 + 32
    _same(w8.mxfp4_quantize_transposed(x.cuda(), ldq=ldq), ref.quantize(x.T, ldq), "wide")
    view = torch.zeros(N, K + 3, dtype=dtype)
    view[:, :K] = x
    _same(w8.mxfp4_quantize_transposed(view.cuda()[:, :K]), ref.quantize(x.T), "view")
    three = torch.stack([x, -x, 2 * x]).cuda()
    q, s = w8.mxfp4_quantize_transposed(three)
    for i in range(3):
        _same((q[i], s[i]), ref.quantize(three[i].T), "batch")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_dequantize(w8, M, K, dtype):
    print(f"[mx] dequantize {M}x{K} {dtype}", flush=True)
    ldq = K + (-K) % 32
    q, s = ref.random_mx(torch.Generator().manual_seed(K), (M, ldq), 0, 256)
    want = ref.values(q, s)[:, :K]
    got = w8.mxfp4_dequantize(q, s, K, dtype=dtype)
    # every product is in range of both types but at the largest scales, where it rounds to an infinity
    assert torch.equal(torch.nan_to_num(got.double(), nan=1.25, posinf=9e99, neginf=-9e99),
                       torch.nan_to_num(want.float().to(dtype).double(), nan=1.25, posinf=9e99, neginf=-9e99))
    # into a view: the columns beside it stay
    big = torch.full((M, K + 5), 3.0, dtype=dtype, device="cuda")
    w8.mxfp4_dequantize(q, s, K, out=big[:, :K])
    assert torch.equal(torch.nan_to_num(big[:, :K]), torch.nan_to_num(got)) and bool((big[:, K:] == 3).all())


def test_round_trip_is_a_projection(w8):
    x = _inputs(50, 544, 3, torch.bfloat16).cuda()
    q, s = w8.mxfp4_quantize(x)
    y = w8.mxfp4_dequantize(q, s)
    z = w8.mxfp4_dequantize(*w8.mxfp4_quantize(y))
    assert torch.equal(y, z)


# ------------------------------------------------------------------ product
LINEAR = [(1, 1, 32), (1, 1024, 1024), (2, 15, 64), (16, 16, 96), (17, 40, 256), (33, 100, 288), (48, 257, 480),
          (64, 64, 512), (65, 130, 544), (130, 520, 1056), (257, 300, 2080), (300, 264, 160), (520, 1000, 768),
          (1100, 257, 512),
          (4200, 4100, 32), (4100, 4104, 1056)]


def _operand(g, rows, K, lo=120, hi=134):
    return ref.random_mx(g, (rows, K), lo, hi)


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(w8, M, N, K):
    print(f"[mx] linear {M} {N} {K}", flush=True)
    g = torch.Generator().manual_seed(M * N + K)
    xq, xs = _operand(g, M, K)
    wq, ws = _operand(g, N, K)
    bias = torch.randn(N, generator=g).bfloat16().cuda()
    x, w = ref.values(xq, xs), ref.values(wq, ws)
    want, mass = x @ w.T, x.abs() @ w.abs().T
    ref.assert_close(w8.mxfp4_linear(xq, xs, wq, ws), want, mass, K, what="no bias")
    b = bias.double()
    ref.assert_close(w8.mxfp4_linear(xq, xs, wq, ws, bias), want + b, mass + b.abs(), K, what="bias")


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_of_whole_numbers_is_exact(w8, M, N, K):
    """Scales 2 and 4 of both sides: products are whole multiples of 1/4 * 4 = 1
    up to 36 * 16, their sums below 2^24 (K <= 2080: 1.2e6): exact in f32
    in any order, so the result is the rounded exact sum."""
    g = torch.Generator().manual_seed(M + N + K)
    xq, xs = _operand(g, M, K, 128, 130)
    wq, ws = _operand(g, N, K, 128, 130)
    want = (ref.values(xq, xs) @ ref.values(wq, ws).T).float().bfloat16()
    assert torch.equal(w8.mxfp4_linear(xq, xs, wq, ws).float(), want.float())


@pytest.mark.parametrize("M,N,K", [(1, 20, 64), (20, 70, 160), (70, 40, 544), (300, 300, 1056)])
def test_nan_scales_and_padding(w8, M, N, K):
    """A NaN scale makes its row (its weight row: the column) NaN, bytes past a
    row's scales are never used."""
    g = torch.Generator().manual_seed(K)
    xq, xs = _operand(g, M, K)
    wq, ws = _operand(g, N, K)
    clean = w8.mxfp4_linear(xq, xs, wq, ws)
    xs[:, K // 32:] = 255
    ws[:, K // 32:] = 255
    assert torch.equal(w8.mxfp4_linear(xq, xs, wq, ws), clean)
    xs[M // 2, K // 32 - 1] = 255
    ws[N // 3, 0] = 255
    y = w8.mxfp4_linear(xq, xs, wq, ws)
    nan = torch.isnan(y)
    assert bool(nan[M // 2].all()) and bool(nan[:, N // 3].all()) and int(nan.sum()) == M + N - 1
    assert torch.equal(y[~nan], clean[~nan])


def test_zero_sizes(w8):
    z = torch.zeros(0, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(0, 16, dtype=torch.uint8, device="cuda")
    w, ws = _operand(torch.Generator().manual_seed(0), 8, 64)
    assert w8.mxfp4_linear(z, s, w, ws).shape == (0, 8)
    assert w8.mxfp4_linear(w, ws, z, s).shape == (8, 0)
    assert w8.mxfp4_dequantize(z, s).shape == (0, 64)


def test_backward_is_the_gradient(w8):
    """dX of the quantized product, dY given: the quantized dY times the
    transposed weight's own values, and within the format's rounding of dY . W."""
    M, N, K = 45, 320, 192
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(N, K, generator=g) * 0.05).bfloat16().cuda()
    dy = torch.randn(M, N, generator=g).bfloat16().cuda()
    dyq, dys = w8.mxfp4_quantize(dy)
    wt, wts = w8.mxfp4_quantize_transposed(w)
    dx = w8.mxfp4_linear_backward_dx(dyq, dys, wt, wts)
    a, b = ref.values(dyq, dys), ref.values(wt, wts)
    ref.assert_close(dx, a @ b.T, a.abs() @ b.abs().T, N)
    # a code is off by at most half a step between magnitudes: 1/4 of its value from 1 on (2^-2 relative
    # and saturation, at most 1/4), 1/4 of the scale below: |error| <= 2^-2 |x| + 2^-2 * 2^e, 2^e <= absmax / 4
    def off(v, axis_len):
        blocks = v.double().view(v.shape[0], axis_len // 32, 32)
        return (0.25 * blocks.abs() + 0.0625 * blocks.abs().amax(2, keepdim=True)).view(v.shape)
    da, db = off(dy, N), off(w.T.contiguous(), N)
    exact = dy.double() @ w.double()
    room = da @ w.double().abs() + dy.double().abs() @ db.T + da @ db.T
    assert bool(((dx.double() - exact).abs() <= room + 2.0 ** -7 * exact.abs() + 2.0 ** -7 * room).all())


def test_another_stream_and_the_same_bits(w8):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(70, 512, generator=g).bfloat16().cuda()
    wq, ws = _operand(g, 300, 512)
    first = w8.mxfp4_linear(*w8.mxfp4_quantize(x), wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = w8.mxfp4_linear(*w8.mxfp4_quantize(x), wq, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, second)


def test_refusals(w8):
    q, s = _operand(torch.Generator().manual_seed(0), 8, 64)
    with pytest.raises(ValueError, match="shape"):
        w8.mxfp4_linear(q, s[:, :8].contiguous(), q, s)
    with pytest.raises(ValueError, match="must be"):
        w8.mxfp4_linear(q, s, *_operand(torch.Generator().manual_seed(0), 8, 96))
    with pytest.raises(TypeError, match="torch.uint8"):
        w8.mxfp4_linear(q.to(torch.int8), s, q, s)
    with pytest.raises(ValueError, match="bias"):
        w8.mxfp4_linear(q, s, q, s, torch.zeros(7, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        w8.mxfp4_linear(q, s, q, s, out=torch.zeros(8, 9, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(8, 64, device="cuda")
    with pytest.raises(w8.W8A8Error, match="SHAPE"):
        w8.mxfp4_quantize(x, ldq=48)
    with pytest.raises(ValueError, match="unit column stride"):
        w8.mxfp4_quantize(x.T)
    with pytest.raises(ValueError):
        w8.mxfp4_quantize(x.view(2, 4, 64).transpose(0, 1))
    with pytest.raises(w8.W8A8Error, match="SHAPE"):
        w8.mxfp4_dequantize(q, s, 65)
    with pytest.raises(TypeError):
        w8.mxfp4_dequantize(q, s, dtype=torch.float16)
