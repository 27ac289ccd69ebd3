"""The 4-bit format and the products of groups where offsets pass 32 bits, and
over very many tiles."""
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
    yield w8
    torch.cuda.empty_cache()


def _codes(kind, shape, seed):
    """Random codes on the GPU: (codes, scales, the 64-bit values of a slice)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    K = shape[-1]
    if kind == "mx":
        q = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, dtype=torch.uint8, device="cuda")
        s = torch.full((*shape[:-1], ref.stride_of(K)), 127, dtype=torch.uint8, device="cuda")
        return q, s, lambda *at: ref.values(q[at], s[at])
    if kind == "int8":
        q = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    else:
        # every finite code of magnitude 0 .. 15.5
        q = torch.randint(0, 88, shape, generator=g, dtype=torch.uint8, device="cuda")
        q = (q | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8, device="cuda") << 7)).view(torch.float8_e4m3fn)
    return q, torch.ones(shape[0], device="cuda"), lambda *at: q.view(torch.uint8)[at].view(q.dtype).double()


def _product(w8, kind):
    return w8.mxfp4_linear_grouped if kind == "mx" else w8.w8a8_linear_grouped


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M", [3, 40, 2500])
def test_weights_beyond_32_bits(w8, kind, M):
    """Three weights of 1.5 GB each: the last one's last rows lie past 2^32 bytes."""
    E, N, K = 3, 45032, 32800 * (2 if kind == "mx" else 1)
    wq, ws, wv = _codes(kind, (E, N, K), 1)
    assert wq.numel() > 2 ** 32
    xq, xs, xv = _codes(kind, (M, K), 2)
    off = torch.tensor([0, 1, 1, M], dtype=torch.int32, device="cuda")
    y = _product(w8, kind)(xq, xs, wq, ws, off)
    some = [0, 2, M // 2, M - 1] if M > 3 else [0, 1, 2]
    for e, n in ((0, 0), (2, N - 70)):
        w = wv(e, slice(n, n + 70))
        at = [m for m in some if (m == 0) == (e == 0)]
        x = xv(torch.tensor(at, device="cuda"))
        peak = ref.peaks(x, w[None], [0, len(at)], len(at)) if kind == "e4m3" else None
        ref.assert_close(y[at, n:n + 70], x @ w.T, x.abs() @ w.abs().T, K, exact_sums=kind == "int8", peak=peak)


@pytest.mark.parametrize("kind", TYPES)
def test_an_output_beyond_32_bits(w8, kind):
    M, N, K = 270001, 8200, 32
    xq, xs, xv = _codes(kind, (M, K), 3)
    wq, ws, wv = _codes(kind, (1, N, K), 4)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    y = _product(w8, kind)(xq, xs, wq, ws, off)
    assert y.numel() > 2 ** 31
    w = wv(0)
    for m in (0, 131072, 262143, M - 60):
        x = xv(slice(m, m + 60))
        peak = ref.peaks(x, w[None], [0, 60], 60) if kind == "e4m3" else None
        ref.assert_close(y[m:m + 60], x @ w.T, x.abs() @ w.abs().T, K, exact_sums=kind == "int8", peak=peak)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N", [(5, 40), (600, 40), (600, 4000), (7000, 4000)])
def test_gathered_rows_of_the_largest_x(w8, kind, M, N):
    """2^31 bytes of codes, and indices on both sides of its end."""
    X, K = 1 << 17, (1 << 14) * (2 if kind == "mx" else 1)
    xq, xs, xv = _codes(kind, (X, K), 5)
    wq, ws, wv = _codes(kind, (1, N, K), 6)
    few = [X - 1, 0, X, -1, X // 2]
    rows = torch.tensor((few * (M // 5 + 1))[:M], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    y = _product(w8, kind)(xq, xs, wq, ws, off, rows=rows)
    x, w = xv(torch.tensor([X - 1, 0, X // 2], device="cuda")), wv(0)
    peak = ref.peaks(x, w[None], [0, 3], 3) if kind == "e4m3" else None
    ref.assert_close(y[[0, 1, 4]], x @ w.T, x.abs() @ w.abs().T, K, exact_sums=kind == "int8", peak=peak)
    assert bool((y[2:4] == 0).all())
    assert torch.equal(y, y[torch.arange(M, device="cuda") % 5])


@pytest.mark.parametrize("kind", TYPES)
def test_a_million_tiles(w8, kind):
    """4096 groups of a row and 32776 columns."""
    E, N, K = 4096, 32776, 32
    xq, xs, xv = _codes(kind, (E, K), 7)
    wq, ws, wv = _codes(kind, (E, N, K), 8)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    y = _product(w8, kind)(xq, xs, wq, ws, off)
    for e in (0, 1, 2047, 4095):
        x, w = xv(slice(e, e + 1)), wv(e)
        peak = ref.peaks(x, w[None], [0, 1], 1) if kind == "e4m3" else None
        ref.assert_close(y[e:e + 1], x @ w.T, x.abs() @ w.abs().T, K, exact_sums=kind == "int8", peak=peak)


def test_quantizers_beyond_32_bits(w8):
    M, K = (1 << 20) + 40, 2080
    x = torch.randn(M, K, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    q, s = w8.mxfp4_quantize(x)
    y = w8.mxfp4_dequantize(q, s)
    for m in (0, M // 2, M - 64):
        a, b = w8.mxfp4_quantize(x[m:m + 64].clone())
        assert torch.equal(a, q[m:m + 64]) and torch.equal(b, s[m:m + 64])
        assert torch.equal(w8.mxfp4_dequantize(a, b), y[m:m + 64])


def test_the_transposed_quantizer_beyond_32_bits(w8):
    N, K = (1 << 17) + 36, 16400
    w = torch.randn(N, K, dtype=torch.bfloat16, device="cuda")
    assert w.numel() > 2 ** 31
    q, s = w8.mxfp4_quantize_transposed(w)
    for k in (0, K // 2, K - 64):
        a, b = w8.mxfp4_quantize(w[:, k:k + 64].T.contiguous())
        assert torch.equal(a, q[k:k + 64]) and torch.equal(b, s[k:k + 64])
