"""What include/w8a8_experts.h says of the sums: e4m3 products are cut off in
groups of 8 codes, int8 sums wrap, sums of 4-bit blocks are f32."""
import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as w8
    yield w8
    torch.cuda.empty_cache()


def _device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def _e4m3(g, spread, rows, K):
    """Normal codes, or codes whose exponents are spread evenly over the type,
    with every second group of 8 cancelling but for its last two."""
    if not spread:
        return torch.randn((rows, K), generator=g, device="cuda").mul(30).to(torch.float8_e4m3fn)
    x = torch.pow(2.0, torch.rand((rows, K), generator=g, device="cuda") * 14 - 6)
    x = torch.where(torch.rand((rows, K), generator=g, device="cuda") < 0.5, x, -x).view(rows, K // 8, 8)
    x[:, ::2, 3:6] = -x[:, ::2, 0:3]
    return x.view(rows, K).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("kind,kernel,M,E,N,K", [k for k in ref.KERNELS if k[0] == "e4m3"])
def test_e4m3_sums_lose_what_the_header_says(w8, kind, kernel, M, E, N, K, spread):
    """Each of a group's 8 products is off by less than 2^-13 of the greatest of
    the 8; K / 8 sums and the rest are f32: K + 4 roundings of 2^-23 of the sum
    of |terms|, as in assert_close; then half a step of bf16.  With a bias: on
    normal codes the bound leaves out a missing one."""
    print(f"[numerics] e4m3 kernel {kernel}: {M} {E} {N} {K}", flush=True)
    assert w8.probe_grouped_kernel(kind, M, N, K, E) == kernel
    g = torch.Generator(device="cuda").manual_seed(kernel)
    offsets = [0]
    for n in ref.uneven(M, E):
        offsets.append(offsets[-1] + n)
    xq = _e4m3(g, spread, M, K)
    wq = torch.stack([_e4m3(g, False, N, K) for _ in range(E)])
    if spread:                                  # weights of one size: the products cancel as the codes do
        wq = torch.where(wq.float() < 0, -16.0, 16.0).view(E, N, K // 8, 8)[..., :1].expand(E, N, K // 8, 8)
        wq = wq.reshape(E, N, K).to(torch.float8_e4m3fn)
    bias = torch.randn((E, N), generator=g, device="cuda").mul(3000).bfloat16()
    y = w8.w8a8_linear_grouped(xq, torch.ones(M, device="cuda"), wq, torch.ones(E, device="cuda"), _device(offsets), bias=bias)
    missed = 0
    for e, a, b in ref.groups_of(offsets, M):
        rows = sorted({a, (a + b) // 2, b - 1}) if b > a else []
        for m in rows:
            x, w = xq[m].double(), wq[e].double()
            terms = x * w                                                   # [N, K]
            want, mass = terms.sum(1) + bias[e].double(), terms.abs().sum(1) + bias[e].double().abs()
            low = terms.abs().view(N, K // 8, 8).amax(2).sum(1) * 8 * 2.0 ** -13 + (K + 4) * 2.0 ** -23 * mass
            bound = low + ref.BF16_HALF_STEP * (want.abs() + low)
            off = (y[m].double() - want).abs()
            assert bool((off <= bound).all()), (m, float((off - bound).max()))
            missed += int(((y[m].double() - (want - bias[e].double())).abs() > bound).sum())
    assert spread or missed > N / 4, missed


INT8 = [(0, 5, 40, 2), (2, 300, 300, 2), (3, 300, 2000, 1), (4, 1000, 2000, 2), (6, 4096, 4096, 1)]


@pytest.mark.parametrize("K", [(1 << 17) - 16, 1 << 17, (1 << 18) + 80])
@pytest.mark.parametrize("kernel,M,N,E", INT8)
def test_int8_sums_wrap(w8, kernel, M, N, E, K):
    """Codes of -128 and -128 but for a few: sums of about K * 2^14, at most 2^31
    - 1 up to K = 2^17 - 1 and modulo 2^32 beyond; one rounding to f32 and one to
    bf16."""
    print(f"[numerics] int8 kernel {kernel}: {M} {N} {K}", flush=True)
    assert w8.probe_grouped_kernel("int8", M, N, K, E) == kernel
    xq, wq = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((E, N, K), -128, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(K)
    more = torch.randint(0, 256, (M,), generator=g, device="cuda")           # added to a row's first code
    less = torch.randint(0, 256, (E, N), generator=g, device="cuda")         # to a weight row's last
    more[0], less[:, 0] = 0, 0
    xq[:, 0] += more.to(torch.uint8).view(torch.int8)
    wq[..., K - 1] += less.to(torch.uint8).view(torch.int8)
    offsets = [0] + [M // 3] * (E - 1) + [M]
    y = w8.w8a8_linear_grouped(xq, torch.full((M,), 2.0 ** -8, device="cuda"), wq, torch.ones(E, device="cuda"), _device(offsets))
    group = torch.tensor([e for e, a, b in ref.groups_of(offsets, M) for _ in range(a, b)], device="cuda")
    sums = (K - 2) * 128 * 128 - 128 * xq[:, :1].long() - 128 * wq[..., K - 1].long()[group]
    wrapped = (sums + 2 ** 31) % 2 ** 32 - 2 ** 31
    assert bool((wrapped == sums).all()) == (K < 1 << 17)
    assert torch.equal(y, (wrapped.float() * 2.0 ** -8).bfloat16())


@pytest.mark.parametrize("kind,kernel,M,E,N,K", [k for k in ref.KERNELS if k[0] == "mx"])
def test_blocks_far_apart_add_up_in_f32(w8, kind, kernel, M, E, N, K):
    """Two terms of 2^20 cancel in a block whose scale is 2^18 times the others',
    a term of 1 stands elsewhere: no sum needs more than 24 bits, so the 1 is
    what is left, wherever it stands."""
    print(f"[numerics] mx kernel {kernel}: {M} {E} {N} {K}", flush=True)
    assert w8.probe_grouped_kernel(kind, M, N, K, E) == kernel
    four, minus, one = 6, 14, 2                                             # codes of 4, -4, 1
    x = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    m = torch.arange(M, device="cuda")
    big = m * 7 % (K // 32)                                                 # the block with the two
    small = (m * 37 + 5) % K
    small = torch.where(small // 32 == big, (small + 32) % K, small)
    x[m, big * 32 + m % 16], x[m, big * 32 + 16 + m % 16], x[m, small] = four, minus, one
    xs = torch.full((M, ref.stride_of(K)), 127, dtype=torch.uint8, device="cuda")
    xs[m, big] = 127 + 18
    # weights of 4 at a scale of 1/4
    wq = torch.full((E, N, K // 2), four * 17, dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N, ref.stride_of(K)), 127 - 2, dtype=torch.uint8, device="cuda")
    offsets = [0]
    for n in ref.uneven(M, E):
        offsets.append(offsets[-1] + n)
    y = w8.mxfp4_linear_grouped(ref.pack(x), xs, wq, ws, _device(offsets))
    assert bool((y == 1).all())
