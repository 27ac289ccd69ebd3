"""Calls of the products of groups that the documentation allows or refuses and
that no product's own test makes."""
import os
import sys

import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as w8
    return w8


@pytest.mark.parametrize("qtype", [0, 1])
def test_weights_that_would_start_off_alignment(w8, qtype):
    """Each weight has to start on a 16-byte boundary, its codes too: refused
    before the first one is quantized; a single weight has no such neighbour."""
    w = torch.randn(2, 5, 24, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    quantized = []
    single, w8.w8a8_quant_weight_tensorwise = w8.w8a8_quant_weight_tensorwise, lambda *a, **k: quantized.append(a)
    try:
        with pytest.raises(ValueError, match="N \\* K"):
            w8.w8a8_quant_weight_grouped(w, qtype)
    finally:
        w8.w8a8_quant_weight_tensorwise = single
    assert not quantized
    wq, _, s = w8.w8a8_quant_weight_grouped(w[:1], qtype)
    a, _, b = single(w[0], qtype)
    assert torch.equal(wq[0].view(torch.uint8), a.view(torch.uint8)) and torch.equal(s, b)
    wq, wt, s = w8.w8a8_quant_weight_grouped(w[:0], qtype, transposed=True)
    assert wq.shape == (0, 5, 24) and wt.shape == (0, 24, 5) and s.shape == (0,)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_the_gradient_beside_scales_of_channels(w8, kind):
    """dX[p] = sum_n dY[p, n] s[g, n] wq[g, n]: the scales go into dY before it is
    quantized, the product takes scales of 1."""
    lengths, N, K = [40, 0, 33, 7], 96, 160
    M, E = sum(lengths), len(lengths)
    group = torch.tensor([g for g, n in enumerate(lengths) for _ in range(n)], device="cuda")
    off = torch.tensor([0, 40, 40, 73, 80], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    qt, top = (w8.INT8, 127.0) if kind == "int8" else (w8.FP8_E4M3, 448.0)
    w = torch.randn(E, N, K, generator=g).cuda() * torch.logspace(-1, 1, N, device="cuda")[None, :, None]
    s = w.abs().amax(2) / top
    wq = w / s[..., None]
    wq = wq.round().to(torch.int8) if kind == "int8" else wq.to(torch.float8_e4m3fn)
    dy = torch.randn(M, N, generator=g).bfloat16().cuda()
    folded = (dy.float() * s[group]).bfloat16()
    dq, ds = w8.w8a8_quant_act_rowwise(folded, qt)
    wt = wq.view(torch.uint8).transpose(1, 2).contiguous().view(wq.dtype)
    dx = w8.w8a8_linear_grouped_backward_dx(dq, ds, wt, torch.ones(E, device="cuda"), off)
    want = torch.zeros(M, K, dtype=torch.float64, device="cuda")
    room = torch.zeros_like(want)
    # folded: a bf16 rounding; dq: half a step of the row's codes (int8: absmax / 254, e4m3: 2^-4 of the value and 2^-10
    # of the scale, half the smallest code); an e4m3 term is off by 2^-13 of the greatest of its eight besides
    for e in range(E):
        at = group == e
        exact = dy[at].double() * s[e].double()
        absmax = folded[at].double().abs().amax(1, keepdim=True)
        off_d = 2.0 ** -8 * exact.abs() + (absmax / 254 if kind == "int8" else
                                           2.0 ** -4 * folded[at].double().abs() + 2.0 ** -10 * absmax / 448) * 1.001
        want[at] = exact @ wq[e].double()
        mass = (exact.abs() + off_d) @ wq[e].double().abs()
        room[at] = off_d @ wq[e].double().abs() + mass * ((N + 4) * 2.0 ** -23 + (8 * 2.0 ** -13 if kind == "e4m3" else 0.0))
    assert bool(((dx.double() - want).abs() <= room + ref.BF16_HALF_STEP * (want.abs() + room)).all())
    with pytest.raises(ValueError, match="multiply dY"):
        w8.w8a8_linear_grouped_backward_dx(dq, ds, wt, s, off)


@pytest.mark.parametrize("kind", ["int8", "e4m3", "mx"])
def test_the_example_without_tokens(w8, kind):
    import experts_block
    b = experts_block.Experts(kind, 3, 64, 96)
    x, choice, weight = experts_block.inputs(0, 64, 3, 2)
    y, saved = b.forward(x, choice, weight)
    dx, dweight = b.backward(torch.zeros_like(y), saved)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and dweight.shape == (0, 2)
