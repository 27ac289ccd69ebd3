"""Calls of the products of groups that the documentation allows or refuses and
that no product's own test makes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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
