"""The operators together: the example's training step lowers its loss, its
gradients follow the chain of the operators' definitions, and a mixed batch
gives what its requests give alone."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lora_block
    return lora_block


def test_training_lowers_the_loss(block):
    print("[block] train", flush=True)
    losses, _ = block.train(steps=40)
    assert losses[-1] < 0.2 * losses[0], (losses[0], losses[-1])


def test_a_mixed_batch_is_its_requests(block):
    """The adapters, norms and codes of a row do not depend on its neighbours;
    sums may run in another order: bf16's rounding, 2^-8, and 2^-7 for values
    that fall on another side of it and of a code."""
    print("[block] serve", flush=True)
    p = block.Projection(256, 384, 16, 2, seed=3)
    p.b = torch.randn(2, 384, 16, generator=torch.Generator().manual_seed(4)).cuda() * 0.1
    batch, alone = block.serve(p)
    batch, alone = batch.float(), alone.float()
    assert bool(((batch - alone).abs() <= 2.0 ** -7 * alone.abs() + 2.0 ** -7).all())


def test_the_backward_chain(block):
    """dx of the whole block against the chain in f64 on the dequantized
    weight.  int8 gradients of the projection are off by half a step of each
    row, absmax / 254, in every element of dy: bounded in the Frobenius norm
    by that step's size against dy's, with the bf16 roundings between."""
    print("[block] chain", flush=True)
    import w8a8_quantized_linear_quant_amd as w8
    K, N, M = 192, 256, 96
    p = block.Projection(K, N, 8, 2, seed=5)
    g = torch.Generator().manual_seed(6)
    p.b = torch.randn(2, N, 8, generator=g).cuda() * 0.1
    p.gamma = 1 + 0.2 * torch.randn(K, generator=g).cuda()
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    dy = torch.randn(M, N, generator=g).bfloat16().cuda()
    plan = w8.lora_plan([40, 56], [1, 0], 2)
    _, saved = p.forward(x, plan)
    dx, _ = p.backward(dy, saved, plan)

    f = torch.float64
    w = p.wq.to(f) * p.sw.to(f)
    a, b = (t.to(f) for t in p.adapters())
    dh = dy.to(f) @ w
    for rows, l in ((slice(0, 40), 1), (slice(40, 96), 0)):
        dh[rows] += dy[rows].to(f) @ b[l] @ a[l]
    xf = x.to(f)
    mean = xf.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((xf - mean) ** 2).mean(1, keepdim=True) + 1e-5)
    h, t = (xf - mean) * rstd, dh * p.gamma.to(f)
    ref = rstd * (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True))
    step = dy.to(f).abs().amax(1, keepdim=True) / 127
    quantization = float((step / 12 ** 0.5 * N ** 0.5).norm() / dy.to(f).norm())
    off = float((dx.to(f) - ref).norm() / ref.norm())
    assert off <= 2 * quantization + 3 * 2.0 ** -9, (off, quantization)
