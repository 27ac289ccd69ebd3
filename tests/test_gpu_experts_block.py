"""The operators together: a block of experts routed on the GPU, forward and
backward, against the chain of the definitions in 64 bits."""
import os
import sys

import pytest
import torch

import experts_helpers as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
KINDS = ["int8", "e4m3", "mx"]


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import experts_block
    return experts_block


def _weights(kind, pair):
    """64-bit values of (codes, scales) [E, N, K]."""
    if kind == "mx":
        return ref.values(*pair)
    return pair[0].double() * pair[1].double()[:, None, None]


def _rows(w8, kind, x):
    """64-bit values of the rows as a product sees them."""
    if kind == "mx":
        return ref.values(*w8.mxfp4_quantize(x))
    q, s = w8.w8a8_quant_act_rowwise(x, w8.INT8 if kind == "int8" else w8.FP8_E4M3)
    return q.double() * s.double()[:, None]


def _each(w, rows, expert):
    """rows[i] times the weight of expert[i], transposed."""
    out = torch.zeros(rows.shape[0], w.shape[1], dtype=torch.float64, device=rows.device)
    for e in range(w.shape[0]):
        at = expert == e
        out[at] = rows[at] @ w[e].T
    return out


def _near(got, want, step, what):
    """Relative Frobenius error of a value that went through bf16 roundings and,
    where the operator's own rounded value was quantized again, another code
    for some of its elements: `step`, the sum of what each may contribute."""
    off = float((got.double() - want).norm() / want.norm())
    assert off <= step, (what, off, step)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,top", [(1, 2), (96, 2), (700, 3)])
def test_the_chain(block, kind, T, top):
    """Each product against the definition on the operator's own bf16 inputs
    (one bf16 rounding, 2^-8, and f32 sums), then the whole."""
    print(f"[experts] {kind} T={T}", flush=True)
    import w8a8_quantized_linear_quant_amd as w8
    E, width, hidden = 6, 192, 320
    b = block.Experts(kind, E, width, hidden)
    x, choice, weight = block.inputs(T, width, E, top)
    y, (routing, h, out, _) = b.forward(x, choice, weight)
    expert = choice.flatten()[routing.order]
    assert bool((expert.diff() >= 0).all()) if expert.numel() > 1 else True
    up, down = _weights(kind, b.up), _weights(kind, b.down)
    want_h = _each(up, _rows(w8, kind, x)[routing.rows.long()], expert)
    _near(h, want_h, 2.0 ** -8, "up")
    a = torch.relu(h).square()
    want_out = _each(down, _rows(w8, kind, a), expert)
    got_out = out.reshape(-1, width)[routing.order]
    _near(got_out, want_out, 2.0 ** -8, "down")
    # rows back at their tokens, weighted
    want_y = torch.zeros(T, width, dtype=torch.float64, device="cuda")
    want_y.index_add_(0, routing.rows.long(), got_out.double() * weight.flatten()[routing.order].double()[:, None])
    _near(y, want_y, 2.0 ** -8, "combined")

    dy = torch.randn(T, width, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    dx, dweight = b.backward(dy, (routing, h, out, weight))
    up_t, down_t = _weights(kind, b.up_t), _weights(kind, b.down_t)
    dout = (dy.float()[:, None, :] * weight[..., None]).bfloat16().view(-1, width)[routing.order]
    want_da = _each(down_t, _rows(w8, kind, dout), expert)
    da = b._product_dx(dout, b.down_t, routing)
    _near(da, want_da, 2.0 ** -8, "down, backward")
    dh = (da.float() * 2.0 * torch.relu(h).float()).bfloat16()
    rows_dx = _each(up_t, _rows(w8, kind, dh), expert)
    want_dx = torch.zeros(T, width, dtype=torch.float64, device="cuda").index_add_(0, routing.rows.long(), rows_dx)
    # two bf16 roundings: the rows' and the sum's; the rows of a token may cancel, so against the rows' norm
    off = float((dx.double() - want_dx).norm())
    assert off <= 2.0 ** -8 * float(rows_dx.norm()) + 2.0 ** -8 * float(want_dx.norm())
    want_dw = (out.double() * dy.double()[:, None, :]).sum(2)
    assert bool(((dweight.double() - want_dw).abs() <= width * 2.0 ** -23 * (out.double() * dy.double()[:, None, :]).abs().sum(2)).all())


def test_the_gradient_of_a_homogeneous_block(block):
    """The block is homogeneous of degree 2 in x (squared ReLU), so <dx, x> =
    2 <y, dy> for each token, and linear in the router's weights.  Four
    quantizations stand between the two sides (x and a forward, dout and dh
    backward), each moving a row by an independent error of at most half a step,
    absmax / 254, an element: uniform, it is 1 / sqrt(3) of that in the root mean
    square, and with rows of absmax below 6 root mean squares 6 / 254 / sqrt(3)
    of the row.  Four of them and the bf16 roundings stay below five."""
    T, E, width, hidden, top = 64, 4, 256, 384, 2
    b = block.Experts("int8", E, width, hidden, seed=5)
    x, choice, weight = block.inputs(T, width, E, top, seed=6)
    g = torch.Generator().manual_seed(7)
    dy = torch.randn(T, width, generator=g).bfloat16().cuda()
    y, saved = b.forward(x, choice, weight)
    dx, dweight = b.backward(dy, saved)
    rows = 2.0 * (y.double() * dy.double()).sum(1)
    lhs = (dx.double() * x.double()).sum(1)
    scale = (y.double().norm(dim=1) * dy.double().norm(dim=1)) * 2
    assert float((lhs - rows).norm() / scale.norm()) <= 5 * 6 / 254 / 3 ** 0.5
    # and the router's weights: linear
    assert torch.allclose((dweight * weight).sum(1), (y.float() * dy.float()).sum(1), rtol=0,
                          atol=float(2.0 ** -8 * 2 * (y.float() * dy.float()).abs().sum(1).max()))


@pytest.mark.parametrize("kind", KINDS)
def test_a_batch_is_its_tokens(block, kind):
    """A token's result does not depend on its neighbours, but for the order of
    sums (other tiles): bf16's rounding, and another code where a hidden value
    falls on the other side of a border: a step of the largest values."""
    b = block.Experts(kind, 5, 256, 256, seed=2)
    x, choice, weight = block.inputs(40, 256, 5, 2, seed=3)
    y, _ = b.forward(x, choice, weight)
    alone = torch.cat([b.forward(x[i:i + 1], choice[i:i + 1], weight[i:i + 1])[0] for i in range(40)])
    assert float((y.double() - alone.double()).norm() / y.double().norm()) <= 2.0 ** -7


def test_captured(block):
    """The whole forward pass, routing included, in one graph, replayed with
    other tokens and routes."""
    b = block.Experts("mx", 6, 192, 320, seed=4)
    x, choice, weight = block.inputs(50, 192, 6, 2, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward(x, choice, weight)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = b.forward(x, choice, weight)
    for seed in (9, 10, 11):
        for to, new in zip((x, choice, weight), block.inputs(50, 192, 6, 2, seed=seed)):
            to.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, b.forward(x, choice, weight)[0]), seed
