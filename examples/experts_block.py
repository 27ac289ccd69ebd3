"""A block of experts with frozen 8-bit or 4-bit weights: served and differentiated.

    python examples/experts_block.py

Each token goes to `top` of E experts; an expert is two projections with a
squared ReLU between.  Tokens are quantized once and gathered by the first product; the second
product's rows are added up per token with the router's weights.  The backward
pass gives the gradient of the tokens and of the router's weights through the
frozen experts.  Routing stays on the GPU: nothing waits for it.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_quantized_linear_quant_amd as w8  # noqa: E402


class Routing:
    """Rows of the experts' products: sorted by expert, tokens in order."""

    def __init__(self, choice, experts):
        flat = choice.flatten()
        self.order = torch.sort(flat, stable=True).indices            # slot of each row
        self.slot_row = torch.empty_like(self.order)                  # row of each slot
        self.slot_row[self.order] = torch.arange(flat.numel(), device=flat.device)
        self.rows = (self.order // choice.shape[1]).int()             # token of each row
        edges = torch.arange(experts + 1, device=flat.device)
        self.offsets = torch.searchsorted(flat[self.order], edges).int()
        self.shape = choice.shape

    def to_tokens(self, rows):
        """[T, top, width] of the rows [T * top, width]."""
        return rows[self.slot_row].view(*self.shape, rows.shape[1])


class Experts:
    """kind: "int8", "e4m3" or "mx" (the 4-bit format)."""

    def __init__(self, kind, experts, width, hidden, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.experts = kind, experts
        up = (torch.randn((experts, hidden, width), generator=g, device="cuda") * width ** -0.5).bfloat16()
        down = (torch.randn((experts, width, hidden), generator=g, device="cuda") * hidden ** -0.5).bfloat16()
        self.up, self.up_t = self._weights(up)
        self.down, self.down_t = self._weights(down)

    def _weights(self, w):
        """(codes and scales, those of the transposes)."""
        if self.kind == "mx":
            return w8.mxfp4_quantize(w), w8.mxfp4_quantize_transposed(w)
        wq, wq_t, scale = w8.w8a8_quant_weight_grouped(w, self._qtype(), transposed=True)
        return (wq, scale), (wq_t, scale)

    def _qtype(self):
        return w8.INT8 if self.kind == "int8" else w8.FP8_E4M3

    def _product(self, x, weights, routing, rows=None):
        if self.kind == "mx":
            return w8.mxfp4_linear_grouped(*w8.mxfp4_quantize(x), *weights, routing.offsets, rows=rows)
        return w8.w8a8_linear_grouped(*w8.w8a8_quant_act_rowwise(x, self._qtype()), *weights, routing.offsets, rows=rows)

    def _product_dx(self, dy, weights_t, routing):
        if self.kind == "mx":
            return w8.mxfp4_linear_grouped_backward_dx(*w8.mxfp4_quantize(dy), *weights_t, routing.offsets)
        return w8.w8a8_linear_grouped_backward_dx(*w8.w8a8_quant_act_rowwise(dy, self._qtype()), *weights_t,
                                                  routing.offsets)

    def forward(self, x, choice, weight):
        """x bf16 [T, width]; choice int64 [T, top]; weight f32 [T, top].  (y bf16, what the backward pass needs.)"""
        routing = Routing(choice, self.experts)
        h = self._product(x, self.up, routing, rows=routing.rows)
        a = torch.relu(h).square()
        out = routing.to_tokens(self._product(a, self.down, routing))
        y = (out.float() * weight[..., None]).sum(1).bfloat16()
        return y, (routing, h, out, weight)

    def backward(self, dy, saved):
        """(dx bf16 [T, width], dweight f32 [T, top])."""
        routing, h, out, weight = saved
        dweight = (out.float() * dy.float()[:, None, :]).sum(2)
        dout = (dy.float()[:, None, :] * weight[..., None]).bfloat16().view(-1, dy.shape[1])[routing.order]
        da = self._product_dx(dout, self.down_t, routing)
        dh = (da.float() * 2.0 * torch.relu(h).float()).bfloat16()
        dx = self._product_dx(dh, self.up_t, routing)
        return routing.to_tokens(dx).float().sum(1).bfloat16(), dweight


def inputs(T, width, experts, top, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, width), generator=g, device="cuda").bfloat16()
    score = torch.randn((T, experts), generator=g, device="cuda")
    weight, choice = torch.softmax(score, 1).topk(top, 1)
    return x, choice, weight


if __name__ == "__main__":
    for kind in ("int8", "e4m3", "mx"):
        block = Experts(kind, 8, 512, 1024)
        x, choice, weight = inputs(256, 512, 8, 2)
        y, saved = block.forward(x, choice, weight)
        dx, dweight = block.backward(torch.ones_like(y), saved)
        one, _ = block.forward(x[:1], choice[:1], weight[:1])
        worst = float((one[0].float() - y[0].float()).abs().max() / y[0].float().abs().max())
        print(f"{kind}: |y| {float(y.float().norm()):.3f} |dx| {float(dx.float().norm()):.3f} "
              f"|dweight| {float(dweight.norm()):.3f}; a token alone within {worst:.1e} of the batch")
