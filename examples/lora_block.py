"""A quantized projection with its norm and low-rank adapters: training and serving.

    python examples/lora_block.py

y = W8A8(LayerNorm(x)) + adapter(LayerNorm(x)), the projection's int8 weight
frozen.  Training: two adapters and the norm's weight and bias learn to
reproduce a teacher's outputs, one adapter for each half of the batch.
Serving: a batch of requests of uneven lengths, each with one of the adapters
or none, through the same projection.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_quantized_linear_quant_amd as w8  # noqa: E402


class Projection:
    """LayerNorm -> frozen int8 linear, with a pool of adapters beside it."""

    def __init__(self, K, N, R, adapters, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
        self.wq, self.wq_t, self.sw = w8.w8a8_quant_weight_tensorwise(w, transposed=True)
        self.gamma, self.beta = torch.ones(K, device="cuda"), torch.zeros(K, device="cuda")
        self.a = torch.randn((adapters, R, K), generator=g, device="cuda") * K ** -0.5
        self.b = torch.zeros((adapters, N, R), device="cuda")
        self.scale = torch.ones(adapters, device="cuda")

    def adapters(self):
        return self.a.bfloat16(), self.b.bfloat16()

    def forward(self, x, plan):
        """(y, what the backward pass needs)."""
        a, b = self.adapters()
        h, mean, rstd = w8.layer_norm_forward(x, self.gamma, self.beta)
        hq, sh = w8.w8a8_quant_act_rowwise(h)
        y = w8.w8a8_linear(hq, sh, self.wq, self.sw)
        y, u = w8.lora_forward(h, a, b, plan, scale=self.scale, base=y, out=y)
        return y, (x, h, mean, rstd, u, a, b)

    def backward(self, dy, saved, plan):
        """(dx, {parameter: gradient})."""
        x, h, mean, rstd, u, a, b = saved
        dyq, sdy = w8.w8a8_quant_act_rowwise(dy)
        dh = w8.w8a8_linear_backward_dx(dyq, sdy, self.wq_t, self.sw)
        dh, da, db = w8.lora_backward(dy, h, u, a, b, plan, scale=self.scale, base=dh, out=dh)
        dx, dgamma, dbeta = w8.layer_norm_backward(dh, x, mean, rstd, self.gamma)
        return dx, dict(a=da, b=db, gamma=dgamma, beta=dbeta)

    def serve(self, x, plan):
        """Without gradients: the norm goes straight to codes, and its bf16
        values are computed for the adapters alone."""
        a, b = self.adapters()
        hq, sh = w8.w8a8_quant_act_rowwise_layer_norm(x, self.gamma, self.beta)
        h, _, _ = w8.layer_norm_forward(x, self.gamma, self.beta)
        y = w8.w8a8_linear(hq, sh, self.wq, self.sw)
        return w8.lora_forward(h, a, b, plan, scale=self.scale, base=y, out=y, save_u=False)[0]


def train(steps=60, M=1024, K=512, N=768, R=16, seed=1):
    """The loss of each step and the trained projection."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher, student = Projection(K, N, R, 2), Projection(K, N, R, 2)
    teacher.b = torch.randn((2, N, R), generator=g, device="cuda") * 0.3
    teacher.gamma += torch.randn(K, generator=g, device="cuda") * 0.1
    plan = w8.lora_plan([M // 2, M - M // 2], [0, 1], 2)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    target = teacher.forward(x, plan)[0].float()
    moments = {}
    losses = []
    for step in range(1, steps + 1):
        y, saved = student.forward(x, plan)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        dy = (2.0 / M * diff).bfloat16()
        _, grads = student.backward(dy, saved, plan)
        for name, grad in grads.items():        # Adam
            m, v = moments.setdefault(name, (torch.zeros_like(grad), torch.zeros_like(grad)))
            m.lerp_(grad, 0.1)
            v.lerp_(grad * grad, 0.01)
            update = (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
            getattr(student, name).sub_(update, alpha=0.01)
    return losses, student


def serve(projection, lengths=(1, 37, 1, 130, 5), adapters=(0, 1, -1, 1, 0), seed=2):
    """A mixed batch in one call, and the same requests one by one."""
    K = projection.gamma.numel()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((sum(lengths), K), generator=g, device="cuda").bfloat16()
    batch = projection.serve(x, w8.lora_plan(lengths, adapters, 2))
    alone, row = [], 0
    for n, l in zip(lengths, adapters):
        alone.append(projection.serve(x[row:row + n], w8.lora_plan([n], [l], 2)))
        row += n
    return batch, torch.cat(alone)


if __name__ == "__main__":
    losses, projection = train()
    print("loss " + " ".join(f"{v:.4f}" for v in losses[::10] + losses[-1:]))
    batch, alone = serve(projection)
    worst = float((batch.float() - alone.float()).abs().max() / alone.float().abs().max())
    print(f"{batch.shape[0]} rows of 5 requests in one batch: within {worst:.1e} of one by one")
