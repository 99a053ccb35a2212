"""Training steps of one mixture-of-experts layer with the library's routing and
Muon operators, as a training loop calls them.

    python examples/moe_layer_step.py [steps]

Each step: two gradient replicas (micro-batches with padded tokens) run
norm -> router -> experts -> loss; slide_route_experts picks the experts and
their weights, slide_route_experts_backward takes the loss's gradient with
respect to those weights back to the router's logits; then one
slide_layer_muon_step updates the router and every expert's matrices by Muon and
the norm by AdamW, and slide_route_bias_step moves the balancing bias by the
load that the step's routing counted.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_adam_grad_gb300 as S  # noqa: E402

HIDDEN, INNER, EXPERTS, TOP_K, GROUPS, TOP_GROUPS = 256, 384, 16, 4, 4, 2
TOKENS, PADDED, REPLICAS = 1024, 57, 2


class Route(torch.autograd.Function):
    """weights [tokens, top_k] and experts of each token; counts the load."""

    @staticmethod
    def forward(ctx, logits, cfg, bias, mask, load):
        tokens = logits.shape[0]
        logits = logits.detach()
        weights = torch.empty(tokens, cfg.top_k, device="cuda")
        experts = torch.empty(tokens, cfg.top_k, dtype=torch.int32, device="cuda")
        S.slide_route_experts(tokens, logits, weights, experts, cfg, bias=bias, token_mask=mask, load=load,
                              logits_type=S.SLIDE_TYPE_BF16, stream=torch.cuda.current_stream())
        ctx.cfg, ctx.mask = cfg, mask
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    def backward(ctx, d_weights, _):
        logits, experts = ctx.saved_tensors
        d_logits = torch.empty_like(logits)
        S.slide_route_experts_backward(logits.shape[0], logits, experts, d_weights.contiguous(), d_logits, ctx.cfg,
                                       token_mask=ctx.mask, logits_type=S.SLIDE_TYPE_BF16,
                                       stream=torch.cuda.current_stream())
        return d_logits, None, None, None, None


class Layer:
    """The layer's parameters, flat in one state: router, experts' up and down matrices, norm."""

    def __init__(self, seed=0):
        shapes = {"router": (1, EXPERTS, HIDDEN), "up": (EXPERTS, INNER, HIDDEN), "down": (EXPERTS, HIDDEN, INNER)}
        self.blocks, self.parts, at = [], {}, 0
        for name, shape in shapes.items():
            self.blocks.append((at, *shape))
            self.parts[name] = (at, shape)
            at += int(np.prod(shape))
        self.parts["norm"] = (at, (HIDDEN,))
        self.numel = at + HIDDEN
        rng = np.random.default_rng(seed)
        theta = np.ones(self.numel, np.float32)
        for off, batch, rows, cols in self.blocks:
            n = batch * rows * cols
            theta[off:off + n] = rng.standard_normal(n, np.float32) / np.sqrt(cols)
        self.state = S.slide_state_create([self.numel], REPLICAS)
        zero = np.zeros(self.numel, np.float32)
        S.slide_layer_set(self.state, 0, master=theta, m=zero, v=zero)
        self.bf16 = torch.from_numpy(theta).cuda().bfloat16()   # what the forward pass reads
        self.ws = torch.empty(max(S.slide_ortho_workspace(*b[1:]) for b in self.blocks), dtype=torch.uint8, device="cuda")
        self.cfg = S.route_config(EXPERTS, TOP_K, n_groups=GROUPS, top_groups=TOP_GROUPS)
        self.bias = torch.zeros(EXPERTS, device="cuda")
        self.load = torch.zeros(EXPERTS, dtype=torch.int64, device="cuda")
        self.muon = S.muon_hparams(lr=0.02, weight_decay=0.01)
        self.adam = S.hparams(lr=1e-3)

    def close(self):
        S.slide_state_destroy(self.state)

    def weights(self):
        leaf = self.bf16.detach().requires_grad_()
        return leaf, {k: leaf[off:off + int(np.prod(shape))].view(shape) for k, (off, shape) in self.parts.items()}

    def forward(self, x, w, mask=None, load=None):
        y = x * torch.rsqrt(x.float().square().mean(dim=1, keepdim=True) + 1e-6).bfloat16() * w["norm"]
        weights, experts = Route.apply(y @ w["router"][0].T, self.cfg, self.bias, mask, load)
        out = torch.zeros(x.shape, device="cuda")
        for e in range(EXPERTS):
            token, slot = torch.nonzero(experts == e, as_tuple=True)
            part = torch.nn.functional.silu(y[token] @ w["up"][e].T) @ w["down"][e].T
            out = out.index_add(0, token, part.float() * weights[token, slot, None])
        return out

    def step(self, batches):
        """One step over a micro-batch (x, target, mask) for each replica; the mean loss."""
        grads, loss = [], 0.0
        for x, target, mask in batches:
            leaf, w = self.weights()
            out = self.forward(x, w, mask, self.load)
            each = ((out - target).square().mean(dim=1) * mask).sum() / mask.sum()
            each.backward()
            grads.append(leaf.grad)
            loss += each.item() / len(batches)
        stream = torch.cuda.current_stream()
        S.slide_layer_muon_step(self.state, 0, self.blocks, grads, self.muon, self.adam, self.ws, stream=stream,
                                bf16_out=self.bf16)
        S.slide_route_bias_step(EXPERTS, self.load, self.bias, 1e-3, stream=stream)
        if S.slide_ortho_status(self.ws, stream=stream) != S.SLIDE_OK:
            raise RuntimeError("a wait inside the optimizer's products ran out")
        return loss


def batch(seed):
    """Tokens around a few centres, each with a map of its own to the target; the last ones are padding."""
    g = torch.Generator(device="cuda").manual_seed(11)
    centre = torch.randn(8, HIDDEN, generator=g, device="cuda")
    maps = torch.randn(8, HIDDEN, HIDDEN, generator=g, device="cuda") / HIDDEN ** 0.5
    g.manual_seed(1000 + seed)
    kind = torch.randint(0, 8, (TOKENS,), generator=g, device="cuda")
    x = centre[kind] + 0.5 * torch.randn(TOKENS, HIDDEN, generator=g, device="cuda")
    target = torch.bmm(maps[kind], x[:, :, None])[:, :, 0]
    mask = torch.ones(TOKENS, dtype=torch.uint8, device="cuda")
    mask[TOKENS - PADDED:] = 0
    return x.bfloat16(), target, mask


def main(steps=60):
    layer = Layer()
    try:
        losses = []
        for t in range(steps):
            losses.append(layer.step([batch(REPLICAS * t + r) for r in range(REPLICAS)]))
            if t % 10 == 0 or t + 1 == steps:
                print("step %3d  loss %.4f" % (t, losses[-1]))
        with torch.no_grad():  # serving: one token
            x, target, _ = batch(10 ** 6)
            one = layer.forward(x[:1], layer.weights()[1])
        print("one token's squared error %.4f" % (one - target[:1]).square().mean().item())
        return losses
    finally:
        layer.close()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
