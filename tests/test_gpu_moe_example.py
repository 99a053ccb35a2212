"""The example that runs routing, its gradient, the Muon step and the balancing
bias together: its gradients against plain autograd, and that it learns."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer_step.py")
    spec = importlib.util.spec_from_file_location("moe_layer_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_router_gradient_is_autograds(moe):
    """d loss / d logits through the operator against autograd in 64 bits over
    the same choice: BF16 logits' gradients are rounded once, 2^-8 of a value at
    most, and 1e-5 of the largest covers FP32 sums of at most 16 terms."""
    layer = moe.Layer(seed=3)
    try:
        g = torch.Generator(device="cuda").manual_seed(5)
        logits = torch.randn(moe.TOKENS, moe.EXPERTS, generator=g, device="cuda").bfloat16()
        up = torch.randn(moe.TOKENS, moe.TOP_K, generator=g, device="cuda")
        mask = moe.batch(0)[2]
        a = logits.clone().requires_grad_()
        weights, experts = moe.Route.apply(a, layer.cfg, layer.bias, mask, layer.load)
        (weights * up).sum().backward()
        live = mask.bool()
        b = logits.double().requires_grad_()
        p = torch.sigmoid(b).gather(1, experts.clamp(min=0).long())
        w = p / (p.sum(dim=1, keepdim=True) + 1e-20)
        ((w * up.double())[live]).sum().backward()
        assert (weights[~live] == 0).all() and (experts[~live] == -1).all()
        assert ((weights.double() - w).abs()[live] <= 1e-6).all()
        assert ((a.grad.double() - b.grad).abs() <= 2.0 ** -8 * b.grad.abs() + 1e-5 * b.grad.abs().max()).all()
        assert layer.load.sum().item() == int(live.sum()) * moe.TOP_K
    finally:
        layer.close()


def test_it_learns(moe):
    """The target's variance is about 1.25 * 256 / 256; the maps are learnt to
    well under half of it."""
    losses = moe.main(60)
    assert losses[0] > 1.0
    assert sum(losses[-5:]) / 5 < 0.5 * losses[0]
