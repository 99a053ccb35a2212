"""slide_norm at its limits, against the formulas.

u = 2^-24 is half a step of FP32.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


def config(S, layer, dt, eps=1e-5):
    t = S.SLIDE_TYPE_FP32 if dt == torch.float32 else S.SLIDE_TYPE_BF16
    return S.norm_config(S.SLIDE_NORM_LAYER if layer else S.SLIDE_NORM_RMS, eps, t, t)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [3, 40, 96, 777, 1000, 1601, 2560, 4099, 16383])
def test_constant_rows(S, cols, kind):
    """Rows of one value whose sums FP32 holds exactly (in 24 bits; 16383 times 30000 = 1875 * 2^4 takes 25):
    the mean is that value, so nothing is left but the bias, however large the value and whatever the width."""
    dt = TYPES[kind]
    values = torch.tensor([1000.0, 3.0, -30000.0, 100.0, 2.0 ** -7, 0.0, -255.0, 1.5 * 2 ** 20], device="cuda")
    assert torch.equal(values.to(dt).float(), values) or dt == torch.bfloat16
    values = values.to(dt)
    x = values[:, None].repeat(1, cols)
    out, mean, rstd = torch.empty_like(x), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    bias = torch.arange(cols, device="cuda").to(dt)
    S.slide_norm(8, cols, x, torch.ones_like(bias), out, config(S, True, dt), bias=bias, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    total = values.double() * cols
    held = total.float().double() == total
    assert held.sum() >= 7
    assert torch.equal(mean[held], values.float()[held])
    assert torch.equal(out[held], bias[None].expand_as(out)[held])
    assert ((rstd - 1e-5 ** -0.5).abs() <= 8 * U * 1e-5 ** -0.5)[held].all()
