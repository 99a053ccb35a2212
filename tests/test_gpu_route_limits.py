"""The routing weights' gradient where it is small beside its terms: against the
formula in 64 bits, to a few roundings of the terms.

With w_i the weights, p the scores (normalised over the chosen ones where they
are renormalised) and g the upstream values, the gradient of expert i is p_i
times sum_j p_j (g_i - g_j) (times 1 - p_i of a sigmoid over its sum, and with
the experts that were not chosen as g_j = 0 where nothing is renormalised).  Each
term is a product of scores of at most 6 ulp each, a difference of one rounding,
and sums of at most 33 terms; the argument of an exponential is a difference of
logits, whose rounding is 2^-24 of it and enters as a factor.  So a value is off
by 2^-24 (48 + 2 D) of the sum of its terms' sizes, with D the row's range of
logits; a score that is itself of the size of an FP32 denormal by 2^-126.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_route import Cfg, S  # noqa: E402, F401


def terms64(x, e, g, c):
    """Gradient and the sum of its terms' sizes, of chosen experts e (all valid)."""
    x, g, T = x.double(), g.double() * c.scale, x.shape[0]
    p = torch.sigmoid(x) if c.score == "sigmoid" else torch.softmax(x, 1)
    up = torch.zeros_like(x).scatter_(1, e, g)
    if c.score == "sigmoid":
        pc = p.gather(1, e)
        total = pc.sum(1, keepdim=True) + 1e-20
        diff = g[:, :, None] - g[:, None, :]
        own = g * 1e-20
        slope = pc * torch.sigmoid(-x.gather(1, e)) / total ** 2
        want = torch.zeros_like(x).scatter_(1, e, slope * ((diff * pc[:, None, :]).sum(2) + own))
        size = torch.zeros_like(x).scatter_(1, e, slope * ((diff.abs() * pc[:, None, :]).sum(2) + own.abs()))
        return want, size
    if c.renorm:
        only = torch.full_like(x, -float("inf")).scatter_(1, e, x.gather(1, e))
        p = torch.softmax(only, 1)
    want, size = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):  # all experts: up is 0 where an expert is not chosen
        d = up[t, :, None] - up[t, None, :]
        want[t], size[t] = p[t] * (d @ p[t]), p[t] * (d.abs() @ p[t])
    return want, size


@pytest.mark.parametrize("c", [Cfg(2, 2, "softmax"), Cfg(8, 2, "softmax"), Cfg(60, 4, "softmax"), Cfg(64, 6, "softmax", scale=2.5),
                               Cfg(300, 32, "softmax"), Cfg(2, 1, "softmax", renorm=False), Cfg(8, 2, "softmax", renorm=False),
                               Cfg(60, 4, "softmax", renorm=False, scale=2.5), Cfg(300, 32, "softmax", renorm=False),
                               Cfg(1000, 7, "softmax", renorm=False), Cfg(1, 1), Cfg(64, 6, scale=2.5), Cfg(300, 32)],
                         ids=lambda c: f"{c.score}{c.E}k{c.K}r{int(c.renorm)}")
@pytest.mark.parametrize("spread", [1.0, 4.0, 16.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_gradients_of_confident_routers(S, c, spread, dtype):
    g = torch.Generator(device="cuda").manual_seed(c.E + c.K)
    x = (torch.randn(200, c.E, generator=g, device="cuda") * spread).to(dtype)
    e = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :c.K]
    up = torch.randn(200, c.K, generator=g, device="cuda")
    up[::4] = up[::4, :1] * (1 + 1e-4 * up[::4])               # nearly equal, and equal
    up[::8] = 1.0
    out = torch.full((200, c.E), float("nan"), dtype=dtype, device="cuda")
    S.slide_route_experts_backward(200, x, e.to(torch.int32).contiguous(), up, out, c.of(S),
                                   logits_type=S.SLIDE_TYPE_FP32 if dtype == torch.float32 else S.SLIDE_TYPE_BF16)
    torch.cuda.synchronize()
    want, size = terms64(x, e, up, c)
    tol = 2.0 ** -24 * (48 + 2 * float(x.float().max() - x.float().min())) * size + 2.0 ** -126
    if dtype == torch.bfloat16:  # the rounding of a value within the tolerance
        assert bool((out >= (want - tol).bfloat16()).all()) and bool((out <= (want + tol).bfloat16()).all())
    else:
        assert bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() / tol).max())


@pytest.mark.parametrize("K", [1, 2, 3, 5])
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("depth", [1.0, 30.0, 150.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_renormalised_softmax_where_the_bias_picks_tiny_scores(S, K, groups, depth, dtype):
    """Weights and gradient are those of the softmax of the chosen logits, down
    to scores that FP32 does not hold.  The picks' biases are further apart than
    their scores are large."""
    g = torch.Generator(device="cuda").manual_seed(K)
    E, T, favoured = 16, 100, torch.tensor([3, 5, 8, 12, 13], device="cuda")
    x = torch.randn(T, E, generator=g, device="cuda")
    x[:, favoured] = -20 - depth * torch.rand(T, 5, generator=g, device="cuda")
    x = x.to(dtype)
    bias = torch.zeros(E, device="cuda")
    bias[favoured] = 2 + 0.01 * favoured.float()
    c = Cfg(E, K, "softmax", groups=groups, top_groups=groups, scale=1.5)
    w, e = torch.empty(T, K, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
    kind = S.SLIDE_TYPE_FP32 if dtype == torch.float32 else S.SLIDE_TYPE_BF16
    S.slide_route_experts(T, x, w, e, c.of(S), bias=bias, logits_type=kind)
    up = torch.randn(T, K, generator=g, device="cuda")
    out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    S.slide_route_experts_backward(T, x, e, up, out, c.of(S), logits_type=kind)
    torch.cuda.synchronize()
    chosen = favoured.flip(0)[:K].expand(T, K)
    assert torch.equal(e.long(), chosen)
    rel = 2.0 ** -24 * (48 + 2 * (depth + 25))
    want = torch.softmax(x.double().gather(1, chosen), 1) * 1.5
    assert bool(((w.double() - want).abs() <= rel * want + 2.0 ** -126).all())
    want, size = terms64(x, chosen, up, c)
    tol = rel * size + 2.0 ** -126
    if dtype == torch.bfloat16:
        assert bool((out >= (want - tol).bfloat16()).all()) and bool((out <= (want + tol).bfloat16()).all())
    else:
        assert bool(((out.double() - want).abs() <= tol).all())
