"""slide_route_experts, its gradient and slide_route_bias_step against their
formulas: the choice on FP32 keys exactly, the numbers in 64 bits.

Tolerances: a weight is a quotient of sums of FP32 scores of up to 2 ulp each,
a gradient the difference of two such products, so 1e-6 of the row's largest
gradient term; a BF16 gradient is the rounding of a value within that.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


class Cfg:
    def __init__(self, E, K, score="sigmoid", groups=1, top_groups=1, group_max=False, renorm=True, scale=1.0):
        self.E, self.K, self.score, self.groups, self.top_groups = E, K, score, groups, top_groups
        self.group_max, self.renorm, self.scale = group_max, renorm, scale

    def of(self, S):
        return S.route_config(self.E, self.K, S.SLIDE_SCORE_SIGMOID if self.score == "sigmoid" else S.SLIDE_SCORE_SOFTMAX,
                              self.groups, self.top_groups, S.SLIDE_GROUP_MAX if self.group_max else S.SLIDE_GROUP_TOP2,
                              self.renorm, self.scale)


def reference(x, c, bias=None, mask=None):
    """experts, weights (64 bits), load.  The FP32 keys are formed on the GPU."""
    x32 = x.float()
    T = x32.shape[0]
    if c.score == "sigmoid":
        s64 = torch.sigmoid(x32.double())
        key = 1.0 / (1.0 + torch.exp(-x32))
    else:
        f = x32.clamp_max(torch.finfo(torch.float32).max).double()
        s64 = torch.softmax(f, 1)
        key = s64.float() if bias is not None or (c.groups > 1 and not c.group_max) else x32 + 0.0
    if bias is not None:
        key = key + bias
    nan = torch.isnan(key).any(1) | torch.isnan(x32).any(1)
    key = torch.where(x32 == -INF, -INF, key).cpu()
    if c.groups > 1:
        per = key.view(T, c.groups, -1)
        best = per.sort(2, descending=True)[0]
        rank = best[:, :, 0].clone()
        if not c.group_max and per.shape[2] > 1:
            rank = torch.where(best[:, :, 1] == -INF, rank, rank + best[:, :, 1])
        order = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :c.top_groups]
        keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep[:, :, None], per, -INF).view(T, -1)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    chosen, none = top[1][:, :c.K], top[0][:, :c.K] == -INF
    nan = nan.cpu()
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu() != 0
    w = torch.where(none, 0.0, s64.cpu().gather(1, chosen))
    if c.renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = w * c.scale
    experts = torch.where(none | nan[:, None] | ~live[:, None], -1, chosen)
    w = torch.where(nan[:, None], NAN, w)
    w = torch.where(live[:, None], w, 0.0)
    load = torch.bincount(experts[experts >= 0].flatten(), minlength=c.E)
    return experts, w, load


def route(S, x, c, bias=None, mask=None, stride=None, load=True):
    T = x.shape[0]
    w = torch.full((T, c.K), -5.0, device="cuda")
    e = torch.full((T, c.K), -5, dtype=torch.int32, device="cuda")
    ld = torch.zeros(c.E, dtype=torch.int64, device="cuda") if load else None
    S.slide_route_experts(T, x, w, e, c.of(S), bias=bias, token_mask=mask, load=ld, logits_stride=stride,
                          logits_type=S.SLIDE_TYPE_FP32 if x.dtype == torch.float32 else S.SLIDE_TYPE_BF16)
    torch.cuda.synchronize()
    return e, w, ld


def same(S, x, c, bias=None, mask=None, stride=None):
    e, w, ld = route(S, x, c, bias, mask, stride)
    e0, w0, ld0 = reference(x, c, bias, mask)
    assert torch.equal(e.cpu().long(), e0)
    assert torch.equal(torch.isnan(w.cpu()), torch.isnan(w0))
    d = (w.cpu().double() - w0).nan_to_num().abs()
    assert float((d - 1e-6 * w0.nan_to_num().abs().amax(1, keepdim=True)).max()) <= 1e-30
    assert torch.equal(ld.cpu(), ld0)
    return e, w


def logits(T, E, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * 1.5).to(dtype)


CONFIGS = [Cfg(1, 1), Cfg(2, 1, "softmax"), Cfg(8, 2, "softmax", renorm=False), Cfg(31, 5), Cfg(33, 32), Cfg(60, 4, "softmax"),
           Cfg(64, 6, groups=8, top_groups=3, scale=2.5), Cfg(96, 8, groups=6, top_groups=2), Cfg(100, 7, groups=20, top_groups=5),
           Cfg(128, 8, "softmax", groups=4, top_groups=2, group_max=True, renorm=False, scale=16.0),
           Cfg(160, 6, groups=8, top_groups=3, group_max=True), Cfg(256, 8, groups=8, top_groups=4), Cfg(256, 8, "softmax"),
           Cfg(257, 9), Cfg(384, 12, groups=64, top_groups=7), Cfg(512, 10, groups=8, top_groups=8), Cfg(513, 3, renorm=False),
           Cfg(1024, 32, groups=1024, top_groups=40), Cfg(1000, 11, "softmax", renorm=False)]


@pytest.mark.parametrize("c", CONFIGS, ids=lambda c: f"{c.score}{c.E}k{c.K}g{c.groups}")
@pytest.mark.parametrize("T", [1, 7, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice_and_weights(S, c, T, dtype):
    same(S, logits(T, c.E, T + c.E, dtype), c)


@pytest.mark.parametrize("c", [c for c in CONFIGS if c.score == "sigmoid"], ids=lambda c: f"{c.E}k{c.K}g{c.groups}")
def test_bias_moves_the_choice_only(S, c):
    g = torch.Generator(device="cuda").manual_seed(1)
    same(S, logits(500, c.E, 3), c, bias=torch.randn(c.E, generator=g, device="cuda") * 0.3)


def test_softmax_with_a_bias(S):
    """Scores enter the choice; far enough apart that their last bits do not."""
    c = Cfg(64, 4, "softmax", groups=4, top_groups=2, renorm=False)
    x = torch.stack([torch.randperm(64) for _ in range(200)]).float().cuda() * 0.05
    same(S, x, c, bias=torch.linspace(-0.003, 0.004, 64, device="cuda"))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lowest(S, score):
    for E, K, G, tg in ((64, 8, 1, 1), (64, 8, 8, 4), (256, 16, 8, 3), (90, 7, 9, 4)):
        c = Cfg(E, K, score, groups=G, top_groups=tg, group_max=score == "softmax")
        x = torch.zeros(4, E, device="cuda")
        x[1] = -0.0
        x[1, ::3] = 0.0
        x[2] = torch.arange(E, device="cuda") % 3
        x[3] = (torch.arange(E, device="cuda") // 5) % 2
        e, _ = same(S, x, c)
        if G == 1:
            assert e[0].tolist() == list(range(K)) and e[1].tolist() == list(range(K))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4])
def test_unavailable_experts(S, score, groups):
    """-inf logits, lowest finite ones, rows with nothing left, infinities and NaN."""
    c = Cfg(32, 6, score, groups=groups, top_groups=max(1, groups // 2), group_max=score == "softmax")
    low = torch.finfo(torch.float32).min
    x = logits(12, 32, 1)
    x[0] = -INF
    x[1] = -INF
    x[1, 5] = 0.25
    x[2] = low
    x[3, 3:] = -INF
    x[4] = low
    x[4, 30] = 1.0
    x[5, 7] = NAN
    x[6, 9] = INF
    x[7, 9] = INF
    x[7, 11] = INF
    x[8] = INF
    x[9, ::2] = -INF
    x[10] = NAN
    x[11, :16] = -INF
    same(S, x, c)
    e, w, _ = route(S, x, c)
    assert (e[0] == -1).all() and (w[0] == 0).all()
    assert (e[5] == -1).all() and torch.isnan(w[5]).all()
    assert (e[1] >= 0).sum() == 1 and float(w[1].max()) == pytest.approx(1.0, rel=1e-6)


def test_bias_can_forbid_an_expert(S):
    c = Cfg(40, 4)
    bias = torch.zeros(40, device="cuda")
    bias[:38] = -INF
    e, w, _ = route(S, logits(50, 40, 2), c, bias=bias)
    assert set(e.unique().tolist()) == {-1, 38, 39} and (w[:, 2:] == 0).all()


def test_masked_tokens_are_not_read(S):
    c = Cfg(256, 8, groups=8, top_groups=4)
    x = logits(777, 256, 8)
    mask = (torch.arange(777, device="cuda") % 3 != 0).to(torch.uint8)
    x[mask == 0] = NAN
    e, w = same(S, x, c, mask=mask)
    assert (e[mask == 0] == -1).all() and (w[mask == 0] == 0).all()
    same(S, x, c, mask=torch.zeros_like(mask))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,stride,first", [(60, 61, 0), (64, 80, 16), (256, 257, 1), (256, 264, 8)])
def test_strided_rows(S, dtype, E, stride, first):
    big = logits(300, stride, 5, dtype)
    x = big.as_strided((299, E), (stride, 1), first)
    c = Cfg(E, 5)
    e0, w0, _ = reference(x.contiguous(), c)
    w, e = torch.empty(299, 5, device="cuda"), torch.empty(299, 5, dtype=torch.int32, device="cuda")
    kind = S.SLIDE_TYPE_FP32 if dtype == torch.float32 else S.SLIDE_TYPE_BF16
    S.slide_route_experts(299, x, w, e, c.of(S), logits_type=kind, logits_stride=stride)
    torch.cuda.synchronize()
    assert torch.equal(e.cpu().long(), e0)
    dw = torch.randn(299, 5, device="cuda")
    out = torch.full_like(big, 9.0)
    dst = out.as_strided((299, E), (stride, 1), first)
    S.slide_route_experts_backward(299, x, e, dw, dst, c.of(S), logits_type=kind, logits_stride=stride, d_logits_stride=stride)
    torch.cuda.synchronize()
    check_back(dst.contiguous(), back64(x.contiguous(), e, dw, c), dtype)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep.as_strided((299, E), (stride, 1), first).fill_(False)
    assert (out[keep] == 9.0).all()


def test_load_is_added_and_the_bias_moves_against_it(S):
    c, T = Cfg(64, 4), 5000
    x = logits(T, 64, 4)
    x[:, :8] += 1.0
    bias, load = torch.zeros(64, device="cuda"), torch.zeros(64, dtype=torch.int64, device="cuda")
    w, e = torch.empty(T, 4, device="cuda"), torch.empty(T, 4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        S.slide_route_experts(T, x, w, e, c.of(S), bias=bias, load=load, stream=side)
    side.synchronize()
    _, _, once = reference(x, c)
    assert torch.equal(load.cpu(), 2 * once)
    S.slide_route_bias_step(64, load, bias, 0.25, stream=side)
    side.synchronize()
    want = 0.25 * torch.sign(once.sum() - once * 64).float()
    assert torch.equal(bias.cpu(), want) and (load == 0).all()
    spread = []
    for _ in range(60):
        S.slide_route_experts(T, x, w, e, c.of(S), bias=bias, load=load, stream=side)
        side.synchronize()
        spread.append(int(load.max()))
        S.slide_route_bias_step(64, load, bias, 0.01, stream=side)
    side.synchronize()
    assert spread[-1] < spread[0]


@pytest.mark.parametrize("E", [1, 3, 255, 1024])
def test_bias_step_compares_in_integers(S, E):
    load = torch.randint(0, 1 << 40, (E,), device="cuda")
    load[0] = load[-1]
    bias = torch.randn(E, device="cuda")
    total = sum(load.tolist())
    want = [b + (0.125 if total > v * E else -0.125 if total < v * E else 0.0) for b, v in zip(bias.tolist(), load.tolist())]
    S.slide_route_bias_step(E, load, bias, 0.125)
    torch.cuda.synchronize()
    assert torch.equal(bias.cpu(), torch.tensor(want, dtype=torch.float64).float()) and (load == 0).all()


# ---- the gradient ------------------------------------------------------------------


def weights64(x, experts, c):
    """The weights of a fixed choice, differentiable; x in 64 bits."""
    s = torch.sigmoid(x) if c.score == "sigmoid" else torch.softmax(x, 1)
    w = torch.where(experts >= 0, s.gather(1, experts.clamp_min(0)), 0.0)
    if c.renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return w * c.scale


def back64(x, experts, dw, c, mask=None):
    x = x.detach().double().requires_grad_()
    e = experts.long()
    if mask is not None:
        e = torch.where(mask[:, None] != 0, e, -1)
    (weights64(x, e, c) * dw.double()).sum().backward()
    return x.grad


def check_back(got, want, dtype):
    # 2e-7: cancellation between terms of the size of the row's gradients before they are subtracted
    tol = 1e-6 * want.abs().amax(1, keepdim=True) + 1e-38 + 2e-7
    if dtype == torch.bfloat16:  # the rounding of a value inside the tolerance; rounding keeps the order
        assert bool((got >= (want - tol).bfloat16()).all()) and bool((got <= (want + tol).bfloat16()).all())
    else:
        assert bool(((got.double() - want).abs() <= tol).all())


BACK = [Cfg(1, 1), Cfg(2, 2, "softmax"), Cfg(8, 2, "softmax", renorm=False), Cfg(31, 5), Cfg(60, 4, "softmax", renorm=False),
        Cfg(64, 6, "softmax", scale=2.5), Cfg(256, 8, scale=2.5), Cfg(256, 8, renorm=False), Cfg(257, 9, "softmax", renorm=False),
        Cfg(512, 32), Cfg(1000, 11, "softmax", renorm=False), Cfg(1024, 32, "softmax", renorm=False)]


@pytest.mark.parametrize("c", BACK, ids=lambda c: f"{c.score}{c.E}k{c.K}r{int(c.renorm)}")
@pytest.mark.parametrize("T", [1, 333])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(S, c, T, dtype):
    x = logits(T, c.E, 6, dtype)
    e, _, _ = route(S, x, c)
    dw = torch.randn(T, c.K, device="cuda")
    mask = (torch.arange(T, device="cuda") % 5 != 3).to(torch.uint8)
    for m in (None, mask):
        out = torch.full((T, c.E), NAN, dtype=dtype, device="cuda")
        S.slide_route_experts_backward(T, x, e, dw, out, c.of(S), token_mask=m,
                                       logits_type=S.SLIDE_TYPE_FP32 if dtype == torch.float32 else S.SLIDE_TYPE_BF16)
        torch.cuda.synchronize()
        check_back(out, back64(x, e, dw, c, m), dtype)


@pytest.mark.parametrize("c", [Cfg(20, 3), Cfg(20, 3, renorm=False), Cfg(20, 3, "softmax"), Cfg(20, 3, "softmax", renorm=False)],
                         ids=lambda c: f"{c.score}r{int(c.renorm)}")
def test_gradient_against_differences(S, c):
    x = logits(6, 20, 9)
    e, _, _ = route(S, x, c)
    dw = torch.randn(6, 3, device="cuda")
    out = torch.empty(6, 20, device="cuda")
    S.slide_route_experts_backward(6, x, e, dw, out, c.of(S))
    torch.cuda.synchronize()
    h = 1e-5
    for j in range(20):
        step = torch.zeros(20, dtype=torch.float64, device="cuda")
        step[j] = h
        up, down = (weights64(x.double() + s * step, e.long(), c) for s in (1, -1))
        diff = ((up - down) / (2 * h) * dw.double()).sum(1)
        # the differences' own error is h^2 times third derivatives of order 1
        assert float((out[:, j].double() - diff).abs().max()) <= 1e-6


def test_gradient_of_unfilled_places(S):
    """Places without an expert, indices out of range and masked infinities contribute nothing."""
    for c in (Cfg(16, 4), Cfg(16, 4, "softmax"), Cfg(16, 4, "softmax", renorm=False)):
        x = logits(5, 16, 1)
        x[0, 2:] = -INF
        x[1] = -INF
        e, w, _ = route(S, x, c)
        e[4, 1] = 16
        e[4, 2] = -9
        dw = torch.randn(5, 4, device="cuda")
        dw[0, 2:] = NAN
        out = torch.full((5, 16), NAN, device="cuda")
        S.slide_route_experts_backward(5, x, e, dw, out, c.of(S))
        torch.cuda.synchronize()
        valid = torch.where((e >= 0) & (e < 16), e, -1)
        want = back64(torch.where(x == -INF, -1e30, x.double()), valid, torch.where(valid >= 0, dw, 0.0), c)
        want[1] = 0
        check_back(out, want, torch.float32)
