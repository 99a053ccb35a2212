"""slide_linear_cross_entropy at its limits, against its formulas in 64 bits: infinite
logits, sums over very many products, and the roundings of its gradients.

u = 2^-24 is half a step of FP32, B = 2^-8 half a step of BF16.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = float("inf")
U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


def call(S, x, w, y, d_x=True, d_weight=True, d_loss=None):
    T, H = x.shape
    V = w.shape[0]
    o = {"loss": torch.empty(T, device="cuda"), "lse": torch.empty(T, device="cuda"), "total": torch.empty(1, device="cuda")}
    if d_x:
        o["d_x"] = torch.empty_like(x)
    if d_weight:
        o["d_weight"] = torch.empty_like(w)
    ws = torch.empty(S.slide_linear_cross_entropy_workspace(T, H, V, d_x, d_weight), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream()
    S.slide_linear_cross_entropy(T, H, V, x, w, y, o["loss"], ws, d_loss=d_loss, lse=o["lse"], total=o["total"], d_x=o.get("d_x"),
                                 d_weight=o.get("d_weight"), stream=s)
    assert S.slide_linear_cross_entropy_status(ws, stream=s) == S.SLIDE_OK
    return o


def overflowing(T, H=64, V=200, seed=0):
    """Finite factors whose logits of word 10 leave FP32 for every other token: 2^100 times -2^100.
    The remaining logits are a few units, what column 0 adds to them at most one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") * 0.1).bfloat16()
    x[:, 0] = 0.0
    x[::2, 0] = 2.0 ** 100
    w[:, 0] = (torch.rand(V, generator=g, device="cuda") * 2.0 ** -100).bfloat16()
    w[10, 0] = -2.0 ** 100
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::4] = 10
    y[1] = 10                                                    # a token for which the word counts
    return x, w, y


def gradients(x, w, y, up):
    """In 64 bits, and the sums of the terms' magnitudes."""
    q = torch.softmax(x.double() @ w.double().T, 1)
    q[torch.arange(len(y), device="cuda"), y] -= 1
    q *= up
    return {"d_x": (q @ w.double(), q.abs() @ w.double().abs()), "d_weight": (q.T @ x.double(), q.abs().T @ x.double().abs())}


def within_terms(o, want, rows=slice(None)):
    """Three roundings of a term and one of the result, the logits' own errors below 1e-4."""
    for k, (r, size) in want.items():
        bad = ~((o[k].double() - r).abs() <= (3.05 * B + 1e-4) * size + 1.01 * B * r.abs())
        if k == "d_x":
            bad = bad[rows]
        assert not bad.any(), (k, bad.nonzero()[0].tolist())


@pytest.mark.parametrize("T", [6, 100, 700])
def test_a_target_of_minus_infinity(S, T):
    """lse is that of the other words, the loss infinite, the gradients those of p = 0."""
    x, w, y = overflowing(T)
    o = call(S, x, w, y)
    z = x.double() @ w.double().T                                # -2^200 in 64 bits: nothing beside the others
    lse = torch.logsumexp(z, 1)
    # sums of 64 products below 8 and of 200 words, the exponential and the logarithm
    assert ((o["lse"].double() - lse).abs() <= 1e-5).all()
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[::4] = True
    assert (o["loss"][gone] == INF).all() and o["total"].item() == INF
    own = z.gather(1, y[:, None])[:, 0]
    assert ((o["loss"].double() - (lse - own)).abs() <= 1e-5)[~gone].all()
    within_terms(o, gradients(x, w, y, 1 / T))


@pytest.mark.parametrize("T", [6, 700])
def test_a_logit_of_plus_infinity(S, T):
    """NaN for its tokens, of which it is the target's for some, and in all of the weight's gradient, which
    they enter; the others are as they are without them."""
    x, w, y = overflowing(T)
    w[10, 0] = 2.0 ** 100
    o = call(S, x, w, y, d_weight=False)
    x2, y2 = x.clone(), y.clone()
    y2[::2] = -1
    x2[::2] = 0
    o2 = call(S, x2, w, y2, d_weight=False, d_loss=torch.full((T,), 1 / T, device="cuda"))
    for k in ("loss", "lse", "d_x"):
        assert torch.isnan(o[k][::2]).all(), k
        assert torch.equal(o[k][1::2], o2[k][1::2]), k
    assert torch.isnan(call(S, x, w, y)["d_weight"]).all()


@pytest.mark.parametrize("T", [6, 700])
def test_a_target_of_minus_infinity_and_others_far_below_zero(S, T):
    """No logit is a reference of the others' size at first: all others lie near -100 or -1000, whose
    exponentials are 0 in FP32."""
    x, w, y = overflowing(T)
    x[:, 1] = 1.0
    x[::8, 1] = 8.0
    w[:, 1] = -120.0
    o = call(S, x, w, y)
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    # sums of magnitudes up to 1000 in at most eight steps, each off by a step of FP32 at most
    assert ((o["lse"].double() - lse).abs() <= 16 * U * lse.abs() + 1e-5).all()
    assert (o["loss"][::4] == INF).all() and torch.isfinite(o["loss"][1::2]).all()
    within_terms(o, gradients(x, w, y, 1 / T))


@pytest.mark.parametrize("T", [6, 700])
@pytest.mark.parametrize("k", [10, 20, 40, 100])
def test_a_target_far_below_the_others(S, T, k):
    """The others' logits lie around 120 or 960; the target's at -2^k, where FP32's steps are up to 2^77,
    so nothing may pass through a difference from it but the loss."""
    x, w, y = overflowing(T)
    x[::2, 0] = 1.0
    w[10, 0] = -2.0 ** k
    x[:, 1] = 1.0
    x[::8, 1] = 8.0
    w[:, 1] = 120.0
    o = call(S, x, w, y)
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    # sums of magnitudes up to 1000 in at most eight steps, each off by a step of FP32 at most
    assert ((o["lse"].double() - lse).abs() <= 16 * U * lse.abs() + 1e-5).all()
    loss = lse - z.gather(1, y[:, None])[:, 0]
    assert ((o["loss"].double() - loss).abs() <= 16 * U * (lse.abs() + loss) + 1e-5).all()
    within_terms(o, gradients(x, w, y, 1 / T))


@pytest.mark.parametrize("T", [65536, 262144, 1000001])
def test_d_weight_of_very_many_tokens(S, T):
    """Every term of these sums is positive, so an addition that cuts shows in their mean.  The
    matrix unit adds 4096 products at a time (256 additions, each off by a step of FP32 at most) and
    the sums of those are rounded.  The terms' roundings and those of the results have no sign of
    their own: at most B/sqrt(3) each in the mean square, over 63 * 256 results five deviations."""
    H, V = 256, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    # (each column has a size of its own: a mean over many tokens is nearly the same in all, and would be
    # rounded the same way)
    size = 1 + torch.rand(H, generator=g, device="cuda")
    x = ((torch.rand(T, H, generator=g, device="cuda") + 0.5) * size).bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") * 0.02 / size).bfloat16()
    o = call(S, x, w, torch.zeros(T, dtype=torch.int64, device="cuda"), d_x=False)
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 65536):
        part = x[a:a + 65536].double()
        want += torch.softmax(part @ w.double().T, 1).T @ part / T
    off = (o["d_weight"].double() / want - 1)[1:]                # word 0 is the target
    assert abs(float(off.mean())) <= (256 + 2) * 2 * U + (T / 4096) * U + 5 * B / 3 ** 0.5 / off.numel() ** 0.5
    assert float(off.abs().max()) <= 3.05 * B


def test_d_x_of_a_very_long_vocabulary(S):
    """The same for d_x, its sums over 98304 words in one part; a token's factor takes the target's rounding
    (B/sqrt(3) at most) onto all of its results, so 9728 of them count, not 9728 * 512."""
    T, H, V = 9728, 512, 98304
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(T, H, generator=g, device="cuda") * 0.05).bfloat16()
    w = ((torch.rand(V, H, generator=g, device="cuda") + 0.5) * (1 + torch.rand(H, generator=g, device="cuda"))).bfloat16()
    w[0] = 0                                                     # the target, so that all terms are positive
    o = call(S, x, w, torch.zeros(T, dtype=torch.int64, device="cuda"), d_weight=False)
    wd, mean = w.double(), 0.0
    for a in range(0, T, 1216):
        off = o["d_x"][a:a + 1216].double() / (torch.softmax(x[a:a + 1216].double() @ wd.T, 1) @ wd / T) - 1
        assert float(off.abs().max()) <= 3.05 * B
        mean += float(off.sum()) / (T * H)
    assert abs(mean) <= (256 + 2) * 2 * U + (V / 4096) * U + 5 * B / 3 ** 0.5 / T ** 0.5


@pytest.mark.parametrize("T,H,V", [(64, 512, 5000), (100, 256, 2000), (128, 1024, 3001), (129, 512, 5000), (400, 512, 5000), (3000, 264, 1003)])
@pytest.mark.parametrize("std", [0.3, 1.2, 3.0])
def test_roundings_of_the_gradients(S, T, H, V, std):
    """The 2-norm of the errors is that of the roundings which the formulas name, and of no other.  With r
    the relative size of one (own: that of the results, in the mean square), they are independent:
      d_x       the result; each other word's e; the token's factor, on the sum of the other words
      d_weight  the result; each other word's e and the token's factor on it; from 129 tokens on the rounding of
                x times the factor, on every term
    (the target's own place costs nothing: the factor takes its rounding out).  r differs by 8 % at most
    between the values' distributions (1.53e-3 to 1.66e-3)."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") * (std / H ** 0.5)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    o = call(S, x, w, y)
    xd, wd = x.double(), w.double()
    q = torch.softmax(xd @ wd.T, 1) / T
    others = q.clone()
    at = torch.arange(T, device="cuda")
    q[at, y] -= 1 / T
    others[at, y] = 0
    want_x, want_w = q @ wd, q.T @ xd
    more_x = (others.square() @ wd.square()).sum() + (others @ wd).square().sum()
    more_w = 2 * (others.square().T @ xd.square()).sum()
    if T > 128:
        more_w = more_w + (q.square().T @ xd.square()).sum()
    for k, want, more in (("d_x", want_x, more_x), ("d_weight", want_w, more_w)):
        own = float((want.bfloat16().double() - want).norm())
        size = float(want.square().sum())
        off = float((o[k].double() - want).norm())
        assert off <= 1.08 * own * (1 + float(more) / size) ** 0.5, (k, off / size ** 0.5, own / size ** 0.5)


@pytest.mark.parametrize("hidden", [512, 1024, 1032, 5120, 16384, 65536])
@pytest.mark.parametrize("sign", ["one", "any"])
def test_logits_are_as_near_as_stated(S, hidden, sign):
    """lse off by 1.1e-6 of the sum of the products' magnitudes in the mean and 2e-6 at most where all have
    one sign, by 3e-7 where they have any, at any width: the figures of the header."""
    g = torch.Generator(device="cuda").manual_seed(hidden + 1)
    T, V = 600, 8
    x, w = torch.rand(T, hidden, generator=g, device="cuda") + 0.5, torch.zeros(V, hidden, device="cuda")
    w[1] = torch.rand(hidden, generator=g, device="cuda") + 0.5
    if sign == "any":
        x, w[1] = torch.randn(T, hidden, generator=g, device="cuda"), torch.randn(hidden, generator=g, device="cuda")
    x, w = (x * (24 / (x @ w[1]))[:, None]).bfloat16(), w.bfloat16()
    size = x.double().abs() @ w[1].double().abs()
    lse = torch.logsumexp(x.double() @ w.double().T, 1)
    o = call(S, x, w, torch.zeros(T, dtype=torch.int64, device="cuda"), d_x=False, d_weight=False)
    off = (o["lse"].double() - lse).abs() / size
    assert float(off.mean()) <= 1.1e-6 and float(off.max()) <= (2e-6 if sign == "one" else 3e-7)
