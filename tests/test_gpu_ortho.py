"""slide_orthogonalize, slide_muon_step and slide_layer_muon_step against their
formulas in 64 bits.

Tolerances.  The orthogonal factor's products round their operands to FP16
(2^-12 relative) and are amplified by the polynomial's cancellations: an
emulation of the roundings gives up to 2.8e-3 (2-norm) over spectra from flat
to falling, so FACTOR = 4e-3; for a matrix of one repeated value, whose
roundings all have one sign, up to 3e-2, so COHERENT = 5e-2.  Rounding
many values to BF16 adds 1.7e-3 (2-norm), BF16 = 2^-9; of a single value it may
be 2^-8, which FACTOR has room for.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FACTOR, COHERENT, BF16 = 4e-3, 5e-2, 2.0 ** -9
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(batch, rows, cols, seed, kind="falling", rms=1e-3):
    g = gen(seed)
    x = torch.randn(batch, rows, cols, generator=g, device="cuda")
    if kind == "falling":
        r = min(16, rows, cols)
        u, v = torch.randn(batch, rows, r, generator=g, device="cuda"), torch.randn(batch, r, cols, generator=g, device="cuda")
        x = x + (u * torch.arange(1, r + 1, device="cuda").rsqrt() * 0.3) @ v
    elif kind == "one value":
        x = torch.ones_like(x)
    return x * rms


def factor64(x, steps=5, coeffs=None, eps=1e-7):
    x = x.double()
    x = x / (x.flatten(1).norm(dim=1).view(-1, 1, 1) + eps)
    for k in range(steps):
        a, b, c = coeffs[k] if coeffs else QUINTIC
        if x.shape[1] <= x.shape[2]:
            p = x @ x.mT
            x = a * x + (b * p + c * (p @ p)) @ x
        else:
            p = x.mT @ x
            x = a * x + x @ (b * p + c * (p @ p))
    return x


def off(got, want):
    """Largest 2-norm error over 2-norm of a batch's matrices."""
    d = (got.double() - want).flatten(1).norm(dim=1)
    return float((d / want.flatten(1).norm(dim=1).clamp_min(1e-300)).max())


def workspace(S, *shape):
    # its contents are irrelevant: all bits set is NaN in every type
    return torch.full((S.slide_ortho_workspace(*shape),), 0xff, dtype=torch.uint8, device="cuda")


def orthogonalize(S, x, params=None, stream=None):
    b, r, c = x.shape
    out = torch.full((b, r, c), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = workspace(S, b, r, c)
    S.slide_orthogonalize(b, r, c, x, out, params or S.ortho_params(), ws,
                          x_type=S.SLIDE_TYPE_FP32 if x.dtype == torch.float32 else S.SLIDE_TYPE_BF16, stream=stream)
    assert S.slide_ortho_status(ws, stream) == S.SLIDE_OK
    return out


SHAPES = [(1, 1, 1), (3, 1, 19), (2, 19, 1), (1, 2, 2), (1, 64, 64), (2, 63, 65), (1, 127, 129), (1, 128, 128),
          (2, 129, 127), (1, 64, 2560), (1, 2560, 64), (1, 128, 1000), (1, 256, 256), (1, 255, 511), (1, 300, 700),
          (2, 700, 300), (1, 1000, 1001), (1, 1001, 1000), (5, 130, 390), (40, 200, 328), (1, 512, 4096), (1, 4097, 513),
          (1, 1537, 1536), (2, 1024, 2560)]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_factor(S, batch, rows, cols, dtype):
    x = matrix(batch, rows, cols, rows * 7 + cols).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert off(orthogonalize(S, x), factor64(x)) <= FACTOR + BF16


@pytest.mark.parametrize("batch,rows,cols", [(1, 129, 1535), (1, 129, 1537), (2, 238, 14962), (3, 2100, 300), (1, 6401, 513),
                                             (25, 200, 2000), (26, 200, 2000), (1, 1025, 2085), (1, 200, 1600), (1, 1900, 400),
                                             (3, 150, 1545)])
@pytest.mark.parametrize("more", [0, 11])
def test_long_sides_of_few_tiles(S, batch, rows, cols, more):
    """The sums over a long side taken apart among CTAs: right, and the same
    bits each time (the parts are added in their order, whoever comes last).
    The steps after the quintic's five draw the singular values to 1, where
    their slope is 0, so they let no error grow."""
    coeffs = [QUINTIC] * 5 + [(1.875, -1.25, 0.375)] * more
    x = matrix(batch, rows, cols, rows + cols)
    params = S.ortho_params(steps=5 + more, coeffs=coeffs)
    first = orthogonalize(S, x, params)
    assert off(first, factor64(x, 5 + more, coeffs)) <= FACTOR + BF16
    for _ in range(5):
        assert torch.equal(orthogonalize(S, x, params).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("rows,cols", [(33, 33), (100, 300), (257, 256), (640, 200), (384, 1500)])
@pytest.mark.parametrize("kind", ["flat", "one value"])
def test_spectra(S, rows, cols, kind):
    x = matrix(2, rows, cols, 5, kind)
    assert off(orthogonalize(S, x), factor64(x)) <= (COHERENT if kind == "one value" else FACTOR) + BF16


@pytest.mark.parametrize("rows,cols", [(60, 200), (300, 520), (520, 300), (400, 400)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7])
def test_steps(S, rows, cols, steps):
    x = matrix(1, rows, cols, steps)
    assert off(orthogonalize(S, x, S.ortho_params(steps=steps)), factor64(x, steps)) <= FACTOR + BF16


def test_own_coefficients(S):
    coeffs = [(3.0, -3.2, 1.2), (2.5, -2.2, 0.7), (1.875, -1.25, 0.375), (1.875, -1.25, 0.375)]
    for rows, cols in ((200, 260), (130, 600), (64, 90)):
        x = matrix(1, rows, cols, 3)
        got = orthogonalize(S, x, S.ortho_params(steps=4, coeffs=coeffs))
        assert off(got, factor64(x, 4, coeffs)) <= FACTOR + BF16


def test_scale_of_the_input_plays_no_part(S):
    x = matrix(1, 200, 300, 9)
    want = factor64(x)
    for s in (1e-6, 1e6, 1e12):
        assert off(orthogonalize(S, x * s, S.ortho_params(eps=0.0)), want) <= FACTOR + BF16


@pytest.mark.parametrize("rows,cols", [(50, 70), (200, 333), (300, 300)])
def test_zeros_and_nonfinite(S, rows, cols):
    """Zeros give zeros (with and without eps); NaN and Inf stay in their matrix."""
    for eps in (1e-7, 0.0):
        x = matrix(4, rows, cols, 11)
        x[1] = 0
        x[2, rows // 2, cols // 2] = float("nan")
        x[3, 0, 0] = float("inf")
        got = orthogonalize(S, x, S.ortho_params(eps=eps))
        assert off(got[:1], factor64(x[:1], eps=eps)) <= FACTOR + BF16
        assert (got[1] == 0).all()
        assert torch.isnan(got[2]).all() and torch.isnan(got[3]).any()


def test_strides(S):
    """Rows and matrices apart, a repeated matrix, odd offsets: only the result's places are written."""
    b, r, c = 3, 150, 203
    big = matrix(b, r + 5, c + 6, 4)
    x = big[:, :r, 1:1 + c]                                    # base not 16-byte aligned
    out = torch.full((b, r + 2, c + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(S, b, r, c)
    S.slide_orthogonalize(b, r, c, x, out[:, :, 3:], S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32,
                          x_row_stride=c + 6, x_batch_stride=(r + 5) * (c + 6), out_row_stride=c + 8,
                          out_batch_stride=(r + 2) * (c + 8))
    assert off(out[:, :r, 3:3 + c], factor64(x)) <= FACTOR + BF16
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[:, :r, 3:3 + c] = False
    assert (out[mask] == -7.0).all()
    one = x[:1].contiguous()
    rep = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    S.slide_orthogonalize(b, r, c, one, rep, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32, x_batch_stride=0)
    assert (rep[0] == rep[1]).all() and (rep[0] == rep[2]).all()


def test_same_bits_again_and_beside_other_work(S):
    x = matrix(2, 700, 1500, 21)
    first = orthogonalize(S, x)
    side = torch.cuda.Stream()
    y = matrix(1, 900, 800, 22)
    torch.cuda.synchronize()
    want = orthogonalize(S, y)
    for _ in range(3):
        out = torch.empty_like(first)
        ws, ws2, o2 = workspace(S, *x.shape), workspace(S, *y.shape), torch.empty_like(want)
        torch.cuda.synchronize()
        S.slide_orthogonalize(*x.shape, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32)
        S.slide_orthogonalize(*y.shape, y, o2, S.ortho_params(), ws2, x_type=S.SLIDE_TYPE_FP32, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(o2, want)


def test_in_a_graph(S):
    x = matrix(1, 300, 500, 2)
    out = torch.zeros(1, 300, 500, dtype=torch.bfloat16, device="cuda")
    ws = workspace(S, 1, 300, 500)

    def call():
        S.slide_orthogonalize(1, 300, 500, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32,
                              stream=torch.cuda.current_stream())
    call()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    x.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


@pytest.mark.parametrize("rows,cols", [(300, 700), (60, 200)])
def test_a_wait_that_runs_out_is_reported(S, monkeypatch, rows, cols):
    x = matrix(1, rows, cols, 1)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    ws = workspace(S, 1, rows, cols)
    monkeypatch.setenv("SLIDE_TEST_PIPELINE_STALL", "1")
    S.slide_orthogonalize(1, rows, cols, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32)
    assert S.slide_ortho_status(ws) == S.SLIDE_ERR_TIMEOUT
    monkeypatch.delenv("SLIDE_TEST_PIPELINE_STALL")
    S.slide_orthogonalize(1, rows, cols, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32)
    assert S.slide_ortho_status(ws) == S.SLIDE_OK
    assert off(out, factor64(x)) <= FACTOR + BF16


# ---- the Muon step ---------------------------------------------------------------


def muon64(grads, mom, th, lr, mu, wd, scale, nesterov, steps=5):
    g = torch.stack([x.double() for x in grads]).mean(0)
    mom = mu * mom.double() + (1 - mu) * g
    u = mu * mom + (1 - mu) * g if nesterov else mom
    o = factor64(u, steps)
    return th.double() * (1 - lr * wd) - lr * scale * o, mom, o


def check_muon(S, th, mom, w, want, lr, scale, th0):
    t64, m64, o = want
    # a few FP32 roundings of values of the terms' size
    assert float(((mom.double() - m64).abs() / (m64.abs() + m64.square().mean().sqrt())).max()) <= 16 * 2.0 ** -24
    err = (th.double() - t64).norm()
    assert float(err) <= 2.0 ** -22 * float(th0.double().norm()) + lr * scale * FACTOR * float(o.norm())
    assert torch.equal(w, th.bfloat16())


@pytest.mark.parametrize("batch,rows,cols,R,dtype,nesterov", [
    (1, 1, 1, 1, "fp32", True), (1, 64, 64, 3, "bf16", True), (2, 130, 70, 8, "bf16", False), (1, 77, 500, 2, "fp32", True),
    (3, 201, 333, 5, "fp32", False), (1, 640, 256, 4, "bf16", True), (7, 100, 273, 2, "fp32", True),
    (1, 515, 517, 1, "bf16", True), (2, 512, 1536, 4, "bf16", True)])
def test_muon_step(S, batch, rows, cols, R, dtype, nesterov):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    common = matrix(batch, rows, cols, 1)
    g = gen(2)
    grads = [(common + torch.randn(common.shape, generator=g, device="cuda") * 1e-3).to(dt) for _ in range(R)]
    mom, th = matrix(batch, rows, cols, 3), torch.randn(common.shape, generator=g, device="cuda") * 0.02
    lr, mu, wd, scale = 0.01, 0.9, 0.1, 0.5
    for it in range(2):
        want = muon64(grads, mom, th, lr, mu, wd, scale, nesterov)
        th0, w = th.clone(), torch.full(th.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        S.slide_muon_step(batch, rows, cols, grads, th, mom, w,
                          S.muon_hparams(lr=lr, momentum=mu, weight_decay=wd, scale=scale, nesterov=nesterov),
                          workspace(S, batch, rows, cols),
                          grads_type=S.SLIDE_TYPE_FP32 if dtype == "fp32" else S.SLIDE_TYPE_BF16)
        torch.cuda.synchronize()
        check_muon(S, th, mom, w, want, lr, scale, th0)


def test_muon_default_scale_and_zero_gradients(S):
    r, c = 96, 160
    th = torch.randn(1, r, c, device="cuda")
    th0, mom = th.clone(), torch.zeros(1, r, c, device="cuda")
    w = torch.empty(1, r, c, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(1, r, c, dtype=torch.bfloat16, device="cuda")
    S.slide_muon_step(1, r, c, [zero], th, mom, w, S.muon_hparams(lr=0.1, weight_decay=0.5), workspace(S, 1, r, c))
    torch.cuda.synchronize()
    assert torch.equal(th, th0 * np.float32(1 - float(np.float32(0.1)) * 0.5)) and (mom == 0).all()
    g = matrix(1, r, c, 8).bfloat16()
    want = muon64([g], mom, th, 0.1, 0.95, 0.0, 0.2 * math.sqrt(c), True)
    th0 = th.clone()
    S.slide_muon_step(1, r, c, [g], th, mom, w, S.muon_hparams(lr=0.1, weight_decay=0.0), workspace(S, 1, r, c))
    torch.cuda.synchronize()
    check_muon(S, th, mom, w, want, 0.1, 0.2 * math.sqrt(c), th0)


@pytest.mark.parametrize("fp32", [False, True])
def test_layer_step_with_matrices(S, fp32):
    """Blocks by Muon, everything else bit for bit as slide_layer_step."""
    blocks = [(0, 2, 64, 96), (2 * 64 * 96 + 128, 1, 200, 72), (2 * 64 * 96 + 128 + 200 * 72 + 8, 1, 33, 35)]
    n = blocks[-1][0] + 33 * 35
    R, dt = 2, torch.float32 if fp32 else torch.bfloat16
    g = gen(5)
    flags = S.SLIDE_FLAG_FP32_GRADS if fp32 else 0
    th = torch.randn(n, generator=g, device="cuda").cpu().numpy() * np.float32(0.02)
    adam, muon = S.hparams(lr=1e-3), S.muon_hparams(lr=0.02, momentum=0.8, scale=1.0)
    a, b = S.slide_state_create([n], R, flags=flags), S.slide_state_create([n], R, flags=flags)
    ws = torch.empty(max(S.slide_ortho_workspace(*x[1:]) for x in blocks), dtype=torch.uint8, device="cuda")
    try:
        inside = np.zeros(n, bool)
        for off_, k, r, c in blocks:
            inside[off_:off_ + k * r * c] = True
        for st in (a, b):
            S.slide_layer_set(st, 0, master=th, step=0)
        mom = np.zeros(n, np.float32)
        for step in range(1, 3):
            grads = [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(dt) for _ in range(R)]
            S.slide_layer_step(a, 0, grads, adam)
            S.slide_layer_muon_step(b, 0, blocks, grads, muon, adam, ws)
            ga, gb = [[np.empty(n, np.float32) for _ in range(3)] + [np.empty(n, np.uint16)] for _ in range(2)]
            old = th.copy()
            assert S.slide_layer_get(a, 0, *ga) == S.slide_layer_get(b, 0, *gb) == step
            for x, y in zip(ga, gb):
                assert (x[~inside].view(np.uint8) == y[~inside].view(np.uint8)).all()
            assert (gb[2][inside] == 0).all()                    # v of the matrices is left alone
            for off_, k, r, c in blocks:
                sl, shape = slice(off_, off_ + k * r * c), (k, r, c)
                at = lambda v: torch.from_numpy(v[sl].copy()).cuda().view(shape)  # noqa: E731
                want = muon64([x[sl].view(shape) for x in grads], at(mom), at(old), 0.02, 0.8, 0.01, 1.0, True)
                w = torch.from_numpy(gb[3][sl].view(np.int16).copy()).cuda().view(torch.bfloat16).view(shape)
                check_muon(S, at(gb[0]), at(gb[1]), w, want, 0.02, 1.0, at(old))
            th, mom = gb[0], gb[1]
            S.slide_layer_set(a, 0, master=ga[0], m=ga[1], v=ga[2], step=step)
    finally:
        S.slide_state_destroy(a)
        S.slide_state_destroy(b)
