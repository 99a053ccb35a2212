"""slide_orthogonalize and the Muon steps at their limits: values at the ends of
their type's range, non-finite ones, waits that run out.  Formulas and
tolerances are test_gpu_ortho's.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_ortho import (BF16, FACTOR, S, check_muon, factor64, gen, matrix, off, orthogonalize,  # noqa: E402, F401
                            workspace)


@pytest.mark.parametrize("batch,rows,cols", [(2, 50, 70), (1, 64, 2560), (2, 3000, 100), (1, 1, 7), (2, 200, 333),
                                             (1, 300, 900), (1, 900, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-16, 1e18, 1e22, 1e30, 1e37])
def test_values_at_the_ends_of_the_range(S, batch, rows, cols, dtype, scale):
    """The squares of finite values, and the norm, may lie outside FP32's range.
    Denormal BF16 and FP32 values are what they are: the formula sees the same."""
    x = matrix(batch, rows, cols, 9, rms=1.0)
    x[batch - 1] *= 0.5                                        # a norm of its own
    x = (x * scale).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert x.isfinite().all() and (x != 0).any()
    assert off(orthogonalize(S, x, S.ortho_params(eps=0.0)), factor64(x, eps=0.0)) <= FACTOR + BF16
    if scale > 1:
        assert off(orthogonalize(S, x), factor64(x)) <= FACTOR + BF16
    r, c = rows + 1, cols + 3                                  # rows apart
    big = torch.zeros(batch, r, c, dtype=x.dtype, device="cuda")
    big[:, :rows, 1:1 + cols] = x
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    S.slide_orthogonalize(batch, rows, cols, big[:, :, 1:], out, S.ortho_params(eps=0.0), workspace(S, batch, rows, cols),
                          x_type=S.SLIDE_TYPE_FP32 if dtype == "fp32" else S.SLIDE_TYPE_BF16, x_row_stride=c,
                          x_batch_stride=r * c)
    assert off(out, factor64(x, eps=0.0)) <= FACTOR + BF16


@pytest.mark.parametrize("rows,cols", [(60, 90), (120, 40), (200, 340)])
def test_one_batch_of_many_magnitudes(S, rows, cols):
    """Each matrix has a range of its own; zeros among them; within a matrix
    values far below the largest play no part."""
    x = matrix(6, rows, cols, 12, rms=1.0)
    for k, s in enumerate((1e-33, 1e30, 0.0, 1.0, 1e-21, 1e21)):
        x[k] *= s
    x[1, ::2] *= 1e-25
    got, want = orthogonalize(S, x, S.ortho_params(eps=0.0)), factor64(x, eps=1e-300)
    assert (got[2] == 0).all()
    keep = [0, 1, 3, 4, 5]
    assert off(got[keep], want[keep]) <= FACTOR + BF16


@pytest.mark.parametrize("rows,cols", [(50, 70), (1, 9), (9, 1), (100, 900), (200, 333), (300, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_nonfinite_value_makes_all_of_its_matrix_nan(S, rows, cols, dtype, bad):
    x = matrix(3, rows, cols, 13).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x[1, rows // 2, cols // 3] = bad
    got = orthogonalize(S, x)
    assert torch.isnan(got[1]).all()
    assert off(got[::2], factor64(x[::2])) <= FACTOR + BF16


@pytest.mark.parametrize("rows,cols", [(64, 300), (300, 100), (200, 331)])
@pytest.mark.parametrize("size", [1e-30, 1e24, 1e33])
def test_muon_step_of_values_at_the_ends_of_the_range(S, rows, cols, size):
    grads = [matrix(2, rows, cols, k, rms=1.0) * size for k in (1, 2)]
    mom, th = matrix(2, rows, cols, 3, rms=1.0) * size, torch.randn(2, rows, cols, generator=gen(4), device="cuda")
    lr, mu, scale = 0.1, 0.9, 0.5
    g = torch.stack([x.double() for x in grads]).mean(0)
    m64 = mu * mom.double() + (1 - mu) * g
    o = factor64(mu * m64 + (1 - mu) * g, eps=0.0)
    want, th0 = (th.double() - lr * scale * o, m64, o), th.clone()
    w = torch.empty(th.shape, dtype=torch.bfloat16, device="cuda")
    S.slide_muon_step(2, rows, cols, grads, th, mom, w, S.muon_hparams(lr=lr, momentum=mu, weight_decay=0.0, scale=scale, eps=0.0),
                      workspace(S, 2, rows, cols), grads_type=S.SLIDE_TYPE_FP32)
    torch.cuda.synchronize()
    check_muon(S, th, mom, w, want, lr, scale, th0)


QUINTIC5 = [(3.4445, -4.7750, 2.0315)] * 5
# coefficients of a steep start, which the last ones bring to 1
STEEP = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in (
    (8.28721, -23.59589, 17.30039), (4.10706, -2.94785, 0.54484), (3.94869, -2.9089, 0.55182), (3.31842, -2.48849, 0.51005),
    (2.30065, -1.6689, 0.41881), (1.9101, -1.3064, 0.39602), (1.9101, -1.3064, 0.39602))]


def strong_directions(batch, rows, cols, count, noise, seed):
    g = gen(seed)
    u, v = torch.randn(batch, rows, count, generator=g, device="cuda"), torch.randn(batch, count, cols, generator=g, device="cuda")
    x = (u * torch.arange(1, count + 1, device="cuda").rsqrt()) @ v / count ** 0.5
    return x + noise * torch.randn(batch, rows, cols, generator=g, device="cuda")


@pytest.mark.parametrize("batch,rows,cols", [(2, 238, 14962), (1, 8000, 300), (1, 640, 4096), (3, 1000, 3000), (1, 100, 3000)])
@pytest.mark.parametrize("coeffs", [QUINTIC5, QUINTIC5 + QUINTIC5[:1], STEEP[:5], STEEP], ids=["quintic5", "quintic6", "steep5", "steep7"])
@pytest.mark.parametrize("count,noise", [(4, 1e-2), (32, 1e-2), (32, 1e-3), (128, 1e-3)])
def test_strong_directions_over_noise(S, batch, rows, cols, coeffs, count, noise):
    """What is amplified to singular values near 1 from far below, beside others
    that are there already.  Five steps are to stay within FACTOR; each step more
    may let an error grow by the square root of 1.8, the quintic's slope over its
    cycle of two.  A side of at most 128 has too few entries for the roundings to
    average: five times that."""
    x = strong_directions(batch, rows, cols, min(count, rows, cols), noise, 5)
    n = len(coeffs)
    allowed = FACTOR * 1.8 ** ((n - 5) / 2) * (5 if min(rows, cols) <= 128 else 1)
    if n == 6 and min(rows, cols) < 300:
        allowed *= 1.25                                        # the groups of two of so small a side
    got = orthogonalize(S, x, S.ortho_params(steps=n, coeffs=coeffs))
    assert off(got, factor64(x, n, coeffs)) <= allowed + BF16


@pytest.mark.parametrize("blocks", [((0, 1, 64, 96), (6144, 1, 200, 72)), ((0, 1, 300, 200), (60000, 1, 64, 96)),
                                    ((0, 1, 200, 200), (40000, 0, 8, 8), (40000, 2, 150, 160), (88000, 3, 40, 8))])
def test_a_wait_that_runs_out_in_a_layers_first_block_is_reported(S, monkeypatch, blocks):
    """By the workspace's word and the layer's, though the blocks after it share
    the workspace; the next step starts afresh."""
    n = blocks[-1][0] + blocks[-1][1] * blocks[-1][2] * blocks[-1][3] + 16
    st = S.slide_state_create([n], 1)
    grads = [torch.randn(n, generator=gen(1), device="cuda").bfloat16()]
    ws = torch.full((max(S.slide_ortho_workspace(*b[1:]) for b in blocks),), 0xff, dtype=torch.uint8, device="cuda")
    try:
        def step():
            S.slide_layer_muon_step(st, 0, blocks, grads, S.muon_hparams(), S.hparams(), ws)
        monkeypatch.setenv("SLIDE_TEST_PIPELINE_STALL", "first")
        step()
        assert S.slide_ortho_status(ws) == S.SLIDE_ERR_TIMEOUT
        assert S.slide_layer_status(st, 0) == S.SLIDE_ERR_TIMEOUT
        monkeypatch.delenv("SLIDE_TEST_PIPELINE_STALL")
        step()
        assert S.slide_ortho_status(ws) == S.SLIDE_OK and S.slide_layer_status(st, 0) == S.SLIDE_OK
        step()
        step()
        assert S.slide_ortho_status(ws) == S.SLIDE_OK and S.slide_layer_status(st, 0) == S.SLIDE_OK
    finally:
        S.slide_state_destroy(st)


def test_status_after_calls_with_nothing_to_do(S):
    """Not what the workspace's memory held before."""
    def fresh():
        return torch.full((4096,), 0xff, dtype=torch.uint8, device="cuda")
    ws = fresh()
    S.slide_orthogonalize(0, 8, 8, None, None, S.ortho_params(), ws)
    assert S.slide_ortho_status(ws) == S.SLIDE_OK
    ws, side = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    S.slide_muon_step(1, 0, 8, [None], None, None, None, S.muon_hparams(), ws, stream=side)
    assert S.slide_ortho_status(ws, side) == S.SLIDE_OK
    st = S.slide_state_create([64], 1)
    try:
        g = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
        for blocks in ((), ((0, 0, 8, 8),)):
            ws = fresh()
            S.slide_layer_muon_step(st, 0, blocks, [g], S.muon_hparams(), S.hparams(), ws)
            assert S.slide_ortho_status(ws) == S.SLIDE_OK
            S.slide_layer_muon_step(st, 0, blocks, [g], S.muon_hparams(), S.hparams(), None)
    finally:
        S.slide_state_destroy(st)


@pytest.mark.parametrize("batch,rows,cols,gap", [(3, 50, 200, 0), (3, 50, 203, 5), (2, 300, 333, 3), (4, 333, 300, 0), (2, 1, 5, 1)])
def test_matrices_beside_one_another(S, batch, rows, cols, gap):
    """[rows, batch, cols]: the matrices' rows take turns, in x and in the result."""
    lead = batch * (cols + gap) + 2
    big = torch.zeros(rows, lead, device="cuda")
    x = big.as_strided((batch, rows, cols), (cols + gap, lead, 1))
    x.copy_(matrix(batch, rows, cols, 3))
    out = torch.full((rows, lead), -7.0, dtype=torch.bfloat16, device="cuda")
    S.slide_orthogonalize(batch, rows, cols, big, out, S.ortho_params(), workspace(S, batch, rows, cols),
                          x_type=S.SLIDE_TYPE_FP32, x_row_stride=lead, x_batch_stride=cols + gap, out_row_stride=lead,
                          out_batch_stride=cols + gap)
    got = out.as_strided((batch, rows, cols), (cols + gap, lead, 1))
    assert off(got, factor64(x)) <= FACTOR + BF16
    keep = torch.ones_like(out, dtype=torch.bool)
    keep.as_strided((batch, rows, cols), (cols + gap, lead, 1)).fill_(False)
    assert (out[keep] == -7.0).all()
    with pytest.raises(S.SlideError):                          # one value less, and they meet
        S.slide_orthogonalize(batch, rows, cols, big, out, S.ortho_params(), workspace(S, batch, rows, cols),
                              x_type=S.SLIDE_TYPE_FP32, x_row_stride=lead, x_batch_stride=cols, out_row_stride=lead,
                              out_batch_stride=cols - 1)
