"""The ways in which slide_orthogonalize and slide_muon_step compute, each at
shapes that choose it: pairs of CTAs and single ones, groups of steps and step by
step, K split, narrow tiles, and the kernels for a small side with long other
sides, whose buffers are used several times.  The shapes are for 152 SMs; that
each still chooses its way is asserted, so that another rule cannot leave a way
untested.  Formulas and tolerances are test_gpu_ortho's.
"""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_ortho import (BF16, FACTOR, S, check_muon, factor64, gen, matrix, muon64, off, orthogonalize,  # noqa: E402, F401
                            workspace)

SMALL, GROUPS, PAIRS, SPLIT, NARROW = 1, 2, 4, 8, 16


def form(S, batch, rows, cols, muon=False, params=None):
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the shapes are for 152 SMs")
    f = S.lib.slide_test_ortho_form
    f.argtypes = [C.c_int32] * 4 + [C.c_void_p]
    p = params or S.ortho_params()
    return f(batch, rows, cols, int(muon), C.addressof(p))


FORMS = [(40, 1000, 1400, PAIRS | GROUPS), (1, 2300, 3301, PAIRS | GROUPS), (1, 3301, 2300, PAIRS | GROUPS),
         (1, 1537, 1536, PAIRS), (1, 2049, 2050, PAIRS), (3, 1500, 1501, PAIRS), (2, 1024, 2560, GROUPS | SPLIT),
         (1, 300, 8000, GROUPS | SPLIT | NARROW), (1, 8000, 300, GROUPS | SPLIT | NARROW), (2, 238, 14962, GROUPS | SPLIT | NARROW),
         (1, 200, 1600, SPLIT | NARROW), (1, 400, 401, NARROW), (5, 320, 320, NARROW), (20, 500, 700, PAIRS), (12, 320, 320, 0),
         (24, 64, 9001, SMALL), (20, 7000, 100, SMALL), (1, 33, 50001, SMALL), (3, 20011, 128, SMALL), (200, 16, 1000, SMALL)]


@pytest.mark.parametrize("batch,rows,cols,want", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_factor_of_each_form(S, batch, rows, cols, want, dtype):
    assert form(S, batch, rows, cols) == want
    x = matrix(batch, rows, cols, rows + cols).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert off(orthogonalize(S, x), factor64(x)) <= FACTOR + BF16


@pytest.mark.parametrize("batch,rows,cols,want", [f for f in FORMS if f[0] * f[1] * f[2] < 3e7])
@pytest.mark.parametrize("dtype,R", [("bf16", 3), ("fp32", 2)])
def test_muon_step_of_each_form(S, batch, rows, cols, want, dtype, R):
    assert form(S, batch, rows, cols, muon=True) == want
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    common, g = matrix(batch, rows, cols, 1), gen(2)
    grads = [(common + torch.randn(common.shape, generator=g, device="cuda") * 1e-3).to(dt) for _ in range(R)]
    mom, th = matrix(batch, rows, cols, 3), torch.randn(common.shape, generator=g, device="cuda") * 0.02
    want64, th0, w = muon64(grads, mom, th, 0.01, 0.9, 0.1, 0.5, True), th.clone(), torch.empty(th.shape, dtype=torch.bfloat16, device="cuda")
    S.slide_muon_step(batch, rows, cols, grads, th, mom, w, S.muon_hparams(lr=0.01, momentum=0.9, weight_decay=0.1, scale=0.5),
                      workspace(S, batch, rows, cols), grads_type=S.SLIDE_TYPE_FP32 if dtype == "fp32" else S.SLIDE_TYPE_BF16)
    torch.cuda.synchronize()
    check_muon(S, th, mom, w, want64, 0.01, 0.5, th0)


@pytest.mark.parametrize("batch,rows,cols,steps,want", [
    (1, 300, 4000, k, GROUPS | SPLIT | NARROW if k > 1 else SPLIT | NARROW) for k in (1, 2, 3, 4, 6)] + [
    (1, 3000, 600, k, GROUPS | SPLIT if k > 1 else SPLIT) for k in (1, 2, 3, 4, 7)] + [
    (1, 2300, 3301, k, PAIRS | GROUPS if k > 1 else PAIRS) for k in (1, 3, 4, 6)] + [
    (6, 100, 1500, k, SMALL) for k in (1, 2, 4, 6)])
def test_numbers_of_steps(S, batch, rows, cols, steps, want):
    p = S.ortho_params(steps=steps)
    assert form(S, batch, rows, cols, params=p) & ~(SPLIT | NARROW) == want & ~(SPLIT | NARROW)
    x = matrix(batch, rows, cols, steps)
    assert off(orthogonalize(S, x, p), factor64(x, steps)) <= FACTOR + BF16


@pytest.mark.parametrize("batch,rows,cols,want", [(5, 1000, 2400, PAIRS | GROUPS), (3, 1500, 1501, PAIRS), (4, 300, 8000, GROUPS),
                                                  (30, 64, 3000, SMALL)])
def test_a_nan_stays_in_its_matrix(S, batch, rows, cols, want):
    assert form(S, batch, rows, cols) & (PAIRS | GROUPS | SMALL) == want
    x = matrix(batch, rows, cols, 7)
    first = orthogonalize(S, x)
    x[1, rows - 1, cols - 1] = float("nan")
    got = orthogonalize(S, x)
    assert torch.isnan(got[1]).all()
    keep = [k for k in range(batch) if k != 1]
    assert torch.equal(got[keep], first[keep])


@pytest.mark.parametrize("rows,cols,dtype,lead,first", [
    (50, 203, "fp32", 206, 1), (50, 203, "bf16", 206, 1), (50, 200, "bf16", 204, 4), (120, 1000, "bf16", 1004, 0),
    (1003, 100, "bf16", 108, 4), (1003, 100, "bf16", 101, 0), (2000, 50, "fp32", 56, 4), (64, 3000, "bf16", 3008, 8)])
def test_strides_of_a_small_side(S, rows, cols, dtype, lead, first):
    """Rows apart, unaligned, aligned to 8 and to 16 bytes; a repeated matrix; only the result's places are written."""
    b, r = 3, rows + 3
    dt, kind = (torch.float32, S.SLIDE_TYPE_FP32) if dtype == "fp32" else (torch.bfloat16, S.SLIDE_TYPE_BF16)
    big = matrix(b, r, lead, 4).to(dt).flatten()
    x = big.as_strided((b, rows, cols), (r * lead, lead, 1), first)
    out = torch.full((b, rows + 2, cols + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(S, b, rows, cols)
    assert form(S, b, rows, cols) == SMALL
    S.slide_orthogonalize(b, rows, cols, x, out[:, :, 3:], S.ortho_params(), ws, x_type=kind, x_row_stride=lead,
                          x_batch_stride=r * lead, out_row_stride=cols + 8, out_batch_stride=(rows + 2) * (cols + 8))
    assert off(out[:, :rows, 3:3 + cols], factor64(x)) <= FACTOR + BF16
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[:, :rows, 3:3 + cols] = False
    assert (out[mask] == -7.0).all()
    rep = torch.empty(b, rows, cols, dtype=torch.bfloat16, device="cuda")
    S.slide_orthogonalize(b, rows, cols, x, rep, S.ortho_params(), ws, x_type=kind, x_row_stride=lead, x_batch_stride=0)
    assert torch.equal(rep[0], rep[1]) and torch.equal(rep[0], rep[2])
    assert off(rep[:1], factor64(x[:1])) <= FACTOR + BF16


@pytest.mark.parametrize("rows,cols,want", [(2300, 3301, PAIRS | GROUPS), (1537, 1536, PAIRS)])
def test_a_wait_of_a_pair_that_runs_out_is_reported(S, monkeypatch, rows, cols, want):
    assert form(S, 1, rows, cols) == want
    x = matrix(1, rows, cols, 1)
    out, ws = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"), workspace(S, 1, rows, cols)
    monkeypatch.setenv("SLIDE_TEST_PIPELINE_STALL", "1")
    S.slide_orthogonalize(1, rows, cols, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32)
    assert S.slide_ortho_status(ws) == S.SLIDE_ERR_TIMEOUT
    monkeypatch.delenv("SLIDE_TEST_PIPELINE_STALL")
    S.slide_orthogonalize(1, rows, cols, x, out, S.ortho_params(), ws, x_type=S.SLIDE_TYPE_FP32)
    assert S.slide_ortho_status(ws) == S.SLIDE_OK
    assert off(out, factor64(x)) <= FACTOR + BF16


@pytest.mark.parametrize("batch,rows,cols,steps,want", [(1, 2300, 3301, 5, PAIRS | GROUPS), (1, 1537, 1536, 5, PAIRS),
                                                        (1, 300, 8000, 5, GROUPS), (2, 700, 300, 16, 0), (6, 100, 1500, 5, SMALL)])
def test_each_form_in_a_graph(S, batch, rows, cols, steps, want):
    """Sixteen steps step by step take two launches with a clearing between them."""
    coeffs = [(3.4445, -4.7750, 2.0315)] * 5 + [(1.875, -1.25, 0.375)] * (steps - 5)
    p = S.ortho_params(steps=steps, coeffs=coeffs)
    assert form(S, batch, rows, cols, params=p) & (PAIRS | GROUPS | SMALL) == want
    x = matrix(batch, rows, cols, 2)
    out, ws = torch.zeros(batch, rows, cols, dtype=torch.bfloat16, device="cuda"), workspace(S, batch, rows, cols)

    def call():
        S.slide_orthogonalize(batch, rows, cols, x, out, p, ws, x_type=S.SLIDE_TYPE_FP32, stream=torch.cuda.current_stream())
    call()
    first = out.clone()
    assert off(first, factor64(x, steps, coeffs)) <= FACTOR + BF16
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for sign in (-1, 1):
        x.mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sign * first)
    assert S.slide_ortho_status(ws) == S.SLIDE_OK
