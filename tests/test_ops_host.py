"""Refusals of the matrix-optimizer and routing entry points: every bad
argument is named before anything touches a device."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


P = 1 << 20          # an aligned address that is never followed


def refused(S, text, call, *a, **k):
    with pytest.raises(S.SlideError) as e:
        call(*a, **k)
    assert e.value.status == S.SLIDE_ERR_INVALID_ARG and text in str(e.value), str(e.value)


def test_ortho_workspace(S):
    w = S.slide_ortho_workspace
    assert w(0, 5, 5) == w(3, 0, 5) == w(3, 5, 0) == 256
    # an m x n matrix: its iterate in two FP16 halves, its second copy or a Muon step's FP32 update, and m x m operands
    assert 8 * 512 * 512 + 6 * 512 * 512 <= w(1, 512, 512) <= 8 * 512 * 512 + 6 * 512 * 512 + (64 << 10)
    assert w(4, 512, 2048) > 3.9 * w(1, 512, 2048)
    for bad in ((-1, 4, 4), (65536, 4, 4), (1, -1, 4), (1, 4, (1 << 20) + 1), (1, 16385, 16385)):
        with pytest.raises(S.SlideError):
            w(*bad)


def test_ortho_refusals(S):
    big = 1 << 40

    def call(batch=1, rows=4, cols=8, x=P, out=2 * P, params=None, ws=4 * P, n=big, **k):
        S.slide_orthogonalize(batch, rows, cols, x, out, params or S.ortho_params(), ws, workspace_bytes=n, **k)
    refused(S, "batch", call, batch=-1)
    refused(S, "16384", call, rows=20000, cols=20000)
    refused(S, "x_type", call, x_type=2)
    refused(S, "steps", call, params=S.ortho_params(steps=0))
    refused(S, "steps", call, params=S.ortho_params(steps=17))
    refused(S, "eps", call, params=S.ortho_params(eps=-1.0))
    refused(S, "eps", call, params=S.ortho_params(eps=float("nan")))
    refused(S, "non-finite", call, params=S.ortho_params(steps=1, coeffs=[(float("inf"), 0, 0)]))
    refused(S, "grows", call, params=S.ortho_params(steps=5, coeffs=[(100.0, 0, 0)] * 5))
    refused(S, "NULL", call, x=None)
    refused(S, "NULL", call, out=None)
    refused(S, "aligned", call, x=P + 1)
    refused(S, "row stride", call, x_row_stride=7)
    refused(S, "row stride", call, out_row_stride=7)
    refused(S, "overlap", call, batch=2, out_batch_stride=31)
    refused(S, "workspace", call, ws=None, n=big)
    refused(S, "256-byte", call, ws=4 * P + 16)
    refused(S, "smaller", call, n=S.slide_ortho_workspace(1, 4, 8) - 1)
    call(batch=0, x=None, out=None, ws=None, n=0)               # nothing to do
    call(rows=0, x=None, out=None, ws=None, n=0)


def test_muon_refusals(S):
    def call(batch=1, rows=4, cols=8, grads=(P,), th=P, mom=P, w=P, hp=None, ws=4 * P, n=1 << 40, **k):
        S.slide_muon_step(batch, rows, cols, list(grads), th, mom, w, hp or S.muon_hparams(), ws, workspace_bytes=n, **k)
    refused(S, "n_replicas", call, grads=())
    refused(S, "n_replicas", call, grads=(P,) * 9)
    refused(S, "grads_type", call, grads_type=7)
    refused(S, "replica", call, grads=(P, None))
    refused(S, "replica", call, grads=(P + 8,))
    refused(S, "master", call, th=None)
    refused(S, "master", call, mom=P + 4)
    refused(S, "master", call, w=P + 2)
    refused(S, "lr", call, hp=S.muon_hparams(lr=-1.0))
    refused(S, "momentum", call, hp=S.muon_hparams(momentum=1.0))
    refused(S, "non-finite", call, hp=S.muon_hparams(scale=float("inf")))
    refused(S, "steps", call, hp=S.muon_hparams(steps=0))
    refused(S, "workspace", call, ws=None)
    refused(S, "smaller", call, n=100)
    call(batch=0, th=None, mom=None, w=None, ws=None, n=0)


def test_route_refusals(S):
    def call(tokens=4, cfg=None, x=P, w=P, e=P, **k):
        S.slide_route_experts(tokens, x, w, e, cfg or S.route_config(64, 4), **k)

    def back(tokens=4, cfg=None, x=P, e=P, dw=P, dx=2 * P, **k):
        S.slide_route_experts_backward(tokens, x, e, dw, dx, cfg or S.route_config(64, 4), **k)
    for f in (call, back):
        refused(S, "tokens", f, tokens=-1)
        refused(S, "logits_type", f, logits_type=3)
        refused(S, "n_experts", f, cfg=S.route_config(0, 1))
        refused(S, "n_experts", f, cfg=S.route_config(1025, 1))
        refused(S, "score", f, cfg=S.route_config(64, 4, score=2))
        refused(S, "group_score", f, cfg=S.route_config(64, 4, group_score=2))
        refused(S, "n_groups", f, cfg=S.route_config(64, 4, n_groups=7))
        refused(S, "n_groups", f, cfg=S.route_config(64, 4, n_groups=0))
        refused(S, "top_groups", f, cfg=S.route_config(64, 4, n_groups=8, top_groups=9))
        refused(S, "top_k", f, cfg=S.route_config(64, 0))
        refused(S, "top_k", f, cfg=S.route_config(64, 33))
        refused(S, "top_k", f, cfg=S.route_config(64, 9, n_groups=8, top_groups=1))
        refused(S, "scale", f, cfg=S.route_config(64, 4, scale=float("nan")))
        refused(S, "stride", f, logits_stride=63)
        refused(S, "NULL", f, x=None)
        refused(S, "aligned", f, x=P + 2)
        refused(S, "NULL", f, e=None)
        f(tokens=0, x=None, e=None)                              # nothing to do
    refused(S, "NULL", call, w=None)
    refused(S, "load", call, load=P + 4)
    refused(S, "bias", call, bias=P + 2)
    refused(S, "stride", back, d_logits_stride=10)
    refused(S, "d_weights", back, dw=None)
    refused(S, "d_logits", back, dx=None)
    refused(S, "must not", back, dx=P)
    refused(S, "n_experts", S.slide_route_bias_step, 0, P, P, 0.1)
    refused(S, "load", S.slide_route_bias_step, 8, None, P, 0.1)
    refused(S, "load", S.slide_route_bias_step, 8, P, P + 2, 0.1)
    refused(S, "rate", S.slide_route_bias_step, 8, P, P, -0.1)
    refused(S, "rate", S.slide_route_bias_step, 8, P, P, float("inf"))


def test_null_structs(S):
    L = S.lib
    assert L.slide_orthogonalize(1, 4, 8, P, 0, 8, 32, P, 8, 32, None, P, 1 << 40, None) == S.SLIDE_ERR_INVALID_ARG
    assert L.slide_muon_step(1, 4, 8, 1, (C.c_void_p * 1)(P), 0, P, P, P, None, P, 1 << 40, None) == S.SLIDE_ERR_INVALID_ARG
    assert L.slide_route_experts(1, P, 1, 64, None, None, None, P, P, None, None) == S.SLIDE_ERR_INVALID_ARG
    assert L.slide_ortho_workspace(1, 4, 4, None) == S.SLIDE_ERR_INVALID_ARG
    assert L.slide_ortho_status(None, None) == S.SLIDE_ERR_INVALID_ARG


@pytest.mark.gpu
def test_layer_muon_refusals(S):
    import torch
    n = 4096
    st = S.slide_state_create([n], 1)
    ws = torch.empty(S.slide_ortho_workspace(1, 32, 64), dtype=torch.uint8, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    try:
        def call(blocks, adam=None, muon=None, grads=None, w=ws, **k):
            S.slide_layer_muon_step(st, k.pop("layer", 0), blocks, grads or [g], muon or S.muon_hparams(),
                                    adam or S.hparams(), w, **k)
        refused(S, "layer", call, [], layer=1)
        refused(S, "blocks", call, [(4, 1, 8, 8)])
        refused(S, "blocks", call, [(0, 1, 8, 8), (32, 1, 8, 8)])
        refused(S, "blocks", call, [(4032, 1, 8, 16)])
        refused(S, "multiple of 8", call, [(0, 1, 3, 3)])
        refused(S, "multiple of 8", call, [(0, 1, 3, 3), (16, 1, 8, 8)])
        refused(S, "clip", call, [(0, 1, 8, 8)], adam=S.hparams(max_grad_norm=1.0))
        refused(S, "lr", call, [(0, 1, 8, 8)], muon=S.muon_hparams(lr=-1.0))
        refused(S, "workspace", call, [(0, 1, 64, 64)], w=ws[:256])
        refused(S, "replica", call, [(0, 1, 8, 8)], grads=[None])
        assert S.slide_layer_get(st, 0) == 0                     # nothing was applied
        call([(0, 1, 32, 64), (2048, 1, 32, 64)])
        assert S.slide_layer_get(st, 0) == 1
    finally:
        S.slide_state_destroy(st)
    st = S.slide_state_create([64], 1, flags=S.SLIDE_FLAG_CHECK_FINITE)
    try:
        with pytest.raises(S.SlideError) as e:
            S.slide_layer_muon_step(st, 0, [(0, 1, 8, 8)], [g], S.muon_hparams(), S.hparams(), ws)
        assert e.value.status == S.SLIDE_ERR_STATE
    finally:
        S.slide_state_destroy(st)


def test_calls_let_other_threads_run(S):
    """A launch can block; the interpreter's lock is not held meanwhile."""
    import threading
    import time

    from mixed_precision_adam_grad_gb300 import _binding
    fast = _binding._fast()
    own = C.cast(S.lib.slide_route_bias_step, C.c_void_p).value
    usleep = C.CDLL(None).usleep                                 # takes the first argument: a call of 0.4 s
    runs, stop = [0], threading.Event()

    def count():
        while not stop.is_set():
            runs[0] += 1
            time.sleep(0.001)
    t = threading.Thread(target=count)
    fast.bind("slide_route_bias_step", C.cast(usleep, C.c_void_p).value)
    try:
        t.start()
        time.sleep(0.05)
        before = runs[0]
        fast.route_bias_step(400000, None, None, 0.0, None)
        during = runs[0] - before
    finally:
        fast.bind("slide_route_bias_step", own)
        stop.set()
        t.join()
    assert during >= 20


def test_layer_muon_step_of_too_few_replicas(S):
    """Refused before the library reads past the addresses that it was given."""
    st = S.SlideState(0, [64], 2, S.SLIDE_RESIDENCY_HBM)
    for grads in ([], [P]):
        refused(S, "replicas", S.slide_layer_muon_step, st, 0, [(0, 1, 8, 8)], grads, S.muon_hparams(), S.hparams(), 4 * P,
                workspace_bytes=1 << 40)
    refused(S, "state is NULL", S.slide_layer_muon_step, st, 0, [(0, 1, 8, 8)], [P, P], S.muon_hparams(), S.hparams(), 4 * P,
            workspace_bytes=1 << 40)
