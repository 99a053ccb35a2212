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


def place(rows, cols, stride, shift, dt, seed):
    """rows x cols values, rows `stride` apart, `shift` elements off an aligned address."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shift + rows * stride, generator=g, device="cuda").to(dt)[shift:].view(rows, stride)[:, :cols]


# contiguous odd rows, padded odd rows, rows off an aligned address, strides that differ modulo eight between the pairs
LAYOUTS = [(513, 0, 0, 0), (1601, 0, 0, 0), (4099, 0, 0, 0), (1000, 7, 0, 0), (77, 0, 0, 3), (520, 0, 1, 1), (1601, 0, 4, 0), (2048, 8, 8, 0)]


@pytest.mark.parametrize("cols,pad,more,shift", LAYOUTS)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [5, 700])
def test_in_place_at_any_width(S, rows, cols, pad, more, shift, kind):
    """out over x and sum over residual, and the other way round; d_x over d_out and d_residual over d_sum, and the
    other way round: what separate results of the same layouts hold, bit for bit, and nothing between the rows."""
    dt = TYPES[kind]
    cfg, drop, s = config(S, True, dt), S.dropout_config(0.2, 3, first=5), torch.cuda.current_stream()
    one, two = cols + pad, cols + pad + more                     # strides of x and d_out, of residual and d_sum

    def tensors():
        return [place(rows, cols, one, shift, dt, 1), place(rows, cols, two, shift, dt, 2), place(rows, cols, one, shift, dt, 3),
                place(rows, cols, two, shift, dt, 4)]
    w = place(1, cols, cols, 0, dt, 5)[0].clone()
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def forward(x, res, total, out):
        S.slide_norm(rows, cols, x, w, out, cfg, residual=res, dropout=drop, sum=total, mean=mean, rstd=rstd, x_stride=x.stride(0),
                     residual_stride=res.stride(0), sum_stride=total.stride(0), out_stride=out.stride(0), stream=s)

    def backward(d, ds, dx, dr):
        S.slide_norm_backward(rows, cols, normed, w, d, dx, cfg, rstd, mean=mean, d_sum=ds, dropout=drop, d_residual=dr,
                              x_stride=normed.stride(0), d_out_stride=d.stride(0), d_sum_stride=ds.stride(0), d_x_stride=dx.stride(0),
                              d_residual_stride=dr.stride(0), stream=s)

    def gaps(t):
        whole = torch.as_strided(t, (rows, t.stride(0)), (t.stride(0), 1), t.storage_offset())
        return whole[:, cols:].clone()
    normed = place(rows, cols, one, shift, dt, 6)
    for call in (forward, backward):
        for swapped in (False, True):
            def results(t, k):                                   # forward: sum, out; backward: d_x, d_residual
                return (t[k], t[k + 1]) if swapped == (call is forward) else (t[k + 1], t[k])
            t, u = tensors(), tensors()
            call(t[0], t[1], *results(t, 2))                     # beside the inputs
            left = [gaps(v) for v in u[:2]]
            call(u[0], u[1], *results(u, 0))                     # over them
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(results(u, 0), results(t, 2))), (call.__name__, swapped)
            assert all(torch.equal(gaps(v), k) for v, k in zip(u[:2], left))
