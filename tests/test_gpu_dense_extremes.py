"""Values at the ends of their types' ranges in the dense operators: where the formula is finite (or infinite), so is the result."""
import pytest

from gpu_helpers import sla, torch, DEV
from test_gpu_dense import randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [12, 40, 20001])
@pytest.mark.parametrize("hidden", [40, 64, 100])
def test_infinity_in_x_is_an_infinity_in_y(hidden, tokens, dtype):
    # all factors positive: g, u, h and y of the row are +inf; hidden units that pad a tile must not make it NaN
    x = randn(tokens, 48, dtype=dtype, seed=210).abs()
    w_in, w_out = (randn(*s, dtype=dtype, seed=211).abs() * 0.1 + 0.01 for s in ((2 * hidden, 48), (24, hidden)))
    want = sla.sla_gated_ffn(x, w_in, w_out, activation="relu")
    bad = tokens // 2
    x[bad, 5] = float("inf")
    keep = torch.arange(tokens, device=DEV) != bad
    for y in (sla.sla_gated_ffn(x, w_in, w_out, activation="relu"),
              sla.sla_gated_ffn(x, w_in, w_out, activation="relu", save=True)[0]):
        assert torch.isposinf(y[bad]).all()
        assert torch.isfinite(y[keep]).all()
    assert torch.equal(sla.sla_gated_ffn(x, w_in, w_out, activation="relu")[keep], want[keep])


@pytest.mark.parametrize("width", [64, 96, 100, 200])
def test_layernorm_of_a_constant_row_of_large_values(width):
    # x - mean = 0, rstd = 1 / sqrt(eps): y = b and dx = rstd (dy - mean dy), whatever |mean| rstd is.  Sums of 2^119 over
    # these widths are exact in float32 as long as the width has less than 24 bits, and their mean is 2^119 or its neighbour
    # (no difference is left then, or rstd is 0 and dx = 0: both are finite)
    rows = 3
    x = randn(rows, width, dtype=torch.float32, seed=220)
    x[1] = 2.0 ** 119
    dy, b = randn(rows, width, dtype=torch.float32, seed=221), randn(width, dtype=torch.float32, seed=222)
    eps = 2.0 ** -20  # rstd = 1024: mean times rstd passes the largest float32
    y, mean, rstd = sla.sla_layernorm(x, None, b, eps=eps, stats=True)
    dx, dw, db = sla.sla_layernorm_backward(dy, x, None, mean, rstd)
    assert torch.isfinite(y).all() and torch.isfinite(dx).all() and torch.isfinite(db).all()
    if float(mean[1]) == 2.0 ** 119:
        assert torch.equal(y[1], b)
        d = dy[1].double()
        # two sums of `width` terms and three roundings
        assert float((dx[1].double() - 1024.0 * (d - d.mean())).abs().max()) <= 1024.0 * 96 * 2.0 ** -24 * float(d.abs().max())
