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
