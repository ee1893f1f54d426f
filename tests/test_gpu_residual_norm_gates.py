"""Gates of the residual norm at the ends of their range, against the definitions in 64 bits.

With z = 0, a block of ones, no norms and no scale, z' is act(gate) and, for dz' = 1, dgate is act'(gate).  The exponential and the
reciprocal are approximate (2^-22 and 2^-23), the exponent's rounding is |g| 2^-23 while the exponential is neither zero nor infinite
(|g| < 128), and the sums and products round a few times: 2^-20 + 128 2^-23 in all, and the result its type's half step.  silu's derivative
is a sum that passes zero near -1.28: relative to its parts, of at most one there.  What is smaller than 2^-126 may be zero: a gate times that, 2^-119.
"""
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

GATES = [0.0, -0.0, 1.0, -1.0, 5.0, -5.0, 20.0, -20.0, 60.0, -60.0, 86.0, -86.0, 87.0, -87.0, 88.0, -88.0, 90.0, -90.0, 120.0, -120.0,
         1e4, -1e4, 6e4, -6e4, 1e10, -1e10, 1e30, -1e30, 1e32, -1e32, 1e38, -1e38, 3e38, -3e38]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("width", [64, 1001, 9000])
def test_gates_at_their_ends(width, act, dtype):
    gates = [v for v in GATES if abs(v) <= torch.finfo(dtype).max]
    g = torch.tensor(gates, device=DEV).repeat(5 * width // len(gates) + 1)[:5 * width].view(5, width).to(dtype)
    ones, zeros = torch.ones_like(g), torch.zeros_like(g)
    how = dict(post_norm=False, gate_activation=act)
    z, _, stats = sla.sla_residual_norm(ones, zeros, g, next_norm=False, stats=True, **how)
    grads = sla.sla_residual_norm_backward(ones, None, ones, zeros, stats, g, want_grad_params=False, **how)
    g64 = g.double()
    s, r = torch.sigmoid(g64), torch.sigmoid(-g64)
    want = s if act == "sigmoid" else g64 * s
    slope = s * r if act == "sigmoid" else s + g64 * s * r
    u = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -119
    rel = 2.0 ** -20 + 128 * 2.0 ** -23
    assert bool((((z.double() - want).abs()) <= (rel + u) * want.abs() + tiny).all())
    parts = slope if act == "sigmoid" else s + (g64 * s * r).abs()
    assert bool(((grads.gate.double() - slope).abs() <= rel * parts + u * slope.abs() + tiny).all())
    assert bool(((grads.block.double() - want).abs() <= (rel + u) * want.abs() + tiny).all())
