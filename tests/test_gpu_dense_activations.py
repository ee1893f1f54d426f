"""The block's activations and their derivatives, value by value, over the range of a gate.

One hidden unit carries the gate itself (x = [g, 1], g exact, u = 1) and w_out is the identity, so y is act(g), and with
dy = 1 dx is [act'(g), act(g)], each rounded once to the data's type: by at most U of its value.  The float32 work: an
exponential of E (E = |g|, g^2 / 2, or |2z| of the tanh form) whose argument is rounded up to four times, by 2^-24 of E
each: 2^-22 E of the result; exponential, reciprocal and a polynomial of ten steps, each within 2^-22 or 2^-23: 2^-19
in all.  A derivative is a sum of two terms, whose errors count by the terms' own sizes.  float16 also rounds what
falls below its normal range, by up to 2^-25.
"""
import math

import pytest

from gpu_helpers import sla, torch, DEV
from test_gpu_dense import ACTS, TYPES, U

pytestmark = pytest.mark.gpu


def exact(g, act):
    """act(g), act'(g), the sizes of the derivative's terms added up, and E, in 64 bits without cancellation."""
    g = g.double()
    if act == "relu":
        return g.clamp(min=0), (g > 0).double(), (g > 0).double(), torch.zeros_like(g)
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        second = g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        return g * phi, phi + second, phi + second.abs(), 0.5 * g * g
    z = g if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    dz = torch.ones_like(g) if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * g * g)
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    second = g * s * rest * dz
    return g * s, s + second, s + second.abs(), z.abs()


def within(got, ref, size, e, dtype):
    work = (2.0 ** -19 + e * 2.0 ** -22) * size
    rounding = U[dtype] * (1.0 + 2.0 ** -10) * ref.abs() if dtype != torch.float32 else 0.0
    bound = work + rounding + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126)
    return (got.double() - ref).abs() <= bound


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("tokens", [16, 20001])  # few tokens; many: the narrow kernel (16 bits), tiles
def test_activation_and_derivative_of_every_gate(act, tokens, dtype):
    g = torch.linspace(-9.0, 9.0, tokens, device=DEV).to(dtype)
    x = torch.zeros(tokens, 8, dtype=dtype, device=DEV)
    x[:, 0], x[:, 1] = g, 1.0
    w_in = torch.zeros(16, 8, dtype=dtype, device=DEV)
    w_in[0, 0] = w_in[8, 1] = 1.0
    w_out = torch.eye(8, dtype=dtype, device=DEV)
    dy = torch.zeros(tokens, 8, dtype=dtype, device=DEV)
    dy[:, 0] = 1.0
    a, da, size, e = exact(g, act)
    y = sla.sla_gated_ffn(x, w_in, w_out, activation=act)
    y2, saved = sla.sla_gated_ffn(x, w_in, w_out, activation=act, save=True)
    dx = sla.sla_gated_ffn_backward(dy, x, w_in, w_out, saved, activation=act)[0]
    for name, got, ref, s in (("y", y[:, 0], a, a.abs()), ("y, saving", y2[:, 0], a, a.abs()),
                              ("du", dx[:, 1], a, a.abs()), ("dg", dx[:, 0], da, size)):
        bad = ~within(got, ref, s, e, dtype)
        assert not bad.any(), (name, int(bad.sum()), g[bad][:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("tokens", [2, 40])
def test_gates_far_from_zero(act, tokens, dtype):
    # act(g) is g or 0, act'(g) 1 or 0, as long as g^2 is finite
    g = torch.tensor([1e14, -1e14], device=DEV).to(dtype).repeat(tokens // 2)
    x = torch.stack((g, torch.ones_like(g)), 1)
    w_in, w_out = torch.eye(2, dtype=dtype, device=DEV), torch.ones(1, 1, dtype=dtype, device=DEV)
    y, saved = sla.sla_gated_ffn(x, w_in, w_out, activation=act, save=True)
    assert torch.equal(y[:, 0], g.clamp(min=0)) and torch.equal(sla.sla_gated_ffn(x, w_in, w_out, activation=act), y)
    dx = sla.sla_gated_ffn_backward(torch.ones_like(y), x, w_in, w_out, saved, activation=act)[0]
    assert torch.equal(dx[:, 0], (g > 0).to(dtype)) and torch.equal(dx[:, 1], g.clamp(min=0))
