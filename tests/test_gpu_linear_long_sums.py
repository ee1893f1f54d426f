"""The linear layer's long sums on the GPU.

A tensor core drops up to a unit 2^-23 of its running sum for every 16 products, half of it on average and 2/3 of that over a sum
that grows as its root: K / 16 * 2^-24 * 2/3 of the sum for K products, always towards zero.  With sums of 2^14 products at most,
whose parts are added in float32 (2^-22), dW may be smaller than it is by 4.1e-5 of itself, however many tokens there are.  The rounding of the
result to its type averages out of that: over N elements it leaves U / sqrt(3 N), below 1e-6 from 2^20 elements on.  Sums over a row have
2^16 products at most.
"""
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

DROPPED = 2 ** 14 / 16 * 2.0 ** -24 * 2 / 3


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,width,out", [(250_003, 2048, 2048), (100_000, 1000, 1500)])
def test_gradient_of_the_weight_over_many_tokens(tokens, width, out, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    x = torch.randn(tokens, width, generator=gen, device=DEV).to(dtype)
    dy = torch.randn(tokens, out, generator=gen, device=DEV).to(dtype)
    w = torch.randn(out, width, generator=gen, device=DEV).to(dtype)
    _, saved = sla.sla_linear(x, w, save=True)
    _, dw, _ = sla.sla_linear_backward(dy, x, w, saved, want_grad_x=False)
    sla.sla_gated_ffn_check()
    ref = torch.zeros(out, width, dtype=torch.float64, device=DEV)
    for i in range(0, tokens, 20_000):
        ref += dy[i:i + 20_000].double().t() @ x[i:i + 20_000].double()
    err = dw.double() - ref
    along = float((err * ref).sum() / (ref * ref).sum())
    assert abs(along) <= DROPPED + 2.0 ** -22 + 1e-6, along
    rounding = float((ref.to(dtype).double() - ref).norm())
    assert float(err.norm()) <= rounding + 2 * (DROPPED + 2.0 ** -22) * float(ref.norm())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("width,out", [(40_000, 33_000), (140_001, 203), (200, 140_000)])
def test_results_over_wide_rows(width, out, dtype):
    """y and dx, whose sums run over the width and the outputs; y with bias, activation and residual behind a sum in parts."""
    tokens = 70
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    x, w, b, r, dy = randn(tokens, width), randn(out, width, scale=width ** -0.5), randn(out), randn(tokens, out), randn(tokens, out)
    y = sla.sla_linear(x, w, b, r, activation="relu")
    _, saved = sla.sla_linear(x, w, save=True)
    dx, _, _ = sla.sla_linear_backward(dy, x, w, saved, want_grad_weight=False)
    sla.sla_gated_ffn_check()
    p = torch.cat([x.double() @ w[i:i + 4000].double().t() for i in range(0, out, 4000)], 1) + b.double()
    ref = sum(dy[:, i:i + 4000].double() @ w[i:i + 4000].double() for i in range(0, out, 4000))
    u = torch.finfo(dtype).eps / 2
    # the result's rounding and what the sums drop (p is no larger than twice y)
    for got, want, products in ((y, torch.relu(p) + r.double(), width), (dx, ref, out)):
        dropped = DROPPED * min(products, 2 ** 16) / 2 ** 14
        assert float((got.double() - want).norm()) <= (u + 2 * (dropped + 2.0 ** -22)) * float(want.norm())
