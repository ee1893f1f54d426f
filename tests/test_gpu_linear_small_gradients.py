"""The linear layer's backward pass on float16 gradients at the ends of float16's range.

dp = dy act'(p) is rounded to float16 scaled to its range, so by 2^-11 of itself (or 2^-39 of the largest of dy), and so is the result, or by
2^-25, half of the smallest number: in L2 over N of them sqrt(N) 2^-25 at most.  The activations add 2^-19, the sums 2^-15 of themselves.
"""
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu


def data(tokens, width, out, seed=1):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    return randn(tokens, width).half(), (randn(out, width) * width ** -0.5).half(), randn(tokens, out)


def gradients(x, w, dy, act):
    p = (x.double() @ w.double().t()).requires_grad_()
    f = torch.nn.functional
    y = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](p)
    dp, = torch.autograd.grad(y, p, dy.double())
    return dp @ w.double(), dp.t() @ x.double(), dp.sum(0)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("scale", [1.0, 1e-4, 2e-6, 3e-7])
@pytest.mark.parametrize("tokens,width,out", [(16_384, 512, 512), (5000, 1001, 903), (300, 64, 72)])
def test_small_gradients(tokens, width, out, scale, act):
    x, w, dy = data(tokens, width, out)
    dy = (dy * scale).half()
    _, saved = sla.sla_linear(x, w, activation=act, save=True)
    got = sla.sla_linear_backward(dy, x, w, saved, activation=act, want_grad_bias=True)
    sla.sla_gated_ffn_check()
    for g, want in zip(got, gradients(x, w, dy, act)):
        n = float(want.norm())
        allowed = (2 * 2.0 ** -11 + 2.0 ** -15 + 2.0 ** -19) * n + 2.0 ** -25 * want.numel() ** 0.5
        assert float((g.double() - want).norm()) <= allowed, (float((g.double() - want).norm()), allowed, n)


def test_gradients_beyond_the_largest_float16():
    """act' may be more than one: dy act'(p) beyond 65504 in sums that come out below it."""
    tokens, width, out = 2048, 1024, 1032
    x, w, dy = data(tokens, width, out)
    w = (w.float() * 2.0 ** -9).half()  # sums of a thousand gradients of 64,000 have to end below 65504
    x = torch.full_like(x, 2.0)
    w[:, 0] = 0.75  # p = 1.5 and a little, where act' is 1.1
    dy = (torch.sign(dy) * 64_000).half()
    _, saved = sla.sla_linear(x, w, activation="gelu", save=True)
    dx, _, _ = sla.sla_linear_backward(dy, x, w, saved, activation="gelu", want_grad_weight=False)
    want, _, _ = gradients(x, w, dy, "gelu")
    assert float(want[:, 1:].abs().max()) < 65504
    assert bool(torch.isfinite(dx[:, 1:]).all())
    assert float((dx[:, 1:].double() - want[:, 1:]).norm()) <= 2.0 ** -10 * float(want[:, 1:].norm())


def test_an_infinite_gradient_stays_one():
    x, w, dy = data(64, 128, 96)
    dy = dy.half()
    dy[7, 5], dy[9, 5] = float("inf"), float("nan")
    _, saved = sla.sla_linear(x, w, activation="silu", save=True)
    dx, _, _ = sla.sla_linear_backward(dy, x, w, saved, activation="silu", want_grad_weight=False)
    bad = torch.zeros(64, dtype=torch.bool, device=DEV)
    bad[7] = bad[9] = True
    assert not bool(torch.isfinite(dx[bad]).any()) and bool(torch.isfinite(dx[~bad]).all())
