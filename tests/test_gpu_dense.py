"""Layer norm and the gated feed-forward block on the GPU against their definitions in 64 bits.

Tolerances (u = the type's unit roundoff: 2^-24, 2^-11, 2^-8 for float32, float16, bfloat16):
  layer norm, per element: the output's own rounding u |y|, plus the float32 work.  A sum of at most
      64 additions in sequence and a tree errs by less than 96 * 2^-24 of the largest |x| of the row;
      divided by the row's deviation and taken twice (mean and variance) that is FP32_LN * max|x| rstd |w|.
  feed-forward block, relative L2: 16-bit data is rounded at g, u, h, dg, du and the output, each by
      at most u per element and u / 2 on average, with derivatives of the activations below 1.2: 4 u
      (8 u in float16, where small values have fewer bits) covers them all.
      float32 data: a sum of K products in the tensor cores loses at most one unit 2^-23 of the running
      sum for every 16 products, half of it on average, 2/3 of it over a sum that grows as sqrt(k):
      K / 16 * 2^-24 * 2/3 = 5e-6 at K = 2048 (no longer run is taken in one); with the splits' 2^-22: 1e-5.
"""
import math

import numpy as np
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
FP32_LN = 2 * 96 * 2.0 ** -24
FFN_TOL = {torch.float32: 1e-5, torch.float16: 8 * 2.0 ** -11, torch.bfloat16: 8 * 2.0 ** -9}


def randn(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def rel(a, b) -> float:
    a, b = a.double(), b.double()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n > 0 else 1.0)


# ------------------------------------------------------------------ layer norm

def ln64(x, w, b, eps):
    x = x.double()
    mu = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mu) * rstd
    y = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y, xh, rstd, mu


def check_ln(x, w, b, y, eps=1e-5):
    ref, xh, rstd, mu = ln64(x, w, b, eps)
    wmax = 1.0 if w is None else w.double().abs()
    amax = x.double().abs().amax(-1, keepdim=True)
    bound = U[x.dtype] * ref.abs() + FP32_LN * (amax * rstd + xh.abs()) * wmax + 4 * 2.0 ** -24 * ref.abs() + 1e-30
    if x.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half of the smallest subnormal
    excess = (y.double() - ref).abs() - bound
    assert float(excess.max()) <= 0, f"{float(excess.max()):.3e} over the bound"


LN_SHAPES = [(1, 1), (3, 2), (5, 7), (1, 64), (33, 64), (257, 96), (64, 250), (2, 1001), (19, 1024), (5003, 136),
             (300, 256), (7, 4099), (9, 4096), (3, 8200), (2, 40000), (2, 40001), (70000, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", LN_SHAPES)
def test_layernorm_forward(rows, width, dtype):
    x = randn(rows, width, dtype=dtype, seed=1, scale=2.0, shift=0.7)
    for pt in {dtype, torch.float32}:
        w, b = randn(width, dtype=pt, seed=2, scale=0.3, shift=1.0), randn(width, dtype=pt, seed=3)
        y, mean, rstd = sla.sla_layernorm(x, w, b, stats=True)
        check_ln(x, w, b, y)
        _, _, r64, m64 = ln64(x, w, b, 1e-5)
        assert rel(mean[:, None], m64) < 1e-4 and rel(rstd[:, None], r64) < 1e-4
        assert torch.equal(y, sla.layer_norm(x, w, b))
    check_ln(x, None, None, sla.layer_norm(x))
    check_ln(x, w, None, sla.layer_norm(x, w))
    check_ln(x, None, b, sla.layer_norm(x, None, b))


def ln_grads64(x, w, b, dy, eps=1e-5):
    leaves = [t.double().requires_grad_() for t in (x, w, b)]
    y, _, _, _ = ln64(leaves[0], leaves[1], leaves[2], eps)
    return torch.autograd.grad(y, leaves, dy.double())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", LN_SHAPES)
def test_layernorm_backward(rows, width, dtype):
    x = randn(rows, width, dtype=dtype, seed=4, scale=2.0, shift=0.7)
    dy = randn(rows, width, dtype=dtype, seed=5)
    w, b = randn(width, dtype=torch.float32, seed=6, scale=0.3, shift=1.0), randn(width, dtype=torch.float32, seed=7)
    for pt in {dtype, torch.float32}:
        wp, bp = w.to(pt), b.to(pt)
        ref = ln_grads64(x, wp, bp, dy)
        _, mean, rstd = sla.sla_layernorm(x, wp, bp, stats=True)
        got = sla.sla_layernorm_backward(dy, x, wp, mean, rstd)
        assert got[0].dtype == dtype and got[1].dtype == pt and got[2].dtype == pt
        # dx: every term is of the size of max|dxh| max(1, xh^2) rstd; the sums over a row as in the forward pass
        _, xh, r64, _ = ln64(x, wp, bp, 1e-5)
        dxh = (dy.double() * wp.double()).abs().amax(-1, keepdim=True)
        size = r64 * dxh * (1 + xh.abs()) * (1 + xh.abs().amax(-1, keepdim=True))
        amp = 1 + x.double().abs().amax(-1, keepdim=True) * r64
        bound = U[dtype] * ref[0].abs() + FP32_LN * size * amp + 1e-30 + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert float(((got[0].double() - ref[0]).abs() - bound).max()) <= 0
        # sums over the rows: the output's rounding and a float32 sum of `rows` terms of size |dy| (1 + |xh|)
        terms = (dy.double().abs() * (1 + xh.abs()) * amp).sum(0)
        for g, r in ((got[1], ref[1]), (got[2], ref[2])):
            bound = U[pt] * r.abs() + 2 * FP32_LN * terms + (2.0 ** -25 if pt == torch.float16 else 0)
            assert float(((g.double() - r).abs() - bound).max()) <= 0
        again = sla.sla_layernorm_backward(dy, x, wp, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        dx, none_w, db = sla.sla_layernorm_backward(dy, x, wp, mean, rstd, want_grad_weight=False)
        assert none_w is None and torch.equal(dx, got[0]) and torch.equal(db, got[2])


def test_layernorm_autograd_and_differences():
    rows, width = 37, 129
    x = randn(rows, width, dtype=torch.float32, seed=8, shift=0.3).requires_grad_()
    w = randn(width, dtype=torch.float32, seed=9, shift=1.0).requires_grad_()
    b = randn(width, dtype=torch.float32, seed=10).requires_grad_()
    dy = randn(rows, width, dtype=torch.float32, seed=11)
    sla.layer_norm(x, w, b).backward(dy)
    for t, s in ((x, 12), (w, 13), (b, 14)):
        v = randn(*t.shape, dtype=torch.float32, seed=s)
        h = 1e-2
        with torch.no_grad():
            args = [x, w, b]
            i = [k for k, a in enumerate(args) if a is t][0]
            f = []
            for sign in (1, -1):
                args[i] = t + sign * h * v
                f.append(float((sla.layer_norm(*args).double() * dy.double()).sum()))
        d = (f[0] - f[1]) / (2 * h)
        # central differences: h^2 / 6 times the third derivative (of order one a term), and float32 rounding / h
        scale = float((t.grad.double() * v.double()).abs().sum())
        assert abs(d - float((t.grad.double() * v.double()).sum())) <= 3e-3 * scale


@pytest.mark.parametrize("dtype", TYPES)
def test_layernorm_strides_offsets_and_leading_dimensions(dtype):
    big = randn(50, 300, dtype=dtype, seed=15, shift=0.5)
    for x in (big[:, :256], big[:, 1:258], big[::2, 8:136], big[3:4, 5:6]):
        check_ln(x, None, None, sla.layer_norm(x))
    x = randn(4, 5, 64, dtype=dtype, seed=16)
    assert torch.equal(sla.layer_norm(x).view(20, 64), sla.layer_norm(x.view(20, 64)))
    xt = randn(64, 40, dtype=dtype, seed=17).t()  # the autograd entry copies what it cannot read in place
    assert torch.equal(sla.layer_norm(xt), sla.layer_norm(xt.contiguous()))
    with pytest.raises(ValueError, match="contiguous"):
        sla.sla_layernorm(xt)
    w = randn(64, dtype=dtype, seed=18).requires_grad_()
    y = sla.layer_norm(xt.contiguous(), w)
    y.sum().backward()  # an expanded dy
    assert torch.isfinite(w.grad).all()


def test_layernorm_special_rows():
    x = randn(6, 200, dtype=torch.float32, seed=19)
    x[1] = 3.5                      # no deviation: rstd = 1 / sqrt(eps), y = 0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    x[4] = 1e4 + x[4]               # far from zero: no cancellation of mean(x^2) - mean^2
    y = sla.layer_norm(x)
    good = [0, 1, 4, 5]
    assert torch.isfinite(y[good]).all() and torch.isnan(y[2:4]).all()
    assert float(y[1].abs().max()) == 0.0
    check_ln(x[good].contiguous(), None, None, y[good])
    none = torch.empty(0, 200, device=DEV, requires_grad=True)
    w = torch.ones(200, device=DEV, requires_grad=True)
    out = sla.layer_norm(none, w)
    out.sum().backward()
    assert out.shape == (0, 200) and none.grad.shape == (0, 200) and float(w.grad.abs().sum()) == 0.0


def test_layernorm_on_another_stream():
    s = torch.cuda.Stream()
    x = randn(4096, 512, dtype=torch.bfloat16, seed=20)
    want = sla.layer_norm(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = sla.layer_norm(x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(20, 8191), (9, 8191), (3, 4095), (1, 8193)])
def test_layernorm_backward_of_fewer_rows_than_blocks(rows, width, dtype):
    # odd widths, so that the rows' starts fall into several classes of alignment and some blocks have no row
    x, dy = (randn(rows, width, dtype=dtype, seed=s, shift=0.4) for s in (21, 22))
    w, b = (randn(width, dtype=torch.float32, seed=s) for s in (23, 24))
    ref = ln_grads64(x, w, b, dy)
    _, mean, rstd = sla.sla_layernorm(x, w, b, stats=True)
    got = sla.sla_layernorm_backward(dy, x, w, mean, rstd)
    # relative L2: the output's rounding (dw, db are float32) and float32 sums of `width` or `rows` terms
    for g, r, u in zip(got, ref, (U[dtype], U[torch.float32], U[torch.float32])):
        assert rel(g, r) <= u + FP32_LN * 4


@pytest.mark.parametrize("width", [1024, 1001])
def test_layernorm_past_32_bit_offsets(width):
    rows, part, dtype = 2_200_003, 100_000, torch.bfloat16
    assert rows * width > 1 << 31
    x, dy = (randn(rows, width, dtype=dtype, seed=s, shift=0.4) for s in (25, 26))
    w, b = (randn(width, dtype=torch.float32, seed=s) for s in (27, 28))
    y, mean, rstd = sla.sla_layernorm(x, w, b, stats=True)
    dx, dw, db = sla.sla_layernorm_backward(dy, x, w, mean, rstd)
    sums, terms = [0.0, 0.0], 0.0
    for r in range(0, rows, part):
        c = slice(r, r + part)
        check_ln(x[c], w, b, y[c])
        _, xh, r64, _ = ln64(x[c], w, b, 1e-5)
        ref = ln_grads64(x[c], w, b, dy[c])
        assert rel(dx[c], ref[0]) <= U[dtype] + FP32_LN * 4
        amp = 1 + x[c].double().abs().amax(-1, keepdim=True) * r64
        terms = terms + (dy[c].double().abs() * (1 + xh.abs()) * amp).sum(0)
        sums = [sums[0] + ref[1], sums[1] + ref[2]]
    for g, r in zip((dw, db), sums):  # as in test_layernorm_backward
        assert float(((g.double() - r).abs() - U[torch.float32] * r.abs() - 2 * FP32_LN * terms).max()) <= 0


# ------------------------------------------------------------------ gated feed-forward block

ACTS = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
        "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}


def ffn64(x, w_in, w_out, b_in, b_out, act):
    gu = torch.nn.functional.linear(x, w_in, b_in)
    g, u = gu.chunk(2, dim=-1)
    return torch.nn.functional.linear(ACTS[act](g) * u, w_out, b_out)


def ffn_inputs(tokens, width, hidden, out, dtype, bias, seed):
    x = randn(tokens, width, dtype=dtype, seed=seed)
    w_in = randn(2 * hidden, width, dtype=dtype, seed=seed + 1, scale=width ** -0.5)
    w_out = randn(out, hidden, dtype=dtype, seed=seed + 2, scale=hidden ** -0.5)
    b_in = randn(2 * hidden, dtype=dtype, seed=seed + 3, scale=0.2) if bias else None
    b_out = randn(out, dtype=dtype, seed=seed + 4, scale=0.2) if bias else None
    return x, w_in, w_out, b_in, b_out


FFN_SHAPES = [(1, 1, 1, 1), (2, 3, 5, 7), (1, 64, 256, 64), (1, 250, 683, 131), (5, 96, 40, 200), (8, 128, 512, 128),
              (13, 768, 200, 77), (16, 256, 128, 256), (17, 72, 264, 72), (31, 64, 250, 33), (33, 65, 129, 66),
              (64, 128, 384, 64), (127, 130, 126, 128), (128, 256, 512, 256), (129, 64, 256, 64), (300, 250, 683, 131),
              (513, 512, 136, 520), (1000, 48, 96, 24), (1531, 256, 1024, 256), (2049, 33, 64, 17)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", FFN_SHAPES)
def test_ffn_forward_and_backward(shape, dtype):
    k = FFN_SHAPES.index(shape) + TYPES.index(dtype)
    # relu's derivative is not continuous: a sum near 0 may fall on the other side, so float32 gradients take the smooth ones
    act = (["silu", "gelu", "gelu_tanh"] if dtype == torch.float32 else list(ACTS))[k % (3 if dtype == torch.float32 else 4)]
    bias = k % 2 == 0
    args = ffn_inputs(*shape, dtype, bias, seed=100 + 7 * k)
    dy = randn(shape[0], shape[3], dtype=dtype, seed=50 + k)
    leaves = [None if t is None else t.double().requires_grad_() for t in args]
    ref = ffn64(*leaves, act)
    grads = torch.autograd.grad(ref, [t for t in leaves if t is not None], dy.double())
    tol = FFN_TOL[dtype]
    y = sla.sla_gated_ffn(*args, activation=act)
    assert rel(y, ref.detach()) <= tol
    y2, saved = sla.sla_gated_ffn(*args, activation=act, save=True)
    assert rel(y2, ref.detach()) <= tol
    got = sla.sla_gated_ffn_backward(dy, args[0], args[1], args[2], saved, activation=act, want_grad_bias=bias)
    for name, g, r in zip(("dx", "dw_in", "dw_out", "db_in", "db_out"), [g for g in got if g is not None], grads):
        assert g.dtype == dtype and rel(g, r) <= tol, (name, rel(g, r))
    again = sla.sla_gated_ffn_backward(dy, args[0], args[1], args[2], saved, activation=act, want_grad_bias=bias)
    assert all(p is None or torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [33, 20000, 60001])
@pytest.mark.parametrize("width,hidden,out", [(64, 256, 64), (40, 50, 24), (128, 130, 128), (17, 192, 5), (72, 448, 16)])
def test_ffn_narrow_forward(width, hidden, out, tokens, dtype):
    """Narrow blocks run in one kernel, which takes several tiles of tokens in turn (one to seven chunks of h a tile)."""
    bias = tokens != 20000
    args = ffn_inputs(tokens, width, hidden, out, dtype, bias, seed=hidden)
    y = sla.sla_gated_ffn(*args, activation="gelu_tanh")
    ref = ffn64(*[None if t is None else t.double() for t in args], "gelu_tanh")
    assert rel(y, ref) <= FFN_TOL[dtype]
    assert float((y.double() - ref).abs().max()) <= 8 * FFN_TOL[dtype] * float(ref.abs().max())
    assert torch.equal(y, sla.sla_gated_ffn(*args, activation="gelu_tanh"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("tokens", [1, 40, 260])
def test_ffn_activations(act, tokens, dtype):
    args = ffn_inputs(tokens, 128, 256, 64, dtype, True, seed=31)
    args[3][:8] = 30.0       # saturated gates, both ends
    args[3][8:16] = -30.0
    y = sla.gated_ffn(*args, activation=act)
    assert rel(y, ffn64(*[t.double() for t in args], act)) <= FFN_TOL[dtype]


def test_ffn_differences():
    args = list(ffn_inputs(40, 24, 72, 16, torch.float32, True, seed=60))
    args = [t.requires_grad_() for t in args]
    dy = randn(40, 16, dtype=torch.float32, seed=61)
    sla.gated_ffn(*args, activation="gelu").backward(dy)
    for i, t in enumerate(args):
        v = randn(*t.shape, dtype=torch.float32, seed=62 + i)
        v = v / v.norm()
        h, f = 1e-2, []
        with torch.no_grad():
            for sign in (1, -1):
                moved = list(args)
                moved[i] = t + sign * h * v
                f.append(float((sla.gated_ffn(*moved, activation="gelu").double() * dy.double()).sum()))
        want = float((t.grad.double() * v.double()).sum())
        # h^2 times third derivatives and float32 rounding / h, relative to the gradient's size
        assert abs((f[0] - f[1]) / (2 * h) - want) <= 2e-3 * float(t.grad.double().norm())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [1, 12, 200])
def test_ffn_rows_do_not_meet(tokens, dtype):
    """A NaN, an infinity or a zero row stays in its row, forward and in dx."""
    x, w_in, w_out, b_in, b_out = ffn_inputs(tokens, 136, 264, 72, dtype, True, seed=70)
    y = sla.sla_gated_ffn(x, w_in, w_out, b_in, b_out)
    bad = tokens // 2
    x2 = x.clone()
    x2[bad, 3] = float("nan")
    y2, saved = sla.sla_gated_ffn(x2, w_in, w_out, b_in, b_out, save=True)
    assert torch.isnan(y2[bad]).all()
    keep = [i for i in range(tokens) if i != bad]
    assert torch.equal(y2[keep], y[keep])
    dx = sla.sla_gated_ffn_backward(torch.ones_like(y), x2, w_in, w_out, saved)[0]
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[bad]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [3, 150])
def test_ffn_strides_and_offsets(tokens, dtype):
    big = randn(2 * tokens, 300, dtype=dtype, seed=80)
    w_in, w_out = randn(256, 128, dtype=dtype, seed=81, scale=0.1), randn(40, 128, dtype=dtype, seed=82, scale=0.1)
    for x in (big[:tokens, :128], big[:tokens, 1:129], big[::2, 8:136], big[:tokens, 131:259]):
        xc = x.contiguous()
        y, saved = sla.sla_gated_ffn(x, w_in, w_out, save=True)
        yc, saved_c = sla.sla_gated_ffn(xc, w_in, w_out, save=True)
        assert rel(y, yc) <= 2.0 ** -20
        gb = randn(tokens, 50, dtype=dtype, seed=83)
        for dy in (gb[:, :40], gb[:, 3:43]):
            got = sla.sla_gated_ffn_backward(dy, x, w_in, w_out, saved)
            want = sla.sla_gated_ffn_backward(dy.contiguous(), xc, w_in, w_out, saved_c)
            assert all(p is None or rel(p, q) <= 2.0 ** -9 for p, q in zip(got, want))
    # weights at an address that no vector load takes
    flat = randn(256 * 128 + 1, dtype=dtype, seed=84, scale=0.1)
    wo = flat[1:].view(256, 128)
    x = big[:tokens, :128].contiguous()
    assert rel(sla.sla_gated_ffn(x, wo, w_out), ffn64(x.double(), wo.double(), w_out.double(), None, None, "silu")) \
        <= FFN_TOL[dtype]


def test_ffn_leading_dimensions_autograd_and_no_tokens():
    args = ffn_inputs(24, 64, 96, 32, torch.float32, True, seed=90)
    x = args[0].view(2, 3, 4, 64).clone().requires_grad_()
    w = [t.clone().requires_grad_() for t in args[1:]]
    y = sla.gated_ffn(x, *w)
    assert y.shape == (2, 3, 4, 32)
    (g,) = torch.autograd.grad(y.sum(), [x], retain_graph=True)  # only some gradients, an expanded dy
    y.sum().backward()
    assert torch.equal(g, x.grad) and all(t.grad is not None for t in w)
    with pytest.raises(RuntimeError):  # no second derivative
        gx = torch.autograd.grad(sla.gated_ffn(x, *w).square().sum(), [x], create_graph=True)[0]
        gx.sum().backward()
    none = torch.empty(0, 64, device=DEV, requires_grad=True)
    w2 = [t.clone().requires_grad_() for t in args[1:]]
    out = sla.gated_ffn(none, *w2)
    out.sum().backward()
    assert out.shape == (0, 32) and all(float(t.grad.abs().sum()) == 0.0 for t in w2)


def test_ffn_past_32_bit_offsets():
    # tokens * hidden passes 2^31 in the saved factors and in their gradients
    tokens, width, hidden, part, dtype = 550_001, 32, 4096, 50_000, torch.bfloat16
    assert tokens * hidden > 1 << 31
    args = ffn_inputs(tokens, width, hidden, width, dtype, True, seed=110)
    dy = randn(tokens, width, dtype=dtype, seed=111)
    y, saved = sla.sla_gated_ffn(*args, save=True)
    got = sla.sla_gated_ffn_backward(dy, *args[:3], saved, want_grad_bias=True)
    sums = [0.0] * 4
    for r in range(0, tokens, part):
        c = slice(r, r + part)
        leaves = [t.double().requires_grad_() for t in (args[0][c], *args[1:])]
        ref = ffn64(*leaves, "silu")
        assert rel(y[c], ref.detach()) <= FFN_TOL[dtype]
        grads = torch.autograd.grad(ref, leaves, dy[c].double())
        assert rel(got[0][c], grads[0]) <= FFN_TOL[dtype]
        sums = [s + g for s, g in zip(sums, grads[1:])]
    for name, g, r in zip(("dw_in", "dw_out", "db_in", "db_out"), got[1:], (sums[0], sums[1], sums[2], sums[3])):
        assert rel(g, r) <= FFN_TOL[dtype], (name, rel(g, r))


def test_ffn_check_reports_nothing_after_good_calls():
    args = ffn_inputs(300, 128, 320, 128, torch.bfloat16, True, seed=115)
    sla.sla_gated_ffn(*args)
    assert sla.sla_gated_ffn_check() is None and sla.sla_gated_ffn_check(torch.cuda.current_device()) is None


def test_ffn_on_another_stream_and_in_a_graph():
    args = ffn_inputs(700, 128, 320, 128, torch.bfloat16, True, seed=95)
    want = sla.sla_gated_ffn(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = sla.sla_gated_ffn(*args)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sla.sla_gated_ffn(*args)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def dense_step(z, w, b, args, dy):
    h, mean, rstd = sla.sla_layernorm(z, w, b, stats=True)
    y, saved = sla.sla_gated_ffn(h, *args[1:], save=True)
    dh = sla.sla_gated_ffn_backward(dy, h, *args[1:3], saved, want_grad_bias=True)
    return (y, *dh, *sla.sla_layernorm_backward(dh[0], z, w, mean, rstd))


def dense_case(tokens, seed):
    # width and out that 8 does not divide and a split k: the calls' workspaces are in use
    args = ffn_inputs(tokens, 100, 320, 100, torch.bfloat16, True, seed=seed)
    w, b = randn(100, dtype=torch.float32, seed=seed + 5, shift=1.0), randn(100, dtype=torch.float32, seed=seed + 6)
    return args[0], w, b, args, randn(tokens, 100, dtype=torch.bfloat16, seed=seed + 7)


def test_dense_workspaces_on_several_streams():
    cases = [dense_case(t, 120 + t) for t in (300, 9, 700, 2000)]
    want = [dense_step(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in cases]
    for _ in range(20):
        for k, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[k].append(dense_step(*c))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for run in runs for a, b in zip(run, w))


def test_dense_workspaces_in_several_threads():
    from concurrent.futures import ThreadPoolExecutor
    cases = [dense_case(t, 140 + t) for t in (300, 9, 700, 2000)]
    want = [dense_step(*c) for c in cases]
    torch.cuda.synchronize()
    with ThreadPoolExecutor(len(cases)) as pool:  # all on the default stream
        got = list(pool.map(lambda c: [dense_step(*c) for _ in range(20)], cases))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for run in runs for a, b in zip(run, w))


def test_dense_workspace_of_a_graph_is_its_own():
    case, other = dense_case(300, 160), dense_case(700, 170)
    want, expect = dense_step(*case), dense_step(*other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dense_step(*case)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # replays and calls side by side
        with torch.cuda.stream(s):
            graph.replay()
        got = dense_step(*other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(got, expect))


# ------------------------------------------------------------------ refusals

def test_refusals():
    x = randn(8, 64, dtype=torch.float32, seed=1)
    w_in, w_out = randn(64, 64, dtype=torch.float32, seed=2), randn(16, 32, dtype=torch.float32, seed=3)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        sla.layer_norm(x.double())
    with pytest.raises(ValueError, match="shape"):
        sla.layer_norm(x, torch.ones(63, device=DEV))
    with pytest.raises(ValueError, match="dtype"):
        sla.layer_norm(x, torch.ones(64, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        sla.layer_norm(x, torch.ones(64))
    with pytest.raises(sla.SlaError):
        sla.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError, match="last dimension"):
        sla.layer_norm(torch.empty(4, 0, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        sla.sla_layernorm(x[:1].expand(8, 64))
    with pytest.raises(ValueError, match="activation"):
        sla.gated_ffn(x, w_in, w_out, activation="swish")
    with pytest.raises(ValueError, match="w_in must be"):
        sla.gated_ffn(x, w_in[:62], w_out)
    with pytest.raises(ValueError, match="shape"):
        sla.gated_ffn(x[:, :60].contiguous(), w_in, w_out)
    with pytest.raises(ValueError, match="dtype"):
        sla.gated_ffn(x.half(), w_in, w_out)
    with pytest.raises(ValueError, match="shape"):
        sla.gated_ffn(x, w_in, w_out, b_out=torch.zeros(32, device=DEV))
    y, saved = sla.sla_gated_ffn(x, w_in, w_out, save=True)
    with pytest.raises(ValueError, match="dy must have shape"):
        sla.sla_gated_ffn_backward(x, x, w_in, w_out, saved)
    with pytest.raises(ValueError, match="saved"):
        sla.sla_gated_ffn_backward(y, x, w_in, w_out, saved.float())
    with pytest.raises(sla.SlaError, match="WORKSPACE"):
        sla.sla_gated_ffn_backward(y, x, w_in, w_out, saved[:256])
