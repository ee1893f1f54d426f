"""The linear layer on the GPU against its definition in 64 bits.

Tolerances, relative L2 (U: the type's unit roundoff, K: the products of a sum):
  16-bit y: the result's rounding, U at most, and the float32 sum's, K / 16 * 2^-24 * 2/3 (what a tensor core drops: a unit
      2^-23 of the running sum for every 16 products at most, half of it on average, 2/3 of that over a sum that grows as its
      root) below 4 * 2^-16 for K <= 2^14.
  16-bit gradients: dp and the result are rounded, each by U at most and, independent of one another, by U / 2
      in L2 on average (a rounding to nearest is off by U / sqrt(3) of the spacing's upper end, less below it): 2 U covers both and the
      activations' own 2^-19.  A sum over one or two rows or columns may have all of one sign: 4 U there.
  float32: runs of 512 products: 512 / 16 * 2^-24 * 2/3 = 1.3e-6, dropped third parts 2^-24, activations 2^-19 = 1.9e-6,
      the sums of splits and runs 2^-22: 5e-6.
"""
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


def y_tol(dtype):
    return 5e-6 if dtype == torch.float32 else U[dtype] + 4 * 2.0 ** -16


def grad_tol(dtype, terms=64):
    if dtype == torch.float32:
        return 5e-6
    return (2 if terms > 8 else 4) * U[dtype] + 4 * 2.0 ** -16


def randn(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def rel(a, b) -> float:
    a, b = a.double(), b.double()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n > 0 else 1.0)


def linear64(x, w, b, r, act):
    p = torch.nn.functional.linear(x, w, b)
    f = torch.nn.functional
    y = {"none": lambda t: t, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"),
         "relu": torch.relu}[act](p)
    return y if r is None else y + r


def data(tokens, width, out, dtype, seed=1):
    return (randn(tokens, width, dtype=dtype, seed=seed), randn(out, width, dtype=dtype, seed=seed + 1, scale=width ** -0.5),
            randn(out, dtype=dtype, seed=seed + 2, scale=0.3), randn(tokens, out, dtype=dtype, seed=seed + 3),
            randn(tokens, out, dtype=dtype, seed=seed + 4))


SIZES = [(1, 1, 1), (1, 1024, 4096), (2, 33, 7), (8, 64, 64), (9, 250, 131), (16, 768, 300), (17, 8, 8), (33, 96, 1),
         (40, 1, 96), (129, 64, 64), (300, 136, 48), (300, 130, 16), (257, 1024, 33), (515, 333, 700), (64, 4500, 40),
         (2049, 250, 131), (5000, 64, 192), (20, 2048, 2048)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,width,out", SIZES)
def test_forward_and_backward(tokens, width, out, dtype):
    x, w, b, r, dy = data(tokens, width, out, dtype)
    for i, act in enumerate(ACTS):
        bias, res = (b if i % 2 == 0 or out == 1 else None), (r if i in (0, 2, 3) else None)
        leaves = [t.double().requires_grad_() for t in (x, w, b)]
        want = linear64(leaves[0], leaves[1], None if bias is None else leaves[2], None if res is None else res.double(), act)
        y, saved = sla.sla_linear(x, w, bias, res, activation=act, save=True)
        assert rel(y, want.detach()) <= y_tol(dtype), (act, rel(y, want.detach()))
        assert torch.equal(y, sla.sla_linear(x, w, bias, res, activation=act))
        if act == "relu" and dtype == torch.float32:
            continue  # where the last bit of a sum decides whether there is a gradient
        grads = torch.autograd.grad(want, leaves if bias is not None else leaves[:2], dy.double())
        got = sla.sla_linear_backward(dy, x, w, saved, activation=act, want_grad_bias=bias is not None)
        for g, ref, terms in zip(got, grads, (out, tokens, tokens)):
            assert rel(g, ref) <= grad_tol(dtype, terms), (act, g.shape, rel(g, ref))
        again = sla.sla_linear_backward(dy, x, w, saved, activation=act, want_grad_bias=bias is not None)
        assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))
        for wants in ((True, False), (False, True)):
            part = sla.sla_linear_backward(dy, x, w, saved, activation=act, want_grad_x=wants[0], want_grad_weight=wants[1])
            assert (part[0] is None) != wants[0] and (part[1] is None) != wants[1] and part[2] is None
            for p, q in zip(part, got):
                assert p is None or rel(p, q) <= 2 * grad_tol(dtype, 1)
    sla.sla_gated_ffn_check()


def test_autograd_and_differences():
    x, w, b, r, dy = data(37, 29, 19, torch.float32, seed=20)
    for act in ("silu", "gelu"):
        leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
        sla.linear(*leaves, activation=act).backward(dy)
        assert torch.equal(leaves[3].grad, dy)
        for i, t in enumerate(leaves):
            v, step = randn(*t.shape, dtype=torch.float32, seed=30 + i), 1e-2
            f = []
            for sign in (1, -1):
                args = [p.detach() for p in leaves]
                args[i] = args[i] + sign * step * v
                f.append(float((sla.linear(*args, activation=act).double() * dy).sum()))
            d = (f[0] - f[1]) / (2 * step)
            # step^2 / 6 times the third derivative, of order one a term, and float32 roundings over the step
            size = float((t.grad.double() * v.double()).abs().sum())
            assert abs(d - float((t.grad.double() * v.double()).sum())) <= 3e-3 * size
    y = sla.linear(x, w.clone().requires_grad_())
    assert y.grad_fn is not None and sla.linear(x, w).grad_fn is None
    only = r.clone().requires_grad_()
    sla.linear(x, w, residual=only).backward(dy)
    assert torch.equal(only.grad, dy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [5, 70])
def test_layouts(tokens, dtype):
    width, out = 72, 40
    x, w, b, r, dy = data(tokens, width, out, dtype, seed=40)
    want = linear64(*(t.double() for t in (x, w, b, r)), "gelu")
    y = sla.sla_linear(x, w, b, r, activation="gelu")
    for pad in (1, 8):  # rows of no alignment, and wider ones that are aligned
        wide = torch.zeros(tokens, width + pad, dtype=dtype, device=DEV)
        wide[:, :width] = x
        rw = torch.zeros(tokens, out + pad, dtype=dtype, device=DEV)
        rw[:, :out] = r
        got, saved = sla.sla_linear(wide[:, :width], w, b, rw[:, :out], activation="gelu", save=True)
        assert rel(got, want) <= y_tol(dtype)
        dw = torch.zeros(tokens, out + pad, dtype=dtype, device=DEV)
        dw[:, :out] = dy
        g = sla.sla_linear_backward(dw[:, :out], wide[:, :width], w, saved, activation="gelu", want_grad_bias=True)
        _, kept = sla.sla_linear(x, w, b, r, activation="gelu", save=True)
        h = sla.sla_linear_backward(dy, x, w, kept, activation="gelu", want_grad_bias=True)
        assert all(rel(p, q) <= 2 * grad_tol(dtype, 1) for p, q in zip(g, h))
    odd = torch.empty(tokens * out + 1, dtype=dtype, device=DEV)[1:].view(tokens, out)
    assert rel(sla.sla_linear(x, w, b, r, activation="gelu", y=odd), want) <= y_tol(dtype)
    shift = torch.empty(w.numel() + 1, dtype=dtype, device=DEV)[1:].view(out, width).copy_(w)
    sb = torch.empty(out + 1, dtype=dtype, device=DEV)[1:].copy_(b)
    assert rel(sla.sla_linear(x, shift, sb, r, activation="gelu"), want) <= y_tol(dtype)
    three = x.view(1, tokens, width)
    assert torch.equal(sla.linear(three, w, b, r.view(1, tokens, out), "gelu")[0], y)
    assert torch.equal(sla.linear(x.t().contiguous().t(), w.t().contiguous().t(), b, r, "gelu"), y)
    assert sla.linear(x, w, b, r.expand(tokens, out), "gelu").shape == (tokens, out)
    dx = torch.autograd.grad(sla.linear(x.requires_grad_(), w).sum(), x)[0]  # an upstream gradient without strides
    assert rel(dx, w.double().sum(0).expand(tokens, width)) <= grad_tol(dtype, 1) * 4


def test_no_tokens():
    x = torch.empty(0, 24, dtype=torch.float16, device=DEV)
    w = torch.ones(40, 24, dtype=torch.float16, device=DEV)
    y, saved = sla.sla_linear(x, w, activation="silu", save=True)
    assert y.shape == (0, 40)
    dx, dw, db = sla.sla_linear_backward(y, x, w, saved, activation="silu", want_grad_bias=True)
    assert dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [6, 300])
def test_what_is_no_number_stays_in_its_row(tokens, dtype):
    x, w, b, r, _ = data(tokens, 100, 50, dtype, seed=60)
    y = sla.sla_linear(x, w, b, r, activation="silu")
    for value in (float("nan"), float("inf")):
        x2, r2 = x.clone(), r.clone()
        x2[3, 7] = value
        r2[4, 9] = value
        y2 = sla.sla_linear(x2, w, b, r2, activation="silu")
        rows = [t for t in range(tokens) if t not in (3, 4)]
        assert torch.equal(y2[rows], y[rows])
        cols = [c for c in range(50) if c != 9]
        assert torch.equal(y2[4, cols], y[4, cols]) and not bool(y2[4, 9].isfinite())
        assert not bool(y2[3].isfinite().all())


def test_streams_graphs_and_a_shared_workspace():
    for dtype in (torch.bfloat16, torch.float32):
        x, w, b, r, dy = data(700, 256, 200, dtype, seed=70)

        def call(ws=None):
            y, saved = sla.sla_linear(x, w, b, r, activation="gelu", save=True, workspace=ws)
            return (y, *sla.sla_linear_backward(dy, x, w, saved, activation="gelu", want_grad_bias=True, workspace=ws))

        want = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = call()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = call(ws)
            graphs.append((graph, out))
        for _ in range(2):
            for graph, out in graphs:
                out[0].zero_()
                graph.replay()
                assert all(torch.equal(p, q) for p, q in zip(out, want))
    sla.sla_gated_ffn_check()


def test_refusals():
    x = randn(20, 16, dtype=torch.float16, seed=80)
    w = randn(24, 16, dtype=torch.float16, seed=81)
    y, saved = sla.sla_linear(x, w, activation="gelu", save=True)
    for call, message in (
            (lambda: sla.sla_linear(x.cpu(), w), "CUDA tensor"),
            (lambda: sla.sla_linear(x.double(), w.double()), "float32, float16"),
            (lambda: sla.sla_linear(x, w[0]), "weight must be"),
            (lambda: sla.sla_linear(x, w[:, :8].contiguous()), "weight must have"),
            (lambda: sla.sla_linear(x, w.float()), "weight must have"),
            (lambda: sla.sla_linear(x, w, w[0]), "bias must have"),
            (lambda: sla.sla_linear(x, w, residual=x), "residual must have"),
            (lambda: sla.sla_linear(x, w, residual=y.float()), "residual must have"),
            (lambda: sla.sla_linear(x, w, activation="tanh"), "unknown activation"),
            (lambda: sla.sla_linear(x, w, y=y[:5]), "y must have"),
            (lambda: sla.sla_linear(x.t(), w), "contiguous"),
            (lambda: sla.sla_linear_backward(x, x, w, saved, activation="gelu"), "dy must have"),
            (lambda: sla.sla_linear_backward(y, x, w, saved.float(), activation="gelu"), "saved must be"),
            (lambda: sla.sla_linear_backward(y, x, w, saved, activation="silu"), "saved is from"),
            (lambda: sla.sla_linear_backward(y[:8], x[:8], w, saved, activation="gelu"), "saved is from")):
        with pytest.raises(ValueError, match=message):
            call()


# Few outputs.  A thread adds up at most tokens / 304 + 2 products of dW in a row: a random walk of roundings, below 2^-24
# sqrt(300) = 1.1e-6 here, within the tolerances above.
FEW = [(17, 1, 1), (19, 3, 2), (33, 7, 3), (40, 64, 8), (301, 250, 5), (70001, 64, 1), (1003, 384, 4), (515, 2047, 8),
       (260, 2048, 2), (100, 2049, 2), (2000, 129, 2), (70, 130, 1), (3, 64, 3), (1, 2048, 8), (5000, 48, 7), (300, 64, 9)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,width,out", FEW)
def test_few_outputs(tokens, width, out, dtype):
    x, w, b, r, dy = data(tokens, width, out, dtype, seed=300)
    for act, bias, res in (("none", b, None), ("gelu", b, r), ("relu", None, r), ("silu", None, None)):
        leaves = [t.double().requires_grad_() for t in (x, w, b)]
        want = linear64(leaves[0], leaves[1], None if bias is None else leaves[2], None if res is None else res.double(), act)
        y, saved = sla.sla_linear(x, w, bias, res, activation=act, save=True)
        for t in (y, sla.sla_linear(x, w, bias, res, activation=act)):
            assert float((t.double() - want.detach()).norm()) <= y_tol(dtype) * float(want.detach().norm() + b.double().norm()), act
        want.backward(dy.double())
        dx, dw, db = sla.sla_linear_backward(dy, x, w, saved, activation=act, want_grad_bias=True)
        # of a single row or column the sums may nearly cancel: relative to the terms' sizes
        p = linear64(leaves[0], leaves[1], None if bias is None else leaves[2], None, "none").detach().requires_grad_()
        linear64(p, torch.eye(out, dtype=torch.float64, device=DEV), None, None, act).backward(dy.double())
        dp, x64, w64 = p.grad.abs(), x.double().abs(), w.double().abs()
        for got, ref, size in ((dx, leaves[0].grad, dp @ w64), (dw, leaves[1].grad, dp.T @ x64)):
            scale = float(ref.norm()) + 2.0 ** -8 * float(size.norm())
            assert float((got.double() - ref).norm()) <= grad_tol(dtype, min(tokens, out)) * scale, act
        if bias is not None:
            scale = float(leaves[2].grad.norm()) + 2.0 ** -8 * float(dp.sum(0).norm())
            assert float((db.double() - leaves[2].grad).norm()) <= grad_tol(dtype, 1) * scale, act


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,out", [(64, 3), (63, 2), (96, 1)])
def test_few_outputs_layouts_and_rows_apart(width, out, dtype):
    tokens = 203
    x, w, b, r, dy = data(tokens, width, out, dtype, seed=320)
    y, saved = sla.sla_linear(x, w, b, r, activation="silu", save=True)
    dx, dw, db = sla.sla_linear_backward(dy, x, w, saved, activation="silu", want_grad_bias=True)
    for pad in (1, 8):
        wide, wide_dy = torch.full((tokens, width + pad), float("nan"), dtype=dtype, device=DEV), torch.zeros_like(dy.repeat(1, 3))
        wide[:, :width], wide_dy[:, 1:1 + out] = x, dy
        xs, dys = wide[:, :width], wide_dy[:, 1:1 + out]
        y2, saved2 = sla.sla_linear(xs, w, b, r, activation="silu", save=True)
        dx2, dw2, db2 = sla.sla_linear_backward(dys, xs, w, saved2, activation="silu", want_grad_bias=True)
        assert rel(y2, y) <= 2 * y_tol(dtype)  # (columns of a thread differ: so does the order of the sums)
        for a, c in ((dx2, dx), (dw2, dw), (db2, db)):
            assert rel(a, c) <= 2 * grad_tol(dtype)
    again = sla.sla_linear_backward(dy, x, w, saved, activation="silu", want_grad_bias=True)
    assert all(torch.equal(a, c) for a, c in zip(again, (dx, dw, db)))
    for value in (float("nan"), float("inf")):  # the last row too, which threads without a row read
        x2 = x.clone()
        x2[tokens - 1, width - 1], x2[3, 0] = value, value
        y2 = sla.sla_linear(x2, w, b, r, activation="none")
        kept = torch.ones(tokens, dtype=torch.bool, device=DEV)
        kept[3] = kept[tokens - 1] = False
        assert torch.equal(y2[kept], sla.sla_linear(x, w, b, r, activation="none")[kept]) and not bool(y2[~kept].isfinite().any())
        if value == value:  # dW_oc = sum dp_o x_c: infinite in those columns, no NaN in any
            _, dw2, _ = sla.sla_linear_backward(dy, x2, w, sla.sla_linear(x2, w, b, save=True)[1])
            assert not bool(dw2[:, 1:width - 1].isinf().any()) and not bool(dw2.isnan().any())
            assert bool(dw2[:, [0, width - 1]].isinf().all())


def test_few_outputs_some_gradients_and_no_tokens():
    x, w, b, r, dy = data(50, 64, 2, torch.float32, seed=340)
    _, saved = sla.sla_linear(x, w, b, save=True)
    full = sla.sla_linear_backward(dy, x, w, saved, want_grad_bias=True)
    x, w, b = (t.clone().requires_grad_() for t in (x, w, b))
    for leaves, want in (((x,), full[:1]), ((w,), full[1:2]), ((b,), full[2:]), ((x, b), (full[0], full[2]))):
        args = [t if any(t is q for q in leaves) else t.detach() for t in (x, w, b)]
        got = torch.autograd.grad(sla.linear(*args), leaves, dy)
        assert all(torch.equal(a, c) for a, c in zip(got, want))
    _, saved = sla.sla_linear(x[:0].detach(), w.detach(), b.detach(), save=True)
    dx, dw, db = sla.sla_linear_backward(dy[:0], x[:0].detach(), w.detach(), saved, want_grad_bias=True)
    assert dx.shape == (0, 64) and not bool(dw.any()) and not bool(db.any())
