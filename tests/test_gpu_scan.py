"""The gated scan on the GPU against its definition in 64 bits, row after row on the CPU.

Tolerances follow the float32 work along the recurrence (u = 2^-24, M the largest |x| or |state| of a channel's sequence, d the
relative error of the smaller of a and 1 - a: the exponential and the reciprocal by approximation, 2^-21 with their
sums and products, and the rounding of the exponent, |g| 2^-23):
    a step x + a (h - x), or of the maps it is put together from, adds at most 2 M (4 u + d (1 - a)) to a times the error
    before it (a's own rounding u and the difference's u, of |h - x| <= 2 M, and the sum's u / 2)
    a step of l, of at most L, adds 2 L (4 u + d min(a, 1 - a)) in the same way
and the result's own rounding to its type on top.  Those bounds are carried along with the recurrences here.
"""
import numpy as np
import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
# a closed gate still lets 2^-126, float32's smallest normal number, of what it is multiplied with through (values up to 16)
TINY = {torch.float32: 2.0 ** -122, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -122}
F = 2.0 ** -24


def randn(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def scan64(x, g, state, marks, reverse, dh=None, dfinal=None):
    """Results and their bounds (without the rounding to a type), from numpy arrays [rows, channels]: step after step, all
    sequences that are long enough at a time."""
    n, c = x.shape
    a, b = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    d = np.abs(g) * 2.0 ** -23 + 2.0 ** -21
    small = np.minimum(a, b)
    h, eh, before, eb = (np.zeros((n, c)) for _ in range(4))
    begin, length = np.array(marks[:-1], dtype=int), np.diff(marks)
    most = np.abs(state)
    for q, (p0, p1) in enumerate(zip(marks[:-1], marks[1:])):
        if p1 > p0:
            most[q] = np.maximum(most[q], np.abs(x[p0:p1]).max(0))

    def rows(t):
        on = np.flatnonzero(length > t)
        return on, (begin + length - 1 - t if reverse else begin + t)[on]

    s, e = state.copy(), np.zeros_like(state)
    steps = int(length.max(initial=0))
    for t in range(steps):
        on, r = rows(t)
        before[r], eb[r] = s[on], e[on]
        s[on] = a[r] * s[on] + b[r] * x[r]
        e[on] = a[r] * e[on] + 2 * most[on] * (4 * F + d[r] * b[r])
        h[r], eh[r] = s[on], e[on]
    out = dict(h=(h, eh), final=(s, e))
    if dh is None:
        return out
    dx, dg, edx, edg, ls = (np.zeros((n, c)) for _ in range(5))
    m, most = dfinal.copy(), np.abs(dfinal)
    for t in reversed(range(steps)):
        on, r = rows(t)
        ls[r] = dh[r] + m[on]
        m[on] = a[r] * ls[r]
        most[on] = np.maximum(most[on], np.abs(ls[r]))
    e = np.zeros_like(state)
    for t in reversed(range(steps)):
        on, r = rows(t)
        l, el = ls[r], e[on] + 2 * F * most[on]
        gap, ab = before[r] - x[r], a[r] * b[r]
        dx[r], edx[r] = b[r] * l, b[r] * (el + (d[r] + 2 * F) * np.abs(l))
        dg[r] = l * gap * ab
        edg[r] = ab * (el * np.abs(gap) + np.abs(l) * (eb[r] + F * (np.abs(before[r]) + np.abs(x[r])))
                       + (3 * d[r] + 4 * F) * np.abs(l * gap))
        e[on] = a[r] * el + 2 * most[on] * (4 * F + d[r] * small[r])
    return dict(out, dx=(dx, edx), dg=(dg, edg), ds=(m, e))


def check(got, want, dtype, what):
    ref, err = want
    got = f64(got).reshape(ref.shape)
    bound = err + U[dtype] * (np.abs(ref) + err) + TINY[dtype]
    excess = np.abs(got - ref) - bound
    assert np.all(np.isfinite(got)), what
    assert excess.max() <= 0, f"{what}: {excess.max():.3e} over the bound at {np.unravel_index(excess.argmax(), ref.shape)}"


def inputs(shape, sequences, dtype, seed, scale=1.5):
    both = torch.cat((randn(*shape, dtype=dtype, seed=seed), randn(*shape, dtype=dtype, seed=seed + 1, scale=scale,
                                                                   shift=1.5)), -1)
    c = shape[-1]
    state = randn(sequences, c, dtype=torch.float32, seed=seed + 2)
    return both[..., :c], both[..., c:], state


UNIFORM = [(1, 1, 1), (3, 1, 5), (64, 1, 64), (5, 1, 130), (1, 2, 3), (2, 15, 64), (5, 16, 2), (4, 17, 66),
           (3, 255, 130), (2, 256, 64), (2, 257, 33), (7, 100, 64), (300, 3, 40), (1, 5000, 70), (1, 20001, 64),
           # many sequences of one length, each a warp's: from the shortest that are taken so, in all phases of the saved states
           (760, 64, 2), (770, 65, 6), (380, 101, 66), (765, 131, 4), (256, 70, 180), (800, 71, 3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("sequences,length,channels", UNIFORM)
def test_sequences_of_one_length(sequences, length, channels, reverse, dtype):
    x, g, state = inputs((sequences, length, channels), sequences, dtype, 10)
    dh = randn(sequences, length, channels, dtype=dtype, seed=14)
    dfinal = randn(sequences, channels, dtype=torch.float32, seed=15)
    n = sequences * length
    flat = [f64(t).reshape(n, channels) for t in (x, g, dh)]
    want = scan64(flat[0], flat[1], f64(state), list(range(0, n + 1, length)), reverse, flat[2], f64(dfinal))
    h, final = sla.sla_gated_scan(x, g, state, reverse=reverse)
    check(h, want["h"], dtype, "h")
    check(final, want["final"], torch.float32, "final")
    h2, final2, saved = sla.sla_gated_scan(x, g, state, reverse=reverse, save=True)
    assert torch.equal(h, h2) and torch.equal(final, final2)
    got = sla.sla_gated_scan_backward(dh, x, g, saved, dfinal, state, reverse=reverse)
    for t, k, dt in zip(got, ("dx", "dg", "ds"), (dtype, dtype, torch.float32)):
        check(t, want[k], dt, k)
    again = sla.sla_gated_scan_backward(dh, x, g, saved, dfinal, state, reverse=reverse)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    sla.sla_gated_ffn_check()


RAGGED = [([0, 1], 0, 0), ([3, 0, 5], 2, 4), ([0, 0, 0], 1, 0), ([17, 16, 15, 0, 1, 1, 64], 0, 3),
          ([300, 1, 0, 700, 255, 257, 2], 5, 130), ([9000, 8500], 0, 1), ([1] * 700, 0, 0), ([40] * 13, 3, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_sequences_of_any_length(case, reverse, dtype):
    lengths, lead, behind = RAGGED[case]
    channels = (66, 3, 64, 131)[case % 4]
    marks = [lead]
    for k in lengths:
        marks.append(marks[-1] + k)
    n = marks[-1] + behind
    x, g, state = inputs((n, channels), len(lengths), dtype, 20)
    dh = randn(n, channels, dtype=dtype, seed=24)
    dfinal = randn(len(lengths), channels, dtype=torch.float32, seed=25)
    outside = [r for r in range(n) if r < lead or r >= marks[-1]]
    for t in (x, g, dh):  # what lies in no sequence is not looked at
        t[outside] = float("nan")
    inside = [np.nan_to_num(f64(t)) for t in (x, g, dh)]
    want = scan64(inside[0], inside[1], f64(state), marks, reverse, inside[2], f64(dfinal))
    for kind in (torch.int32, torch.int64):
        how = dict(offsets=torch.tensor(marks, dtype=kind, device=DEV), reverse=reverse)
        h, final, saved = sla.sla_gated_scan(x, g, state, save=True, **how)
        check(h, want["h"], dtype, "h")
        check(final, want["final"], torch.float32, "final")
        got = sla.sla_gated_scan_backward(dh, x, g, saved, dfinal, state, **how)
        for t, k, dt in zip(got, ("dx", "dg", "ds"), (dtype, dtype, torch.float32)):
            check(t, want[k], dt, k)
    kept = torch.full_like(h, 7.0)
    out, _ = sla.sla_gated_scan(x, g, state, h=kept, **how)
    assert out is kept and bool((kept[outside] == 7.0).all())
    assert torch.equal(torch.cat((kept[lead:marks[-1]],)), h[lead:marks[-1]])


def test_gates_at_their_ends():
    # closed (a = 0 to float32) and open (1 - a = 0) gates, infinite ones too; a constant gate close to one over a long way
    n, c = 3000, 8
    x = randn(n, c, dtype=torch.float32, seed=30)
    g = torch.empty(n, c, device=DEV)
    g[:] = torch.tensor([0.0, -0.0, 200.0, -200.0, float("inf"), float("-inf"), 12.0, -12.0], device=DEV)
    state = randn(1, c, dtype=torch.float32, seed=31)
    dh = randn(n, c, dtype=torch.float32, seed=32)
    dfinal = randn(1, c, dtype=torch.float32, seed=33)
    h, final, saved = sla.sla_gated_scan(x, g, state, save=True)
    dx, dg, ds = sla.sla_gated_scan_backward(dh, x, g, saved, dfinal, state)
    with np.errstate(over="ignore"):
        want = scan64(f64(x), np.clip(f64(g), -700, 700), f64(state), [0, n], False, f64(dh), f64(dfinal))
    for t, k in ((h, "h"), (final, "final"), (dx, "dx"), (dg, "dg"), (ds, "ds")):
        check(t, want[k], torch.float32, k)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_is_no_number_stays_in_its_sequence_and_channel(value):
    length, c, dtype = 700, 64, torch.bfloat16
    x, g, state = inputs((3, length, c), 3, dtype, 40)
    x = x.clone()
    base, final = sla.sla_gated_scan(x, g, state)
    x[1, 300, 5] = value
    for which in ("x", "state", "gate"):
        xs, gs, st = x.clone(), g.clone(), state.clone()
        if which != "x":
            xs[1, 300, 5] = 0.25
            if which == "state":
                st[1, 5] = value
            else:
                gs[1, 300, 5] = float("nan")
        h, fin, saved = sla.sla_gated_scan(xs, gs, st, save=True)
        others = torch.ones_like(h, dtype=torch.bool)
        others[1, :, 5] = False
        assert torch.equal(h[others], base[others])
        bad = h[1, :, 5].isfinite().logical_not()
        first = 0 if which == "state" else 300
        assert bool(bad[first:].any()) and not bool(bad[:first].any())
        rest = torch.ones_like(fin, dtype=torch.bool)
        rest[1, 5] = False
        assert torch.equal(fin[rest], final[rest])


@pytest.mark.parametrize("dtype", TYPES)
def test_a_state_is_carried_from_call_to_call(dtype):
    # single steps, or two pieces, with the state kept in place: each within the bounds of one call over all rows
    q, length, c = 5, 40, 96
    x, g, state = inputs((q, length, c), q, dtype, 50)
    n = q * length
    want = scan64(f64(x).reshape(n, c), f64(g).reshape(n, c), f64(state), list(range(0, n + 1, length)), False)
    for cuts in (range(length + 1), (0, 17, 40)):
        kept, parts = state.clone(), []
        for t0, t1 in zip(cuts[:-1], cuts[1:]):
            out, same = sla.sla_gated_scan(x[:, t0:t1].contiguous(), g[:, t0:t1].contiguous(), kept, final=kept)
            assert same is kept
            parts.append(out)
        check(torch.cat(parts, 1), want["h"], dtype, "h")
        check(kept, want["final"], torch.float32, "final")


def test_nothing_to_scan():
    for shape, q in (((0, 5, 8), 0), ((3, 0, 8), 3), ((0, 8), 1)):
        x = torch.empty(shape, dtype=torch.float16, device=DEV)
        state = randn(q, 8, dtype=torch.float32, seed=60)
        h, final, saved = sla.sla_gated_scan(x, x, state, save=True)
        assert h.shape == x.shape and torch.equal(final, state)
        dx, dg, ds = sla.sla_gated_scan_backward(x, x, x, saved, state, state)
        assert dx.shape == x.shape and torch.equal(ds, state)
        _, final = sla.sla_gated_scan(x, x)
        assert final.shape == (q, 8) and not bool(final.any())
    x = randn(6, 8, dtype=torch.float16, seed=61)  # rows, but no sequence
    h, final = sla.sla_gated_scan(x, x, offsets=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert not bool(h.any()) and final.shape == (0, 8)


def test_offsets_that_are_none_touch_nothing_outside():
    # falling and far offsets: results have no meaning, but the call ends and writes its own arrays alone
    n, c = 700, 64
    x, g, _ = inputs((n, c), 1, torch.bfloat16, 70)
    x, g = x.clone(), g.clone()
    guard = torch.full((n + 2, c), 3.0, dtype=torch.bfloat16, device=DEV)
    for marks in ([0, 500, 100, 700], [-50, 2000, 10], [900, 950], [5, -3, 800, 20, 700], [0, 1 << 31, 700]):
        for reverse in (False, True):
            off = torch.tensor(marks, dtype=torch.int64, device=DEV)
            state = randn(len(marks) - 1, c, dtype=torch.float32, seed=71)
            guard.fill_(3.0)
            sla.sla_gated_scan(x, g, state, offsets=off, reverse=reverse, h=guard[1:-1])
            _, _, saved = sla.sla_gated_scan(x, g, state, offsets=off, reverse=reverse, save=True)
            sla.sla_gated_scan_backward(x, x, g, saved, state, state, offsets=off, reverse=reverse)
            sla.sla_gated_ffn_check()
            assert bool((guard[0] == 3.0).all()) and bool((guard[-1] == 3.0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_layouts(dtype):
    n, c = 530, 70
    wide = randn(n, 2 * c + 3, dtype=dtype, seed=80)
    x, g = wide[:, :c], wide[:, c + 1:2 * c + 1]  # rows and columns of no alignment
    state = randn(1, c + 1, dtype=torch.float32, seed=81)[:, 1:].contiguous()
    want, final = sla.sla_gated_scan(x.contiguous(), g.contiguous(), state)
    h, got = sla.sla_gated_scan(x, g, state)
    assert torch.equal(h, want) and torch.equal(final, got)
    h, got = sla.gated_scan(x.t().contiguous().t(), g.expand(n, c), state)  # a copy is made where rows are not whole
    assert torch.equal(h, want) and torch.equal(final, got)
    x4 = randn(2, 3, 11, 6, dtype=dtype, seed=82)
    h, final = sla.gated_scan(x4, x4)
    h3, final3 = sla.gated_scan(x4.reshape(6, 11, 6), x4.reshape(6, 11, 6))
    assert torch.equal(h.reshape(6, 11, 6), h3) and torch.equal(final, final3)
    gaps = randn(4, 9, 20, dtype=dtype, seed=83)[:, :7, :10]  # sequences with rows between them
    h, _ = sla.gated_scan(gaps, gaps)
    assert torch.equal(h, sla.gated_scan(gaps.contiguous(), gaps.contiguous())[0])
    odd = torch.empty(n * c + 1, dtype=dtype, device=DEV)[1:].view(n, c)  # an output of no alignment
    assert torch.equal(sla.sla_gated_scan(x, g, state, h=odd)[0], want)


def test_autograd_and_differences():
    q, length, c = 3, 37, 10
    x, g, state = (t.clone().requires_grad_() for t in inputs((q, length, c), q, torch.float32, 90))
    dh, dfinal = randn(q, length, c, dtype=torch.float32, seed=94), randn(q, c, dtype=torch.float32, seed=95)

    def loss(*args):
        h, final = sla.gated_scan(*args)
        return float((h.double() * dh).sum() + (final.double() * dfinal).sum())

    h, final = sla.gated_scan(x, g, state)
    torch.autograd.backward([h, final], [dh, dfinal])
    for i, t in enumerate((x, g, state)):
        v = randn(*t.shape, dtype=torch.float32, seed=96 + i)
        step = 1e-2
        with torch.no_grad():
            args = [x, g, state]
            f = []
            for sign in (1, -1):
                args[i] = t + sign * step * v
                f.append(loss(*args))
        want = (f[0] - f[1]) / (2 * step)
        # step^2 / 6 times the third derivative, of order one a term, and float32 roundings over the step
        size = float((t.grad.double() * v.double()).abs().sum())
        assert abs(want - float((t.grad.double() * v.double()).sum())) <= 3e-3 * size
    # one of the two results alone
    for which in (0, 1):
        leaves = [t.detach().requires_grad_() for t in (x, g, state)]
        out = sla.gated_scan(*leaves)
        got = torch.autograd.grad(out[which], leaves, (dh, dfinal)[which])
        ref = [t.detach().double().requires_grad_() for t in (x, g, state)]
        s, rows = ref[2], []
        for t in range(length):
            a = torch.sigmoid(ref[1][:, t])
            s = a * s + (1 - a) * ref[0][:, t]
            rows.append(s)
        want = torch.autograd.grad((torch.stack(rows, 1), s)[which], ref, (dh, dfinal)[which].double())
        for p, r in zip(got, want):
            # dstate is a product of `length` values a, each right to d = 2^-21 + |g| 2^-23 (|g| < 8 here)
            assert float((p.double() - r).norm() / r.norm()) <= length * (2.0 ** -21 + 8 * 2.0 ** -23)
    frozen = sla.gated_scan(x, g.detach(), None)[0]
    assert torch.autograd.grad(frozen.sum(), x)[0].shape == x.shape


def test_other_streams_graphs_and_shared_workspaces():
    x, g, state = inputs((2, 3000, 130), 2, torch.bfloat16, 100)
    dh = randn(2, 3000, 130, dtype=torch.bfloat16, seed=104)
    want = sla.sla_gated_scan(x, g, state, save=True)
    grads = sla.sla_gated_scan_backward(dh, x, g, want[2], None, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h, final = sla.sla_gated_scan(x, g, state)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0]) and torch.equal(final, want[1])
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)  # both graphs use it, one after another
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sla.sla_gated_scan(x, g, state, save=True, workspace=ws)
            out = (*out, *sla.sla_gated_scan_backward(dh, x, g, out[2], None, state, workspace=ws))
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out[0].zero_()
            graph.replay()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            assert all(torch.equal(p, q) for p, q in zip(out[3:], grads))
    sla.sla_gated_ffn_check()


def test_refusals():
    x = randn(4, 6, 8, dtype=torch.float16, seed=110)
    state = torch.zeros(4, 8, device=DEV)
    off = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    _, _, saved = sla.sla_gated_scan(x, x, state, save=True)
    for call, message in (
            (lambda: sla.sla_gated_scan(x[0, 0], x[0, 0]), "x must be"),
            (lambda: sla.sla_gated_scan(x, x[:, :5]), "gate must have"),
            (lambda: sla.sla_gated_scan(x, x.float()), "gate must have"),
            (lambda: sla.sla_gated_scan(x.double(), x.double()), "float32, float16"),
            (lambda: sla.sla_gated_scan(x.transpose(0, 1), x.transpose(0, 1)), "contiguous"),
            (lambda: sla.sla_gated_scan(x, x, state[:3]), "state must have"),
            (lambda: sla.sla_gated_scan(x, x, state.half()), "state must have"),
            (lambda: sla.sla_gated_scan(x, x, offsets=off), "with offsets"),
            (lambda: sla.sla_gated_scan(x[0], x[0], offsets=off.float()), "offsets must be"),
            (lambda: sla.sla_gated_scan(x[0], x[0], offsets=[0, 6]), "offsets must be"),
            (lambda: sla.sla_gated_scan(x[0], x[0], offsets=off[:0]), "offsets must be"),
            (lambda: sla.sla_gated_scan(x[0], x[0], offsets=off.cpu()), "offsets must be"),
            (lambda: sla.sla_gated_scan(x, x, h=x[:2].clone()), "h must have"),
            (lambda: sla.sla_gated_scan(x, x, final=state[:1]), "final must have"),
            (lambda: sla.sla_gated_scan_backward(x[:2], x, x, saved), "dh must have"),
            (lambda: sla.sla_gated_scan_backward(x, x, x, saved, dfinal=state[:1]), "dfinal must have"),
            (lambda: sla.sla_gated_scan_backward(x, x, x, saved.float()), "saved must be"),
            (lambda: sla.sla_gated_scan_backward(x, x, x, saved, reverse=True), "saved is from"),
            (lambda: sla.sla_gated_scan_backward(x[:2], x[:2], x[:2], saved), "saved is from")):
        with pytest.raises(ValueError, match=message):
            call()
    with pytest.raises(sla.SlaError):  # the C call's own check: a saved buffer of 16 bytes
        s = sla.scan._Scan(x, x, None, False, False)
        sla.scan._check(sla.lib().sla_gated_scan(s.ref, s.x, s.ldx, s.gate, s.ldg, None, s.x, None, s.x, 16, None, 0, 0),
                        "sla_gated_scan")
