"""Linear layers, gated scan, residual norm and gated feed-forward block together, as a network calls them.

Tolerance, relative L2 of each result against the same network in 64 bits: float32 adds up the parts' (5e-6 a linear layer, less
for the others; seven of them, and the norms' factors below two): 5e-5.  16-bit data is rounded at about 24 places on the way
through and back, each by at most U and independent of the others: sqrt(24) U, twice that for what the norms and gates
make of it.
"""
import os
import sys
import threading

import pytest

from gpu_helpers import sla, torch, DEV

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

F = torch.nn.functional
TOL = {torch.float32: 5e-5, torch.float16: 2 * 24 ** 0.5 * 2.0 ** -11, torch.bfloat16: 2 * 24 ** 0.5 * 2.0 ** -8}


def randn(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def weights(width, hidden, dtype, seed=1):
    return [randn(2 * width, width, dtype=dtype, seed=seed, scale=width ** -0.5),
            torch.cat((torch.zeros(width, device=DEV), torch.full((width,), 2.0, device=DEV))).to(dtype),
            randn(width, width, dtype=dtype, seed=seed + 1, scale=width ** -0.5),
            randn(width, width, dtype=dtype, seed=seed + 2, scale=width ** -0.5),
            randn(width, dtype=torch.float32, seed=seed + 3, scale=0.1, shift=0.5),
            randn(width, dtype=torch.float32, seed=seed + 4, scale=0.1, shift=1.0),
            randn(width, dtype=torch.float32, seed=seed + 5, scale=0.1),
            randn(2 * hidden, width, dtype=dtype, seed=seed + 6, scale=width ** -0.5),
            randn(width, hidden, dtype=dtype, seed=seed + 7, scale=hidden ** -0.5)]


def network(z, y, state, p, offsets=None, reverse=False):
    """A mixing block and a feed-forward block: (residual stream, normed, states)."""
    w, b, w_gate, w_back, scale, nw, nb, w_in, w_out = p
    x, g = sla.linear(y, w, b).chunk(2, -1)
    h, final = sla.gated_scan(x, g, state, offsets, reverse)
    z, y = sla.residual_norm(sla.linear(h, w_back), z, sla.linear(y, w_gate, activation="silu"), scale, nw, nb, nw, nb,
                             norm="rms", gate_activation="sigmoid")
    z = sla.linear(sla.gated_ffn(y, w_in, w_out), w_back, residual=z)
    return z, sla.layer_norm(z, nw, nb), final


def network64(z, y, state, p, marks, reverse):
    w, b, w_gate, w_back, scale, nw, nb, w_in, w_out = p

    def rms(t):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-5) * nw + nb

    x, g = F.linear(y, w, b).chunk(2, -1)
    rows, final = [None] * x.shape[0], []
    for i, (p0, p1) in enumerate(zip(marks[:-1], marks[1:])):
        s = state[i]
        for t in (range(p1 - 1, p0 - 1, -1) if reverse else range(p0, p1)):
            s = s + torch.sigmoid(-g[t]) * (x[t] - s)
            rows[t] = s
        final.append(s)
    h = torch.stack(rows)
    z = z + scale * torch.sigmoid(F.silu(F.linear(y, w_gate))) * rms(F.linear(h, w_back))
    y = rms(z)
    g, u = F.linear(y, w_in).chunk(2, -1)
    z = F.linear(F.linear(F.silu(g) * u, w_out), w_back) + z
    return z, F.layer_norm(z, z.shape[-1:], nw, nb, 1e-5), torch.stack(final)


@pytest.mark.parametrize("dtype", list(TOL))
@pytest.mark.parametrize("width,hidden,marks,reverse", [(64, 128, [0, 150, 300], False), (50, 70, [0, 1, 1, 200, 333], True),
                                                        (48, 40, [0, 1, 2, 3], False)])
def test_a_training_step(width, hidden, marks, reverse, dtype):
    n, q = marks[-1], len(marks) - 1
    p = weights(width, hidden, dtype)
    z, y = randn(n, width, dtype=dtype, seed=20), randn(n, width, dtype=dtype, seed=21)
    state = randn(q, width, dtype=torch.float32, seed=22)
    ups = [randn(n, width, dtype=dtype, seed=23), randn(n, width, dtype=dtype, seed=24),
           randn(q, width, dtype=torch.float32, seed=25)]
    offsets = torch.tensor(marks, dtype=torch.int32, device=DEV)
    leaves = [t.clone().requires_grad_() for t in (z, y, state, *p)]
    out = network(*leaves[:3], leaves[3:], offsets, reverse)
    got = [*out, *torch.autograd.grad(out, leaves, ups)]
    ref = [t.detach().double().cpu().requires_grad_() for t in leaves]
    want = network64(*ref[:3], ref[3:], marks, reverse)
    want = [*want, *torch.autograd.grad(want, ref, [t.double().cpu() for t in ups])]
    for i, (a, r) in enumerate(zip(got, want)):
        err = float((a.detach().double().cpu() - r.detach()).norm() / r.detach().norm())
        assert err <= TOL[dtype], (i, err)
    sla.sla_gated_ffn_check()


def test_step_by_step_from_a_graph():
    # serving: one row of each sequence at a time, the state kept in place, every step a replay of one graph
    width, q, steps, dtype = 64, 6, 9, torch.bfloat16
    p = weights(width, 96, dtype)
    z, y = randn(steps, q, width, dtype=dtype, seed=30), randn(steps, q, width, dtype=dtype, seed=31)
    w, b, w_gate, w_back, scale, nw, nb, _, _ = p

    def block(z, y, state, final):
        both = sla.sla_linear(y, w, b).view(q, 1, 2 * width)
        h, _ = sla.sla_gated_scan(both[..., :width], both[..., width:], state, final=final)
        return sla.sla_residual_norm(sla.sla_linear(h.view(q, width), w_back), z, sla.sla_linear(y, w_gate), scale, nw, nb, nw,
                                     nb, gate_activation="sigmoid")

    state, want = torch.zeros(q, width, device=DEV), []
    for t in range(steps):
        want.append([r.clone() for r in block(z[t], y[t], state, state)])
    zin, yin, kept = torch.empty_like(z[0]), torch.empty_like(y[0]), torch.zeros(q, width, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(zin, yin, kept, kept)
    kept.zero_()
    for t in range(steps):
        zin.copy_(z[t])
        yin.copy_(y[t])
        graph.replay()
        assert all(torch.equal(a, r) for a, r in zip(out, want[t]))
    assert torch.equal(kept, state)


def test_several_calls_at_once():
    # long scans, whose blocks wait for one another, and products on several streams from several threads
    dtype, width = torch.bfloat16, 64
    p = weights(width, 128, dtype)
    data = [(randn(60000, width, dtype=dtype, seed=40 + i), randn(60000, width, dtype=dtype, seed=50 + i)) for i in range(3)]
    offsets = torch.tensor([0, 59000, 60000], dtype=torch.int64, device=DEV)
    want = [network(z, y, None, p, offsets) for z, y in data]
    torch.cuda.synchronize()
    found = [[] for _ in data]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(6):
                found[i].append(network(*data[i], None, p, offsets))
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, many in zip(want, found):
        assert len(many) == 6
        for got in many:
            assert all(torch.equal(a, r) for a, r in zip(got, w))
    sla.sla_gated_ffn_check()


def test_an_expired_wait_is_reported_by_the_next_call():
    x, w = randn(40, 32, dtype=torch.bfloat16, seed=60), randn(16, 32, dtype=torch.bfloat16, seed=61)
    for call in (lambda: sla.sla_linear(x, w), lambda: sla.sla_gated_scan(x, x)):
        call()
        torch.cuda.synchronize()
        sla.sla_test_expire_wait()
        torch.cuda.synchronize()
        with pytest.raises(sla.SlaError, match="TIMEOUT"):
            call()
        call()
    sla.sla_gated_ffn_check()
    # (autograd's thread hears of it too)
    loss = sla.linear(x.clone().requires_grad_(), w).sum()
    try:
        loss.backward()
    except sla.SlaError:
        pass


def test_the_example_with_mixing():
    from learned_conductivity import ConductivityNet, Diffusion, train
    losses, err = train(m=16, steps=3, mixing=True)
    assert len(losses) == 3 and all(map(lambda v: v == v and abs(v) < float("inf"), losses))
    problem, net = Diffusion(12), ConductivityNet(width=32, hidden=48, mixing=True)
    b = torch.randn(144, generator=torch.Generator().manual_seed(2)).double().cuda()

    def loss():
        return (problem.matrix(torch.exp(net(problem.cells))).solve(b, rtol=1e-12, maxit=5000) ** 2).sum()

    loss().backward()
    mix = net.mixing[0]
    for p in (mix.w_scan, mix.b_scan, mix.w_back, mix.w_gate, mix.scale, net.w_in[1], net.embed, net.head):
        v = torch.randn(p.shape, generator=torch.Generator().manual_seed(3)).cuda()
        v /= v.norm()
        h, f = 1e-2, []
        with torch.no_grad():
            start = p.clone()
            for sign in (1, -1):
                p.copy_(start + sign * h * v)
                f.append(float(loss()))
            p.copy_(start)
        d, g = (f[0] - f[1]) / (2 * h), float((p.grad.double() * v.double()).sum())
        # h^2 of the third derivative, and float32 rounding of the network (1e-6 of the loss) over h
        assert abs(d - g) <= 2e-3 * float(p.grad.norm()) + 2e-4 * f[0], (d, g)


def test_a_training_step_from_a_graph():
    dtype, width, n = torch.bfloat16, 64, 600
    p = weights(width, 96, dtype)
    data = [randn(n, width, dtype=dtype, seed=70), randn(n, width, dtype=dtype, seed=71),
            randn(2, width, dtype=torch.float32, seed=72)]
    offsets = torch.tensor([0, 250, n], dtype=torch.int32, device=DEV)
    up = randn(n, width, dtype=dtype, seed=73)

    def step(leaves):
        z, y, final = network(*leaves[:3], leaves[3:], offsets)
        return [z, y, final, *torch.autograd.grad([z, y], leaves, [up, up])]

    want = [t.detach().clone() for t in step([t.clone().requires_grad_() for t in (*data, *p)])]
    leaves = [t.clone().requires_grad_() for t in (*data, *p)]  # of the graph alone
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves)
    for _ in range(3):
        for t in out:
            t.detach().zero_()
        graph.replay()
        assert all(torch.equal(a, r) for a, r in zip(out, want))
    sla.sla_gated_ffn_check()


def test_arrays_of_more_than_2_31_elements():
    # the last rows of large arrays against a call on them alone
    width, dtype, tail = 64, torch.bfloat16, 5000
    n = (1 << 31) // width + 7 * tail
    base = randn(1 << 16, width, dtype=dtype, seed=80)
    x = base.repeat(n // (1 << 16) + 1, 1)[:n]
    last = x[-tail:].clone()
    w, b = randn(width, width, dtype=dtype, seed=81, scale=width ** -0.5), randn(width, dtype=dtype, seed=82)
    y = sla.sla_linear(x, w, b, residual=x)
    assert torch.equal(y[-tail:], sla.sla_linear(last, w, b, residual=last))
    del y
    z, y, stats = sla.sla_residual_norm(x, x, scale=b, weight=b, stats=True)
    z1, y1, stats1 = sla.sla_residual_norm(last, last, scale=b, weight=b, stats=True)
    assert torch.equal(z[-tail:], z1) and torch.equal(y[-tail:], y1) and torch.equal(stats[-tail:], stats1)
    del z, y
    g = sla.sla_residual_norm_backward(x, x, x, x, stats, scale=b, weight=b, want_grad_params=False)
    g1 = sla.sla_residual_norm_backward(last, last, last, last, stats1, scale=b, weight=b, want_grad_params=False)
    assert torch.equal(g.block[-tail:], g1.block) and torch.equal(g.z[-tail:], g1.z)
    del g, stats
    # tiles (one long sequence before the last) and walks (sequences of `tail` rows); the last sequence has the same rows, but
    # tiles of others: float32 steps apart, a rounding of the result
    for how in (dict(offsets=torch.tensor([0, n - tail, n], dtype=torch.int64, device=DEV)), dict()):
        rows = x if how else x[n % tail:].view(-1, tail, width)
        h, final, saved = sla.sla_gated_scan(rows, rows, save=True, **how)
        h1, final1, saved1 = sla.sla_gated_scan(last, last, save=True)
        flat = h.view(-1, width)
        assert float((final[-1:] - final1).abs().max()) <= 2.0 ** -18
        assert float((flat[-tail:].float() - h1.float()).abs().max()) <= 2.0 ** -7 * float(h1.abs().max())
        dx, dg, _ = sla.sla_gated_scan_backward(rows, rows, rows, saved, **how)
        dx1, dg1, _ = sla.sla_gated_scan_backward(last, last, last, saved1)
        for a, r in ((dx, dx1), (dg, dg1)):
            assert float((a.view(-1, width)[-tail:].float() - r.float()).abs().max()) <= 2.0 ** -7 * float(r.abs().max())
        del h, saved, flat, dx, dg
    sla.sla_gated_ffn_check()
