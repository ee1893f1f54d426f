"""The example that trains a network through the solve: layer norm, gated feed-forward block and adjoint together."""
import os
import sys

import numpy as np
import pytest

from gpu_helpers import sla, torch
from workloads import diffusion_dirichlet

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_matrix_of_the_cells_is_the_diffusion_matrix():
    from learned_conductivity import Diffusion
    m = 6
    k = np.random.default_rng(1).lognormal(0.0, 0.5, (m, m))
    h = np.concatenate((k[:, :1], (k[:, 1:] + k[:, :-1]) / 2, k[:, -1:]), 1)
    v = np.concatenate((k[:1], (k[1:] + k[:-1]) / 2, k[-1:]), 0)
    want = diffusion_dirichlet(m, np.concatenate((h.reshape(-1), v.reshape(-1))))
    got = Diffusion(m).matrix(torch.tensor(k, device="cuda"))
    assert np.array_equal(got.row_ptr.cpu().numpy(), want.row_ptr)
    assert np.array_equal(got.col_idx.cpu().numpy(), want.col_idx)
    np.testing.assert_allclose(got.values.cpu().numpy(), want.values, rtol=1e-14)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_through_the_solve_lowers_the_loss(dtype):
    from learned_conductivity import train
    losses, err = train(m=24, steps=40, dtype=dtype)
    assert np.isfinite(losses).all() and losses[-1] < 0.2 * losses[0]


def test_gradient_of_the_chain_against_differences():
    from learned_conductivity import ConductivityNet, Diffusion
    problem, net = Diffusion(12), ConductivityNet(width=32, hidden=48)
    b = torch.randn(144, generator=torch.Generator().manual_seed(2)).double().cuda()

    def loss():
        return (problem.matrix(torch.exp(net(problem.cells))).solve(b, rtol=1e-12, maxit=5000) ** 2).sum()

    loss().backward()
    for p in (net.w_in[0], net.w_out[1], net.norm_w[0], net.embed):
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
