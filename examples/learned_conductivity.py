"""A conductivity field learned through the solve.

A network maps features of each grid cell (one token a cell) to the logarithm of its conductivity; the
cells' conductivities make the values of a five-point diffusion matrix; the matrix is solved for a few
sources; the loss compares the solutions with those of the true field.  Its gradient flows back through
the adjoint solve (grad_values = -lambda_i x_j) into the network's layer norms and gated feed-forward blocks.

With mixing, blocks that carry information from cell to cell stand between those: a linear layer makes inputs and gates of
a scan along the grid's lines, there and back, along x and along y in turn, a second one leads back to the residual stream, and
a residual norm joins the two.

    python examples/learned_conductivity.py [--mixing]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402
from workloads import poisson_5pt  # noqa: E402


class Mixing(torch.nn.Module):
    """z, y -> the residual stream and the next block's input, after scans along the lines of an m x m grid, there and back."""

    def __init__(self, width, param, device):
        super().__init__()
        # inputs and gates of the two directions; gates start open, so that a state lasts some twenty cells
        self.w_scan = param(4 * width, width, scale=width ** -0.5)
        self.b_scan = torch.nn.Parameter(torch.cat((torch.zeros(width), torch.full((width,), 3.0)) * 2).to(device,
                                                                                                         self.w_scan.dtype))
        self.w_gate = param(width, width, scale=width ** -0.5)
        self.w_back = param(width, 2 * width, scale=(2 * width) ** -0.5)
        self.scale = torch.nn.Parameter(torch.full((width,), 0.5, device=device))
        self.norms = torch.nn.ParameterList([torch.nn.Parameter(f(width, device=device))
                                             for f in (torch.ones, torch.zeros, torch.ones, torch.zeros)])

    def forward(self, z, y, m, along_x):
        width = z.shape[-1]

        def lines(t):  # [m lines][m cells of a line][..]
            t = t.view(m, m, -1)
            return t if along_x else t.transpose(0, 1)

        x0, g0, x1, g1 = lines(sla.linear(y, self.w_scan, self.b_scan)).split(width, -1)
        there, _ = sla.gated_scan(x0, g0)
        back, _ = sla.gated_scan(x1, g1, reverse=True)
        h = lines(torch.cat((there, back), -1)).reshape(m * m, 2 * width)
        w1, b1, w2, b2 = self.norms
        return sla.residual_norm(sla.linear(h, self.w_back), z, sla.linear(y, self.w_gate), self.scale, w1, b1, w2, b2,
                                 gate_activation="sigmoid")


class ConductivityNet(torch.nn.Module):
    """Fourier features of a cell's position -> residual blocks z + ffn(norm(z)) -> log conductivity."""

    def __init__(self, features=16, width=64, hidden=128, blocks=2, dtype=torch.float32, device="cuda", seed=0,
                 mixing=False):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def param(*shape, scale):
            return torch.nn.Parameter((torch.randn(*shape, generator=gen) * scale).to(device, dtype))

        self.register_buffer("freq", torch.randn(2, features, generator=gen).to(device) * 3.0)
        self.embed = param(width, 2 * features, scale=(2 * features) ** -0.5)
        self.norm_w = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width, device=device))
                                              for _ in range(blocks + 1)])
        self.norm_b = torch.nn.ParameterList([torch.nn.Parameter(torch.zeros(width, device=device))
                                              for _ in range(blocks + 1)])
        self.w_in = torch.nn.ParameterList([param(2 * hidden, width, scale=width ** -0.5) for _ in range(blocks)])
        self.w_out = torch.nn.ParameterList([param(width, hidden, scale=0.5 * hidden ** -0.5) for _ in range(blocks)])
        self.head = param(1, width, scale=0.1 * width ** -0.5)
        self.mixing = torch.nn.ModuleList([Mixing(width, param, device) for _ in range(blocks if mixing else 0)])

    def forward(self, xy):
        phase = 2.0 * math.pi * (xy @ self.freq)
        z = torch.cat((phase.sin(), phase.cos()), -1).to(self.embed.dtype) @ self.embed.t()
        if self.mixing:
            return self.forward_mixing(z, math.isqrt(xy.shape[0]))
        for i, (w_in, w_out) in enumerate(zip(self.w_in, self.w_out)):
            z = z + sla.gated_ffn(sla.layer_norm(z, self.norm_w[i], self.norm_b[i]), w_in, w_out, activation="silu")
        return (sla.layer_norm(z, self.norm_w[-1], self.norm_b[-1]) @ self.head.t()).squeeze(-1)

    def forward_mixing(self, z, m):
        y = sla.layer_norm(z, self.norm_w[0], self.norm_b[0])
        for i, (mix, w_in, w_out) in enumerate(zip(self.mixing, self.w_in, self.w_out)):
            z, y = mix(z, y, m, i % 2 == 0)
            z, y = sla.residual_norm(sla.gated_ffn(y, w_in, w_out), z, weight=self.norm_w[i + 1], bias=self.norm_b[i + 1],
                                     post_norm=False)
        return sla.linear(y, self.head).squeeze(-1)


class Diffusion:
    """Five-point diffusion on an m x m grid, Dirichlet boundary, from the cells' conductivities: an edge has the
    mean of its two cells', a boundary edge its cell's."""

    def __init__(self, m, device="cuda"):
        P = poisson_5pt(m)
        self.m = m
        self.row_ptr, self.col_idx = torch.tensor(P.row_ptr, device=device), torch.tensor(P.col_idx, device=device)
        there = torch.ones(m, m, 5, dtype=torch.bool, device=device)  # north, west, centre, east, south
        there[0, :, 0] = there[:, 0, 1] = there[:, -1, 3] = there[-1, :, 4] = False
        self.there = there.reshape(-1)
        c = (torch.arange(m, device=device) + 0.5) / m
        self.cells = torch.stack(torch.meshgrid(c, c, indexing="ij"), -1).reshape(-1, 2)

    def matrix(self, kappa):
        k = kappa.reshape(self.m, self.m).double()
        h, v = (k[:, 1:] + k[:, :-1]) / 2, (k[1:] + k[:-1]) / 2
        west, east = torch.cat((k[:, :1], h), 1), torch.cat((h, k[:, -1:]), 1)
        north, south = torch.cat((k[:1], v), 0), torch.cat((v, k[-1:]), 0)
        stencil = torch.stack((-north, -west, north + west + east + south, -east, -south), -1)
        return sla.CSRMatrix(self.row_ptr, self.col_idx, stencil.reshape(-1)[self.there])


def true_field(cells):
    x, y = cells[:, 0], cells[:, 1]
    return torch.exp(0.8 * torch.sin(2 * math.pi * x) * torch.cos(math.pi * y) - 0.5 * y)


def train(m=32, steps=80, sources=4, lr=3e-3, dtype=torch.float32, seed=0, report=None, mixing=False):
    """Returns the losses and the relative error of the learned field."""
    problem = Diffusion(m)
    gen = torch.Generator().manual_seed(seed)
    rhs = [torch.randn(m * m, generator=gen).double().cuda() for _ in range(sources)]
    target_k = true_field(problem.cells)
    with torch.no_grad():
        A = problem.matrix(target_k)
        targets = [A.solve(b, rtol=1e-10, maxit=20000) for b in rhs]
    net = ConductivityNet(dtype=dtype, seed=seed, mixing=mixing)
    opt = torch.optim.Adam(net.parameters(), lr=lr)
    losses = []
    for step in range(steps):
        opt.zero_grad()
        A = problem.matrix(torch.exp(net(problem.cells).float()))
        loss = sum(((A.solve(b, rtol=1e-8, maxit=20000) - t) ** 2).sum() / (t ** 2).sum()
                   for b, t in zip(rhs, targets)) / sources
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if report and (step % report == 0 or step == steps - 1):
            print(f"step {step:4d}  loss {losses[-1]:.3e}")
    with torch.no_grad():
        k = torch.exp(net(problem.cells).float())
    return losses, float((k - target_k).norm() / target_k.norm())


if __name__ == "__main__":
    losses, err = train(steps=200, report=20, mixing="--mixing" in sys.argv[1:])
    print(f"relative error of the field: {err:.3f}")
