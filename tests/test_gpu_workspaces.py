"""Workspaces that the caller brings to the solvers: one that fits is used, one that is no dense memory of the device is refused."""
import numpy as np
import pytest

from gpu_helpers import sla, t, to_dev, torch, DEV
from workloads import poisson_5pt

pytestmark = pytest.mark.gpu


def test_workspaces_of_the_solvers():
    P = poisson_5pt(12)
    A = to_dev(P)
    b = t(np.random.default_rng(1).standard_normal(P.n))
    values, rhs = A.values.repeat(2, 1), b.repeat(2, 1)
    calls = [lambda ws: sla.sla_cg_solve(A, b, workspace=ws)[0],
             lambda ws: sla.sla_cg_adjoint(A, b, b, workspace=ws)[0],
             lambda ws: sla.sla_cg_solve_batched(A, values, rhs, workspace=ws)[0],
             lambda ws: sla.sla_cg_adjoint_batched(A, values, rhs, rhs, workspace=ws)[0],
             lambda ws: sla.sla_bicgstab_solve(A, b, workspace=ws)[0],
             lambda ws: sla.sla_bicgstab_adjoint(A, b, b, workspace=ws)[0],
             lambda ws: sla.sla_eig_smallest(A, workspace=ws)[1],
             lambda ws: sla.sla_eigsh(A, 2, workspace=ws)[1]]
    n = 1 << 23
    for call in calls:
        for bad, message in ((torch.empty(n, dtype=torch.uint8), "CUDA tensor"),
                             (torch.empty(1, dtype=torch.uint8, device=DEV).expand(n), "contiguous"),
                             (torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2], "contiguous")):
            with pytest.raises(ValueError, match=message):
                call(bad)
        want = call(None)
        assert torch.equal(call(torch.empty(n, dtype=torch.uint8, device=DEV)), want)
        assert torch.equal(call(torch.empty(n // 8, dtype=torch.float64, device=DEV)), want)
