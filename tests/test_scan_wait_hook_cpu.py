"""Arguments of the scan's test hook, without a GPU."""
import pytest

from differentiable_sparse_iterative_gb300 import _abi, build as sla_build

torch = pytest.importorskip("torch")

import differentiable_sparse_iterative_gb300 as sla  # noqa: E402


def test_bounds_of_the_waits():
    sla_build.build()
    lib = _abi.load()
    for bad in ((2, 0), (-1, 0), (0, -1), (1, 4_000_000_001)):
        assert lib.sla_test_set_scan_wait(*bad) == _abi.SLA_INVALID_ARG
        with pytest.raises(sla.SlaError):
            sla.sla_test_set_scan_wait(*bad)
    sla.sla_test_set_scan_wait(1, 1000)
    sla.sla_test_set_scan_wait(0, 0)
