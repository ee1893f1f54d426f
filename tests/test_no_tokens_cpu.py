"""Sizes of scratch and saved buffers for calls over no tokens: asked for in a process of their own, which they must not end."""
import subprocess
import sys

import pytest

from differentiable_sparse_iterative_gb300 import build as sla_build

torch = pytest.importorskip("torch")

SIZES = """
import ctypes, sys
from differentiable_sparse_iterative_gb300 import _abi
lib = _abi.load()
for dtype in (_abi.SLA_F32, _abi.SLA_F16, _abi.SLA_BF16):
    for act in range(4):
        for width, out in ((64, 64), (1, 1), (100, 3000), (2048, 8)):
            f = ctypes.byref(_abi.sla_ffn(0, width, 72, out, dtype, act))
            sizes = [lib.sla_gated_ffn_saved_bytes(f), lib.sla_gated_ffn_workspace_bytes(f),
                     lib.sla_gated_ffn_backward_workspace_bytes(f)]
            for a in (act, _abi.SLA_ACT_NONE):
                f = ctypes.byref(_abi.sla_layer(0, width, out, dtype, a))
                sizes += [lib.sla_linear_saved_bytes(f), lib.sla_linear_workspace_bytes(f),
                          lib.sla_linear_backward_workspace_bytes(f)]
            assert all(0 <= s < 1 << 32 for s in sizes), sizes
print("done")
"""


def test_sizes_for_no_tokens():
    sla_build.build()
    if torch.cuda.is_available():
        pytest.skip("asked for by every call there")
    r = subprocess.run([sys.executable, "-c", SIZES], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["done"], (r.returncode, r.stderr)
