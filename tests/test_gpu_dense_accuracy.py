"""How near the gated feed-forward block comes to its definition in 64 bits: bounds of what its roundings cost, so that one more of
them, or a longer run of products in one accumulator, is seen.

16-bit data (u = the type's unit roundoff).  Rounding a value to the type errs evenly within +-u of the power of two below
it: u / sqrt 3 of the value at most, root mean square.  Such errors do not depend on one another, and a product with
random factors keeps their relative size; k roundings one after another make u sqrt(k / 3) in relative L2:
    y: h, y -> k = 2;  dw_out: h, dw_out -> 2;  db_out: 1;  dx, dw_in, db_in: the factor kept for the backward pass, dg
    or du, the result -> 3.
float32 work (sums, activations) is below 1e-5 of that.

float32 data.  A run of 512 products in one accumulator loses up to a unit 2^-23 of its sum for every 16, half of it on
average, and the sum grows as the square root of the run: 512 / 16 * 2^-24 * 2 / 3 = 1.3e-6, always towards zero, so that
more runs make the same relative error (a run of 2,048 products makes four times as much).  Beside it: the first product,
32 or 256 long, 0.1e-6 or 0.3e-6, its activation, 0.4e-6, and the sums of the runs, 2^-24 of each of up to 38: together less
than 2.0e-6 when the independent ones add by squares.
"""
import ctypes
import math

import pytest

from gpu_helpers import sla, torch
from test_gpu_dense import ACTS, U, ffn64, ffn_inputs, randn, rel

from differentiable_sparse_iterative_gb300 import _abi

pytestmark = pytest.mark.gpu

ROUNDINGS = {"y": 2, "dx": 3, "dw_in": 3, "dw_out": 2, "db_in": 3, "db_out": 1}
RUNS = 2.0e-6


def training_step(args, dy, act):
    y, saved = sla.sla_gated_ffn(*args, activation=act, save=True)
    return (y, *sla.sla_gated_ffn_backward(dy, *args[:3], saved, activation=act, want_grad_bias=True))


def reference(args, dy, act):
    leaves = [t.double().requires_grad_() for t in args]
    y = ffn64(*leaves, act)
    return (y.detach(), *torch.autograd.grad(y, leaves, dy.double()))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("shape", [(12, 768, 2048, 768), (2049, 250, 683, 131), (4096, 256, 1024, 256), (20000, 64, 256, 64)])
def test_16_bit_block_loses_no_more_than_its_roundings(shape, act, dtype):
    args = ffn_inputs(*shape, dtype, True, seed=300)
    dy = randn(shape[0], shape[3], dtype=dtype, seed=306)
    ref = reference(args, dy, act)
    assert rel(sla.sla_gated_ffn(*args, activation=act), ref[0]) <= U[dtype] * math.sqrt(ROUNDINGS["y"] / 3)
    for (name, k), got, want in zip(ROUNDINGS.items(), training_step(args, dy, act), ref):
        assert rel(got, want) <= U[dtype] * math.sqrt(k / 3), (name, rel(got, want) / U[dtype])


def test_float32_block_of_long_sums():
    # 152 x 128 tokens, 8,192 hidden units, 256 outputs: no product is split, so that dx adds up 16,384 products, dw_in and
    # dw_out 19,456 and y 8,192, all in runs of one accumulator
    shape = tokens, width, hidden, out = 152 * 128, 32, 8192, 256
    f = _abi.sla_ffn(*shape, _abi.SLA_F32, _abi.SLA_ACT_GELU)
    packs = 6 * (tokens * width + 2 * hidden * width + out * hidden)
    runs = torch.cuda.get_device_properties(0).multi_processor_count * 128 * 128 * 4
    split = sla.lib().sla_gated_ffn_workspace_bytes(ctypes.byref(f)) - (6 * tokens * hidden + packs + runs)
    assert split == 0 or runs != 152 * 128 * 128 * 4  # sums of splits: none on this GPU
    args = ffn_inputs(*shape, torch.float32, True, seed=310)
    dy = randn(tokens, out, dtype=torch.float32, seed=316)
    errors = {name: rel(got, want) for name, got, want in
              zip(ROUNDINGS, training_step(args, dy, "gelu"), reference(args, dy, "gelu"))}
    assert max(errors.values()) <= RUNS, errors
