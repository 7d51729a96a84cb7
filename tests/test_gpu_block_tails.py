"""Activations and slopes of rd_block.h where they leave the range of f32.

The logistic function is 0 where its value is below 2^-126 and the normal distribution's tail where exp(-z^2 / 2) is, so a value
or slope is either as precise as elsewhere or, below what stands there, 0:

* silu: at z = -126 ln 2 the value is 87.34 * 2^-126 and the slope 86.34 * 2^-126 in size;
* tanh form: 2 sqrt(2 / pi) (z + 0.044715 z^3) is -126 ln 2 at z = -10.001, the value 10.01 * 2^-126 and the slope
  10.01 * 1.5958 * (1 + 0.13415 * 100.1) * 2^-126, 230 * 2^-126;
* gelu: z = -13.22, the value 13.22 * 0.0301 * 2^-126 and the slope 5.25 * 2^-126.
"""
import math

import numpy as np
import pytest

from oracle import block

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
TINY = 2.0 ** -126
VALUE_LOST = {block.SILU: 87.5 * TINY, block.GELU_TANH: 10.1 * TINY, block.GELU: 0.41 * TINY}
SLOPE_LOST = {block.SILU: 86.5 * TINY, block.GELU_TANH: 232 * TINY, block.GELU: 5.4 * TINY}
RANGE = {block.SILU: (-92, -78), block.GELU_TANH: (-10.6, -9), block.GELU: (-14.2, -12)}


def _arguments(kind):
    """bf16 numbers across the edge, in 64 bits, and the size of the exponential's argument at each."""
    z = torch.linspace(*RANGE[kind], 1024).to(torch.bfloat16)
    z64 = z.double().numpy()
    u = z64 * z64 / 2 if kind == block.GELU else np.abs(z64)
    if kind == block.GELU_TANH:
        u = np.abs(2 * math.sqrt(2 / math.pi) * (z64 + 0.044715 * z64 ** 3))
    return z, z64, u


def _check(got, ref, tol, lost):
    right = np.abs(got - ref) <= tol
    gone = (got == 0) & (np.abs(ref) <= lost)
    bad = ~(right | gone)
    assert not bad.any(), (got[bad][:4], ref[bad][:4])
    assert right.any() and gone.any()              # both sides of the edge are there


@pytest.mark.parametrize("kind", list(RANGE))
def test_values(rd_lib, kind):
    z, z64, u = _arguments(kind)
    x = torch.zeros(8, 8, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    w = torch.zeros(8, 1024, dtype=torch.bfloat16)
    w[0] = z
    got = rd_lib.linear(x.to(DEV), w.to(DEV), act=kind, out_dtype=torch.float32)[0].double().cpu().numpy()
    ref = block.act(z64, kind)
    # the tests' tolerance of values elsewhere; what is below 2^-126 itself has the steps of its subnormal numbers
    _check(got, ref, (2.0 ** -18 + 2.0 ** -21 * u) * np.abs(ref) + 2.0 ** -148, VALUE_LOST[kind])
    assert VALUE_LOST[kind] <= (1.1e-36 if kind == block.SILU else 1.2e-37)


@pytest.mark.parametrize("kind", list(RANGE))
def test_slopes(rd_lib, kind):
    z, z64, u = _arguments(kind)
    # one row: the bias' gradient is the slope, unrounded
    _, got = rd_lib.linear_act_bwd(torch.ones(1, 1024, device=DEV), z[None].to(DEV), kind)
    s, b = block.slope_terms(z64, kind)
    tol = (2.0 ** -18 + 2.0 ** -21 * u) * (np.abs(s) + np.abs(b)) + 2.0 ** -148
    _check(got.double().cpu().numpy(), s + b, tol, SLOPE_LOST[kind])
    assert SLOPE_LOST[kind] <= 3e-36
