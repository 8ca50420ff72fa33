"""Gradients at the ends of the value range: finite inputs whose gradients have
finite values do not pass through infinities on the way."""

import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.test_gpu_gated_ffn_backward import _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [40, 4200])
def test_large_gradients_behind_closed_gates(m):
    """dh u above fp32's range where the gate's slope is zero to fp32's precision:
    the gradient is 0 there, in a block whose other values are ordinary."""
    f, k = (128, 128) if m == 40 else (1024, 128)
    acts, wg, wu = _inputs(m, f, k, "f32", 1.0)
    dh, _, g, u = acts
    g[:, 3], g[::2, 70] = -200.0, -1e4
    dh[:, 3], dh[::2, 70] = 2.0 ** 90, 2.0 ** 10
    u[:, 3], u[::2, 70] = -2.0 ** 60, 2.0 ** 120
    got = _run(acts, wg, wu, out_dtype=torch.float32)
    assert all(torch.isfinite(t).all() for t in got)
    _check(acts, wg, wu, got, "f32")
