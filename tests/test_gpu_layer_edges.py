"""The layer operators where other values or another loop come in: non-finite
inputs beside a row's ragged end, many rows to a workgroup, long runs and long
rows, and gradients against differences along their own signs."""
import math

import pytest
import torch

import layer_reference as ref
import test_gpu_layer as base
from test_gpu_layer import DEV, cpu, rand, within

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("D", [34, 33])
@pytest.mark.parametrize("L", [1, 5, 16, 70, 128, 1500])
def test_glr_a_nonfinite_last_input_stays_out_of_the_parameters(L, D, gate, bad):
    """With k = 1 the last token's x enters its own h, y and dz and nothing else:
    every other gradient is the one for a finite x, whatever the row's length."""
    _, s, grad = base.glr_inputs((2, L, D, "f32", gate, False, 9, True, None), seed=11)
    dirty = dict(s, x=s["x"].clone())
    dirty["x"][:, -1] = bad
    want, got = ssd.ssd_glr_bwd(**s, **grad), ssd.ssd_glr_bwd(**dirty, **grad)
    exact = base.glr_reference(s).backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in ("dA", "dbias", "dinit", "dx", "dg"):
        assert torch.equal(got[k], want[k]), k
        within(k, got[k], exact[k], torch.float32)
    if gate:
        assert torch.equal(got["dz"][:, :-1], want["dz"][:, :-1]) and not torch.isfinite(got["dz"][:, -1]).any()
