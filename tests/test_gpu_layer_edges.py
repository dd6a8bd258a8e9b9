"""The layer in 8 bits on the GPU where its kernels change their way: against its formulas in 64 bits (oracle/layer.py), with the
tolerances that test_gpu_layer.py derives."""
import numpy as np
import pytest
import torch

import compressed_sgd_b200 as gs
from oracle import layer
from test_gpu_layer import (TYPES, check_norm, close, dev, f64, gradient, laid, normal, quants, status_ok, sums_tolerance,
                            untouched)

pytestmark = pytest.mark.gpu


# dout's planes as rows of one tile: as many tiles as pairs of SMs, one fewer, one more
@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("tokens", [9, 85, 128])
@pytest.mark.parametrize("channels,depth", [(300, 18688), (300, 18689), (60, 18944), (300, 18944), (2500, 18944), (300, 18945), (300, 32768)])
def test_gradient_input_of_wide_rows(dtype, tokens, channels, depth):
    w = quants(200, channels, depth, spread=3)
    dout, _ = laid(gradient(201, tokens, channels) / 256, TYPES[dtype])
    dx, buf = laid(np.zeros((tokens, depth)), TYPES[dtype], stride=depth + 1)
    st = gs.status_tensor()
    gs.linear_q8_grad_input(dout, w, out=dx, d_status=st)
    status_ok(st)
    untouched(dx, buf, float("nan"))
    g, wq, ws = f64(dout), w.q.cpu().numpy(), f64(w.scale)
    want = layer.linear_grad_input(g, wq, ws)
    planes = {"fp16": 2, "fp32": 3}[dtype]
    close(dx, want, sums_tolerance(layer.linear_grad_input(np.abs(g), np.abs(wq.astype(float)), ws), planes * channels, dtype, want, dtype), "dx")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("depth", [7, 11, 15, 1003, 1007, 4095])
def test_norm_weight_that_ends_at_its_last_entry(dtype, depth):
    """Contiguous rows of an odd length; behind the weight, in the same 16 bytes, stands something else."""
    x, buf = dev(normal(202, 9, depth, scale=2.0), TYPES[dtype]), torch.full((depth + 5,), float("nan"), device="cuda")
    w = buf[:depth]
    w.copy_(dev(1 + 0.1 * normal(203, depth)))
    check_norm(x, w, dtype)
