"""The layer in 8 bits on the GPU where its kernels change their way: against its formulas in 64 bits (oracle/layer.py), with the
tolerances that test_gpu_layer.py derives."""
import numpy as np
import pytest
import torch

import compressed_sgd_b200 as gs
from oracle import layer
from test_gpu_layer import (TINY, TYPES, U, check_norm, close, dev, f64, gradient, laid, normal, quants, status_ok, sums_tolerance,
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


def check_borders(r, weight, eps):
    """The 8 bits against the formula in 64 bits on the GPU: scales exact, steps up to 2^-38 of one (the 64 bits' own)."""
    h = r.h.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()
    top = y.abs().amax(-1)
    m, e = torch.frexp(top)
    scale = torch.ldexp(torch.ones_like(top), torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(-126, 121))
    assert torch.equal(r.q.scale.double(), scale)
    steps = (y / scale[:, None]).clamp(-127.0, 127.0)
    assert float((r.q.q.double() - steps).abs().max()) <= 0.5 + 2.0 ** -38
    return y


# the root mean square of rows whose r, and whose r w, leave the range in which an fp32 number has bits to spare
@pytest.mark.parametrize("dtype,exponent", [(d, e) for d in ("fp32", "bf16") for e in (23, 25, 60, 100, 109, 112, 116, 120, 124, -23, -25, -60, -100, -120)]
                         + [("fp16", 13), ("fp16", -12)])
@pytest.mark.parametrize("eps", [2.0 ** -120, 2.0 ** -20])
@pytest.mark.parametrize("size", [1.0, 1e-4, 2.0 ** 40])
def test_norm_of_rows_of_any_size(dtype, exponent, eps, size):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(exponent + 200)
    for rows, depth in ((1200, 1000), (700, 333), (4000, 60), (100, 9000)):
        x = (torch.randn(rows, depth, device="cuda", generator=gen).clamp(-7.5, 7.5).double() * 2.0 ** exponent).to(TYPES[dtype])
        assert bool(torch.isfinite(x).all())
        w = size * (1 + 0.2 * torch.randn(depth, device="cuda", generator=gen))
        r = gs.rms_norm(x, w, eps=eps, want_q=True, want_y=True, want_rstd=True)
        y = check_borders(r, w, eps)
        fine = y.abs() < torch.finfo(TYPES[dtype]).max
        off = (r.y.double() - y).abs() - (torch.finfo(TYPES[dtype]).eps / 2 + 1.01 * U) * y.abs() - 1.01 * TINY[dtype]
        assert not bool((off[fine] > 0.0).any())
        assert torch.equal(gs.rms_norm(x, w, eps=eps, want_y=True).y, r.y)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("depth", [8, 333, 512, 1001, 4096, 16384])
def test_norm_of_large_rows_among_others(dtype, depth):
    """Rows of any size side by side, some without values, with the residual, in place, and without h."""
    rows = 24
    x, res = (normal(204 + i, rows, depth).astype(np.float64) for i in (0, 1))
    for k in range(rows):
        x[k] *= 2.0 ** (10 * k - 112)
        res[k] *= 2.0 ** (10 * k - 112)
    x[3] = res[3] = 0.0
    x[20, depth // 2] = np.inf
    x[22, depth - 1] = np.nan
    t, s = dev(x, TYPES[dtype]), dev(res, TYPES[dtype])
    w = dev(1 + 0.1 * normal(206, depth))
    for eps in (1e-6, 2.0 ** -126):
        a = check_norm(t, w, dtype, s, eps=eps)
        check_norm(t, w, dtype, eps=eps)
        u = t.clone()
        b = gs.rms_norm(u, w, s, eps=eps, want_q=True, h=u)
        q, scale = torch.empty_like(a.q.q), torch.empty_like(a.q.scale)
        stride = -(-depth // 16) * 16
        q = torch.zeros(rows, stride, dtype=torch.int8, device="cuda")
        gs._on_device(t.device, "gsparse_rms_norm", t.data_ptr(), depth, s.data_ptr(), depth, w.data_ptr(), 0, gs._DTYPES[t.dtype], rows, depth, eps,
                      None, 0, None, 0, q.data_ptr(), stride, scale.data_ptr(), None)
        for other, sc in ((b.q.q, b.q.scale), (q[:, :depth], scale)):
            assert torch.equal(other, a.q.q) and torch.equal(sc.nan_to_num(7.0), a.q.scale.nan_to_num(7.0))
        assert torch.equal(u.nan_to_num(7.0), a.h.nan_to_num(7.0)) and bool((q[:, depth:] == 0).all())
