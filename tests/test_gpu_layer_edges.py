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


def parts_of_a_sum(products, at):
    """(dout's column, q's column): 2^24, then 1.5 in one of every 16 products, as many as `products` hold; at: another small one."""
    g, q = np.zeros(products, np.float32), np.zeros(products)
    g[5::16], q[5::16] = 1.5, 1
    g[0], q[0] = 2.0 ** 18, 64
    if at is not None:
        g[at], q[at] = 2.0 ** 15, 2
    return g, q


# The matrix unit cuts each 1.5 off a sum of 2^24, whose last bit is 2; the sums that it gives out later are added with rounding. So no
# more than the 1.5s of its first C products may be lost, and a last bit's half at each addition. (C goes by whole blocks of 64
# products: 128 for up to 7 of them, 256 for up to 31. 500 products are 8 blocks, of which 15 of 16 1.5s may be lost at C = 256: 22.5.)
@pytest.mark.parametrize("products,unit", [(300, 128), (500, 256), (600, 256), (1900, 256), (4100, 512)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_sums_leave_the_matrix_unit(dtype, products, unit):
    g, q = parts_of_a_sum(products, None)
    unit = min(unit, 256) if dtype == "fp32" else unit
    tol = 1.5 * unit / 16 + products / unit + 1
    want = float(np.sum(g.astype(np.float64) * q))
    dout, rows = dev(g[:, None] * np.ones((1, 40)), TYPES[dtype]), gs.QuantRows(dev(q[:, None] * np.ones((1, 32)), torch.int8), torch.ones(products, device="cuda"))
    assert float((gs.linear_q8_grad_weight(dout, rows).double() - want).abs().max()) <= tol
    dx = gs.linear_q8_grad_input(dout.t().contiguous(), rows, dtype=torch.float32)
    assert float((dx.double() - want).abs().max()) <= tol


@pytest.mark.parametrize("depth", [32, 32768])       # the latter has tiles that one pair sums from end to end
def test_gradient_sums_of_16_bits_leave_the_matrix_unit(depth):
    """2^24 + 2^16 lies in the middle between two bf16 numbers: 190 more, of which 48 may be lost, and it is the upper one."""
    g, q = parts_of_a_sum(2048, 1)
    g, q = np.concatenate([g, np.zeros(2000, np.float32)]), np.concatenate([q, np.zeros(2000)])
    rows = gs.QuantRows(dev(q[:, None], torch.int8).expand(4048, depth).contiguous(), torch.ones(4048, device="cuda"))
    dx = gs.linear_q8_grad_input(dev(np.ones((40, 1)) * g, torch.bfloat16), rows)
    assert bool((dx == 2.0 ** 24 + 2.0 ** 17).all())


def test_short_gradient_sums_of_16_bits_leave_the_matrix_unit():
    """The same with 27 more, of which 12 may be lost (C = 128)."""
    g, q = parts_of_a_sum(300, 1)
    rows = gs.QuantRows(dev(q[:, None] * np.ones((1, 32)), torch.int8), torch.ones(300, device="cuda"))
    dx = gs.linear_q8_grad_input(dev(np.ones((40, 1)) * g, torch.bfloat16), rows)
    assert bool((dx == 2.0 ** 24 + 2.0 ** 17).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("depth", [1001, 1024])
def test_norm_weight_gradient_in_short_chains(dtype, depth):
    """2^24 in row 0 and 0.5 in each of 2046 others. A block takes two rows, b and b + 1024: 2^24 (a half is lost) or 1. Each of the
    join's 32 warps adds 32 blocks in four chains of 8, so the chain with the 2^24 loses up to 7 ones to its last bit of 2; the
    joins of the chains and of the warps round 2 + 5 times by up to 1."""
    dy = torch.full((2047, depth), 0.5, device="cuda", dtype=TYPES[dtype])
    dy[0] = 2.0 ** 24
    ones = torch.ones((2047, depth), device="cuda", dtype=TYPES[dtype])
    r = gs.rms_norm_backward(ones, torch.ones(depth, device="cuda"), torch.ones(2047, device="cuda"), dy)
    assert float((r.dweight.double() - (2.0 ** 24 + 1023)).abs().max()) <= 0.5 + 7 + 7


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [1, 2, 3, 8, 9, 50])
def test_gradients_with_scales_that_are_no_powers_of_two(dtype, tokens):
    """Up to 8 tokens in fp32: a rounding of the scaled factor, chains of at most 4 and 8 of each of two splits, a dozen joins; then
    the 8-bit operand's values in fp32 (u) and bf16 (2^-8)."""
    x, w = quants(207, tokens, 72), quants(208, 60, 72)
    rng = np.random.default_rng(209)
    x, w = gs.QuantRows(x.q, dev(rng.uniform(0.5, 2.0, tokens))), gs.QuantRows(w.q, dev(rng.uniform(0.5, 2.0, 60)))
    dout = dev(gradient(210, tokens, 60), TYPES[dtype])
    g, xq, xs, wq, ws = f64(dout), x.q.cpu().numpy(), f64(x.scale), w.q.cpu().numpy(), f64(w.scale)
    part = 50 * U if tokens <= 8 else 2.0 ** -8 + 100 * U
    close(gs.linear_q8_grad_weight(dout, x), layer.linear_grad_weight(g, xq, xs), part * layer.linear_grad_weight(np.abs(g), np.abs(xq.astype(float)), xs),
          "dweight")
    close(gs.linear_q8_grad_input(dout, w, dtype=torch.float32), layer.linear_grad_input(g, wq, ws),
          part * layer.linear_grad_input(np.abs(g), np.abs(wq.astype(float)), ws), "dx")
