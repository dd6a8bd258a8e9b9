"""A layer in 8 bits on the GPU against its formulas in 64 bits (oracle/layer.py), at the sizes, types, layouts and values
where rows and tiles can go wrong.

Tolerances count roundings, u = 2^-24 (half a step of fp32), half = eps / 2 of the result's type:
 - rows in 8 bits: exact, with a norm up to entries within 2^-38 of a border between two steps (127 times 2^-45 for the
   norm's arithmetic in two parts, and 2^-46 for the oracle's own).
 - the norm: y is a sum of two parts rounded to fp32 (u), then to its type (half); rstd is rounded once (u).
 - its gradient: xh = h r carries r's rounding and its own (2 u), g one; the mean of g xh is a chain of at most 16 terms, 10
   joins and 3 more roundings a term: 32 u of the mean of |g xh|. dx adds 4 roundings to each part. dweight: a chain over a
   block's rows and over the blocks' parts.
 - the product: the sum is exact, it is rounded to fp32 and two factors multiply it: 3 u, then half.
 - the gradients: sums of S products that are exact in fp32, C of them in the matrix unit (256 of an fp32 gradient, else 512
   for results in fp32 and 2048 for results of 16 bits): C / 16 accumulations, each cut off rather than rounded (2 u of what is
   held), and 17 aligned terms in a product's own: C / 8 + 34 u; then S / C + 12 additions in fp32, all of the sum of
   |products|, then u or half for the result."""
import threading

import numpy as np
import pytest
import torch

import compressed_sgd_b200 as gs
from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}   # half of the smallest step


def half(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def overflow(dtype):
    """Where rounding to the nearest leaves the type: half of its last step 2^e eps above its largest number 2^e (2 - eps)."""
    info = torch.finfo(TYPES[dtype])
    return info.max * (1 + info.eps / 2 / (2 - info.eps))


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def laid(values, dtype, stride=None, first=0, fill=float("nan")):
    """(view, buffer): a matrix with rows `stride` apart, `first` elements into a buffer whose other elements are `fill`."""
    t = torch.as_tensor(np.asarray(values)).to(dtype)
    rows, cols = t.shape
    stride = cols if stride is None else stride
    buf = torch.full((first + max(rows, 1) * stride + 32,), fill, dtype=dtype, device="cuda")
    view = buf.as_strided((rows, cols), (stride, 1), first)
    view.copy_(t)
    return view, buf


def untouched(view, buf, fill):
    """What stands around and between the rows of `view` in `buf` is still `fill`."""
    other = buf.clone()
    other.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(fill)
    assert torch.equal(torch.nan_to_num(other.float(), nan=77.0), torch.full_like(other, fill).float().nan_to_num(nan=77.0))


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), what
    fine = ~nan & ~inf
    off = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert off.size == 0 or off.max() <= 0, (what, off.max(), np.abs(got - want)[fine].max())


def normal(seed, *shape, scale=1.0):
    return (np.random.default_rng([seed, *shape]).normal(size=shape) * scale).astype(np.float32)


# rows in 8 bits ---------------------------------------------------------------------------------------

ROWS = [(1, 1), (3, 7), (1, 64), (5, 255), (4, 256), (7, 257), (9, 512), (2, 513), (3, 1001), (6, 4096), (2, 8200), (1, 16384),
        (2, 16385), (2, 32768)]


def check_quantize(x, dtype):
    rows, depth = x.shape
    q, qbuf = laid(np.full((rows, depth), 55), torch.int8, stride=-(-depth // 16) * 16 + 16, fill=55)
    r = gs.quantize_rows(x, out=gs.QuantRows(q, torch.empty(rows, device="cuda")))
    want_q, want_s = layer.quantize_rows(f64(x))
    assert np.array_equal(f64(r.scale), want_s, equal_nan=True)
    assert np.array_equal(r.q.cpu().numpy(), want_q)
    untouched(q, qbuf, 55)
    values = want_q * want_s[:, None]
    for t in ("bf16", "fp32"):
        out, buf = laid(np.zeros((rows, depth)), TYPES[t], stride=depth + 3, first=1)
        gs.dequantize_rows(r, out=out)
        assert np.array_equal(f64(out), values, equal_nan=True)   # exact in both
        untouched(out, buf, float("nan"))
    half_out = gs.dequantize_rows(r, torch.float16)
    fit = torch.as_tensor(values).to(torch.float16)
    assert np.array_equal(f64(half_out), f64(fit), equal_nan=True)
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", ROWS)
def test_quantize_sizes(dtype, rows, depth):
    for stride, first in ((depth, 0), (depth + 5, 1), (-(-depth // 8) * 8 + 8, 8)):
        x, _ = laid(normal(1, rows, depth), TYPES[dtype], stride, first)
        check_quantize(x, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_borders(dtype):
    """Halves go to even; the largest entry at 127 steps, and just above."""
    top = {"fp32": np.nextafter(np.float32(127), np.float32(128)), "bf16": 127.5, "fp16": 127.0625}[dtype]
    x = np.zeros((8, 24), np.float32)
    x[0, :8] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]
    x[1, :4] = [top, 1.0, 3.0, -1.0]
    x[2, :3] = [-127 * 2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -11]
    x[3, 5] = torch.finfo(TYPES[dtype]).max
    x[3, 6] = -torch.finfo(TYPES[dtype]).max
    x[4, 1] = torch.finfo(TYPES[dtype]).smallest_normal
    x[5, 1:3] = [TINY[dtype] * 2, -TINY[dtype] * 6]
    x[6] = -0.0
    x[7] = 1.0
    check_quantize(dev(x, TYPES[dtype]), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("depth", [5, 512, 4099])
def test_quantize_rows_without_values(dtype, bad, depth):
    x = normal(2, 5, depth)
    x[1, depth - 1] = bad
    x[3, 0] = bad
    check_quantize(dev(x, TYPES[dtype]), dtype)


def test_quantize_broadcast_rows():
    x = dev(normal(3, 1, 100), torch.bfloat16).expand(6, 100)
    r = gs.quantize_rows(x)
    want_q, want_s = layer.quantize_rows(f64(x))
    assert np.array_equal(r.q.cpu().numpy(), want_q) and np.array_equal(f64(r.scale), want_s)


def test_rows_beyond_32_bits():
    """2.2e9 entries: places past 2^31 in what is read and in what is written."""
    rows, depth = 270000, 8192
    x = torch.empty((rows, depth), dtype=torch.float16, device="cuda")
    part = dev(normal(4, 1000, depth), torch.float16)
    for a in range(0, rows, 1000):
        x[a:a + 1000] = part * (1 + a % 7)
    r = gs.quantize_rows(x)
    y = gs.dequantize_rows(r, torch.bfloat16)
    for a in (0, rows // 2 // 1000 * 1000, rows - 1000):
        want = gs.quantize_rows((part * (1 + a % 7)).contiguous())
        assert torch.equal(r.q[a:a + 1000], want.q) and torch.equal(r.scale[a:a + 1000], want.scale)
        assert torch.equal(y[a:a + 1000].float(), want.q.float() * want.scale[:, None])


# norm -------------------------------------------------------------------------------------------------

def check_norm(x, weight, dtype, residual=None, eps=1e-6, h=None):
    rows, depth = x.shape
    total = f64(x)
    if residual is not None:
        total = f64((x.float() + residual.float()).to(TYPES[dtype]))
    w = f64(weight)
    r = gs.rms_norm(x, weight, residual, eps=eps, want_y=True, want_q=True, want_rstd=True, h=h)
    torch.cuda.synchronize()
    eps = float(np.float32(eps))
    assert np.array_equal(f64(r.h), total, equal_nan=True)
    with np.errstate(all="ignore"):
        y, rstd = layer.rms_norm(total, w, eps)
        close(r.rstd, rstd, U * rstd * (1 + 2.0 ** -20), "rstd")
        fits = np.where(np.abs(y) >= overflow(dtype), np.sign(y) * np.inf, y)
        close(r.y, fits, (half(dtype) + U * 1.01) * np.abs(np.nan_to_num(y, posinf=0, neginf=0)) + TINY[dtype] * 1.01, "y")
        q, scale = layer.quantize_rows(y)
    got_s, got_q = f64(r.q.scale), r.q.q.cpu().numpy()
    assert np.array_equal(got_s, scale, equal_nan=True)
    fine = ~np.isnan(scale)
    steps = y[fine] / scale[fine][:, None]
    assert (np.abs(got_q[fine] - steps) <= 0.5 + 2.0 ** -38).all()
    assert (got_q[~fine] == 0).all()
    alone = gs.rms_norm(x if h is None else r.h, weight, residual if h is None else None, eps=eps, want_q=True)   # the same without y and rstd
    assert torch.equal(alone.q.q, r.q.q) and torch.equal(alone.q.scale.nan_to_num(7.0), r.q.scale.nan_to_num(7.0))
    return r


NORMS = [(1, 1), (3, 7), (1, 64), (5, 255), (4, 256), (7, 257), (9, 512), (2, 513), (3, 1001), (6, 4096), (2, 8200), (2, 16384)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", NORMS)
def test_norm_sizes(dtype, rows, depth):
    w = dev(1 + 0.1 * normal(5, depth))
    for stride, first in ((depth, 0), (depth + 5, 1), (-(-depth // 8) * 8 + 8, 8)):
        x, _ = laid(normal(6, rows, depth, scale=2.0), TYPES[dtype], stride, first)
        res, _ = laid(normal(7, rows, depth, scale=5.0), TYPES[dtype], stride + 1, first)
        check_norm(x, w, dtype, res)
        check_norm(x, w, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", [(9, 1), (9, 3), (17, 9), (11, 249), (9, 250), (10, 257), (9, 505), (9, 506), (9, 513), (17, 1023), (9, 3086),
                                        (9, 8191), (9, 8186), (9, 16377), (9, 16378), (9, 16383)])
def test_norm_rows_between_boundaries(dtype, rows, depth):
    """Contiguous rows of an odd length: every place between two 16-byte boundaries, in all of x, residual, h and y."""
    x, res = dev(normal(120, rows, depth, scale=2.0), TYPES[dtype]), dev(normal(121, rows, depth, scale=2.0), TYPES[dtype])
    w = dev(1 + 0.1 * normal(122, depth))
    a = check_norm(x, w, dtype, res)
    apart, _ = laid(f64(x), TYPES[dtype], stride=depth + 11, first=3)        # the same entry by entry
    b = gs.rms_norm(apart, w, res, want_y=True, want_q=True, want_rstd=True)
    assert torch.equal(a.h, b.h) and torch.equal(a.q.q, b.q.q) and torch.equal(a.q.scale, b.q.scale)
    q, buf = laid(np.full((rows, depth), 55), torch.int8, stride=-(-depth // 16) * 16 + 16, fill=55)
    h, hbuf = laid(np.zeros((rows, depth)), TYPES[dtype], stride=depth, first=16)
    gs.rms_norm(x, w, res, h=h, q=gs.QuantRows(q, torch.empty(rows, device="cuda")))
    assert torch.equal(q, a.q.q) and torch.equal(h, a.h)
    untouched(q, buf, 55)
    untouched(h, hbuf, float("nan"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", [(9, 1), (9, 7), (9, 8), (17, 15), (9, 249), (9, 257), (9, 511), (9, 5459), (9, 32761), (9, 32762), (9, 32767)])
def test_quantize_rows_between_boundaries(dtype, rows, depth):
    for stride, first in ((depth, 0), (depth, 3), (depth + 2, 5)):
        x, _ = laid(normal(123, rows, depth), TYPES[dtype], stride, first)
        check_quantize(x, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("depth", [8, 13, 700])
def test_norm_scales_at_their_border(dtype, depth):
    """The largest entry a step of fp32 or two from 127 * 2^e, on either side: the scale is the formula's."""
    rng = np.random.default_rng(124)
    for k in range(40):
        x = rng.normal(size=(1, depth)).astype(np.float32)
        x[0, depth // 2] = 2.0 + 6.0 * rng.random()
        t = dev(x, TYPES[dtype])
        h = f64(t)
        rstd = 1.0 / np.sqrt(np.mean(h * h) + float(np.float32(1e-6)))
        at = np.float32(127 * 2.0 ** rng.integers(-9, 3) / (h[0, depth // 2] * rstd))
        for step in range(-3, 4):
            w = np.full(depth, at / 64, np.float32)
            w[depth // 2] = np.float32(at + step * np.spacing(at))
            y, _ = layer.rms_norm(h, w.astype(np.float64), float(np.float32(1e-6)))
            r = gs.rms_norm(t, dev(w), want_q=True)
            assert float(r.q.scale[0]) == layer.scale_of(float(np.abs(y).max())), (k, step)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", [(16384, 2048), (30000, 200), (40000, 333)])
def test_norm_borders(dtype, rows, depth):
    """Millions of entries, some of them within 10^-8 steps of a border: 64 bits on the GPU (2^-38, as above)."""
    gen = torch.Generator(device="cuda")
    for seed in range(3):
        gen.manual_seed(seed)
        x, res = (torch.randn(rows, depth, device="cuda", generator=gen).to(TYPES[dtype]) for _ in range(2))
        w = 1 + 0.2 * torch.randn(depth, device="cuda", generator=gen)
        r = gs.rms_norm(x, w, res, eps=1e-5, want_q=True)
        h = r.h.double()
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + float(np.float32(1e-5))) * w.double()
        assert float(((r.q.q.double() - y / r.q.scale.double()[:, None]).abs() - 0.5).max()) <= 2.0 ** -38


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weight_dtype", TYPES)
@pytest.mark.parametrize("depth", [24, 1001, 2048])
def test_norm_weight_types(dtype, weight_dtype, depth):
    x, w = dev(normal(8, 4, depth), TYPES[dtype]), dev(normal(9, depth), TYPES[weight_dtype])
    check_norm(x, w, dtype, dev(normal(10, 4, depth), TYPES[dtype]), eps=1e-5)
    shifted = torch.zeros(depth + 1, dtype=TYPES[weight_dtype], device="cuda")[1:]   # no 16-byte boundary
    shifted.copy_(w)
    check_norm(x, shifted, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("depth", [8, 333, 512, 4096])
def test_norm_in_place(dtype, depth):
    x, res, w = dev(normal(11, 5, depth), TYPES[dtype]), dev(normal(12, 5, depth), TYPES[dtype]), dev(normal(13, depth))
    want = gs.rms_norm(x, w, res, want_q=True)
    for at in (0, 1):
        a, b = x.clone(), res.clone()
        r = gs.rms_norm(a, w, b, want_q=True, h=(a, b)[at])
        assert torch.equal((a, b)[at], want.h) and torch.equal(r.q.q, want.q.q) and torch.equal(r.q.scale, want.q.scale)
        assert torch.equal((b, a)[at], (res, x)[at])


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_values(dtype):
    """Zeros, the type's ends, an infinity, NaN, a single large entry; small and large eps."""
    big = float(torch.finfo(TYPES[dtype]).max)
    x = np.zeros((9, 300), np.float32)
    x[1] = normal(14, 300) * big / 16
    x[2] = normal(15, 300) * float(torch.finfo(TYPES[dtype]).smallest_normal) * 8
    x[3, 7] = big
    x[4, 8] = np.inf
    x[5, 9] = np.nan
    x[6] = 1.0
    x[7, ::2] = -1e-3
    x[8] = np.where(np.arange(300) == 150, 1e4, 1e-4)
    t = dev(x, TYPES[dtype])
    for eps in (1e-30, 1e-6, 1.0):
        check_norm(t, dev(normal(16, 300)), dtype, eps=eps)


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_sum_overflows(dtype):
    """A sum with the residual that leaves the type is an infinity: the row has no 8 bits."""
    big = float(torch.finfo(TYPES[dtype]).max)
    x = dev(np.full((2, 16), 1.0, np.float32), TYPES[dtype])
    x[1, 3] = big
    r = gs.rms_norm(x, torch.ones(16, device="cuda"), x.clone(), want_q=True, want_y=True, want_rstd=True)
    assert torch.isinf(r.h[1, 3]) and torch.isnan(r.q.scale[1]) and (r.q.q[1] == 0).all() and r.rstd[1] == 0
    assert torch.isnan(r.y[1, 3]) and (r.y[1, :3] == 0).all() and torch.isfinite(r.q.scale[0])


def grad_tolerance(h, w, eps, dy, dh, dtype, chain):
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    xh, g = h * r, dy * w
    s = np.mean(np.abs(g * xh), axis=1, keepdims=True)
    part = r * (4 * np.abs(g) + np.abs(xh) * (36 + 4) * s) * U
    dx, dw = layer.rms_norm_grad(h, w, eps, dy, dh)
    part = part + (0 if dh is None else U * np.abs(dx))
    return part + half(dtype) * (np.abs(dx) + part) * 1.01 + TINY[dtype] * 1.01, (chain + 4) * U * np.sum(np.abs(dy * xh), axis=0) + 2.0 ** -149


def check_norm_backward(h, w, dy, dh, dtype, eps=1e-6, **kw):
    H, W, DY, DH = f64(h), f64(w), f64(dy), None if dh is None else f64(dh)
    eps = float(np.float32(eps))
    rstd = dev(1.0 / np.sqrt(np.mean(H * H, axis=1) + eps))
    r = gs.rms_norm_backward(h, w, rstd, dy, dh, **kw)
    dx, dw = layer.rms_norm_grad(H, W, eps, DY, DH)
    # at most 8 rows at once in each of 148 * 4 blocks: rows after one another, then 8 in a block, then the blocks
    rows = h.shape[0]
    t_dx, t_dw = grad_tolerance(H, W, eps, DY, DH, dtype, rows / 148 + 8 + 148 * 4 / 32 + 6)
    close(r.dx, dx, t_dx, "dx")
    if r.dweight is not None:
        close(r.dweight, dw, t_dw, "dweight")
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,depth", NORMS + [(1500, 40), (700, 512), (5000, 130), (333, 2056)])
def test_norm_backward_sizes(dtype, rows, depth):
    w = dev(1 + 0.1 * normal(17, depth))
    for stride, first in ((depth, 0), (depth + 3, 1)):
        h, _ = laid(normal(18, rows, depth, scale=2.0), TYPES[dtype], stride, first)
        dy, _ = laid(normal(19, rows, depth), TYPES[dtype], stride, first)
        dh, _ = laid(normal(20, rows, depth), TYPES[dtype], stride, first)
        dx, buf = laid(np.zeros((rows, depth)), TYPES[dtype], stride, first)
        a = check_norm_backward(h, w, dy, dh, dtype, dx=dx)
        untouched(dx, buf, float("nan"))
        b = check_norm_backward(h, w, dy, None, dtype)
        assert torch.equal(a.dweight, b.dweight)     # the same sums in the same order
        assert torch.equal(gs.rms_norm_backward(h, w, dev(1.0 / np.sqrt(np.mean(f64(h) ** 2, axis=1) + float(np.float32(1e-6)))), dy,
                                                want_dweight=False).dx, b.dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weight_dtype", TYPES)
@pytest.mark.parametrize("which", ["h", "dy", "dh"])
def test_norm_backward_in_place(dtype, weight_dtype, which):
    t = {k: dev(normal(21 + i, 30, 520), TYPES[dtype]) for i, k in enumerate(("h", "dy", "dh"))}
    w = dev(normal(24, 520), TYPES[weight_dtype])
    rstd = torch.rsqrt(t["h"].float().square().mean(-1) + 1e-6)
    want = gs.rms_norm_backward(t["h"], w, rstd, t["dy"], t["dh"])
    r = gs.rms_norm_backward(t["h"], w, rstd, t["dy"], t["dh"], dx=t[which])
    assert torch.equal(t[which], want.dx) and torch.equal(r.dweight, want.dweight)


def test_norm_backward_without_rows():
    h, w = torch.empty((0, 16), device="cuda"), torch.ones(16, device="cuda")
    r = gs.rms_norm_backward(h, w, torch.empty(0, device="cuda"), h)
    assert r.dx.shape == (0, 16) and (r.dweight == 0).all()


# the product ------------------------------------------------------------------------------------------

def quants(seed, rows, depth, pad=0, spread=6):
    """Rows in 8 bits of every value, with scales apart by powers of two."""
    rng = np.random.default_rng([seed, rows, depth])
    q, _ = laid(rng.integers(-127, 128, (rows, depth)), torch.int8, stride=-(-depth // 16) * 16 + pad, fill=99)
    scale = 2.0 ** rng.integers(-spread, spread + 1, rows)
    return gs.QuantRows(q, dev(scale))


def status_ok(st):
    torch.cuda.synchronize()
    assert int(st.item()) == 0


def check_product(x, w, dtype, stride=None, first=0):
    tokens, channels = x.q.shape[0], w.q.shape[0]
    out, buf = laid(np.zeros((tokens, channels)), TYPES[dtype], stride, first)
    st = gs.status_tensor()
    gs.linear_q8(x, w, out=out, d_status=st)
    status_ok(st)
    with np.errstate(all="ignore"):
        want = layer.linear(x.q.cpu().numpy(), f64(x.scale), w.q.cpu().numpy(), f64(w.scale))
        wide = np.abs(want) >= overflow(dtype)
        tol = (3 * U * 1.01 + half(dtype) * 1.01) * np.abs(want) + 1.01 * TINY[dtype]
        close(out, np.where(wide, np.sign(want) * np.inf, want), np.where(wide | np.isnan(want), 0, tol), "out")
    untouched(out, buf, float("nan"))
    return out


SIZES = [(1, 1, 1), (1, 5, 16), (2, 7, 15), (3, 100, 33), (5, 16, 64), (8, 129, 100), (9, 130, 512), (16, 1000, 31), (17, 255, 128),
         (64, 64, 127), (65, 300, 129), (127, 257, 256), (128, 256, 48), (129, 511, 257), (200, 128, 1001), (255, 513, 160),
         (256, 256, 1024), (257, 260, 130), (300, 77, 4096), (520, 1030, 272), (33, 2500, 512), (4, 600, 8192), (1, 85, 32768),
         (12, 90, 32768)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,depth", SIZES)
def test_product_sizes(dtype, tokens, channels, depth):
    x, w = quants(30, tokens, depth), quants(31, channels, depth, pad=16)
    check_product(x, w, dtype, stride=-(-channels // 8) * 8)            # rows at 16-byte boundaries
    check_product(x, w, dtype)
    check_product(x, w, dtype, stride=channels + 3, first=1)


@pytest.mark.parametrize("tokens", [1, 3, 8, 12, 150])
def test_product_extremes(tokens):
    """-128 and 127 in every place of the longest rows: the sums' ends."""
    depth, channels = 32768, 6
    rng = np.random.default_rng(32)
    xq = rng.choice([-128, 127], (tokens, 1)) * np.ones((1, depth))
    wq = rng.choice([-128, 127], (channels, 1)) * np.ones((1, depth))
    x, w = (gs.QuantRows(dev(q, torch.int8), dev(2.0 ** np.arange(q.shape[0]) / 2 ** (q.shape[0] // 2))) for q in (xq, wq))
    if tokens < 100:
        check_product(x, w, "fp32")
        check_product(x, w, "bf16")
    y = gs.linear_q8(gs.QuantRows(x.q, torch.ones(tokens, device="cuda")), gs.QuantRows(w.q, torch.ones(channels, device="cuda")), torch.float32)
    assert torch.equal(y.double().cpu(), torch.as_tensor(xq @ wq.T).to(torch.float32).double())


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_scales(dtype, tokens):
    """Scales that are no powers of two, 0, NaN, infinite; results beyond the type."""
    x, w = quants(33, tokens, 200), quants(34, 50, 200)
    x = gs.QuantRows(x.q, dev(np.random.default_rng(3).uniform(0.1, 3, tokens)))
    w = gs.QuantRows(w.q, dev(np.random.default_rng(4).uniform(0.1, 3, 50)))
    check_product(x, w, dtype)
    x.scale[1] = float("nan")
    w.scale[3], w.scale[4], w.scale[5] = 0.0, float("inf"), 2.0 ** 90
    x.scale[0] = 2.0 ** 20
    x.q[0] = 1
    w.q[4] = 1
    w.q[5] = 1
    check_product(x, w, dtype)


def test_product_single_rows_have_no_stride():
    """One row whose stride says nothing, as slices and views have them."""
    x, w = quants(35, 4, 100), quants(36, 20, 100)
    one = gs.QuantRows(x.q[2:3], x.scale[2:3].clone())
    assert torch.equal(gs.linear_q8(one, w, torch.float32), gs.linear_q8(x, w, torch.float32)[2:3])
    odd = gs.QuantRows(x.q[2:3].as_strided((1, 100), (1, 1)), one.scale)
    assert torch.equal(gs.linear_q8(odd, w, torch.float32), gs.linear_q8(x, w, torch.float32)[2:3])


def test_product_layout():
    x, w = quants(37, 9, 64), quants(38, 1001, 64)
    out = gs.linear_q8(x, w)
    assert out.shape == (9, 1001) and out.stride(0) == 1008 and out.dtype is torch.bfloat16
    assert gs.linear_q8(x, quants(38, 1008, 64), torch.float16).is_contiguous()
    assert gs.linear_q8(x, quants(38, 1000, 64), torch.float32).is_contiguous()


@pytest.mark.parametrize("tokens", [1, 7, 300])
def test_product_shares_rows(tokens):
    """A stride of 0: every token the same row."""
    one = quants(39, 1, 96)
    x = gs.QuantRows(one.q.as_strided((tokens, 96), (0, 1)), one.scale.expand(tokens).contiguous())
    if tokens == 1:
        assert gs.linear_q8(x, quants(40, 33, 96)).shape == (1, 33)
    else:
        with pytest.raises(gs.GsparseError, match="invalid argument"):   # rows in 8 bits are rows of their own
            gs.linear_q8(x, quants(40, 33, 96))


# its gradients ------------------------------------------------------------------------------------------

def sums_tolerance(size, terms, dtype, want, gradient="bf16"):
    """size: the sum of |products|; gradient: the type of dout."""
    unit = 256 if gradient == "fp32" else 512 if dtype == "fp32" else 2048
    part = (unit / 8 + 34 + terms / unit + 12) * U * size
    return part + half(dtype) * (np.abs(want) + part) * 1.01 + 1.01 * TINY[dtype]


def gradient(seed, tokens, channels):
    """As a loss over the channels makes it: many small entries, one near -1; padding."""
    rng = np.random.default_rng([seed, tokens, channels])
    p = np.exp(2.0 * rng.normal(size=(tokens, channels)))
    p /= p.sum(1, keepdims=True)
    p[np.arange(tokens), rng.integers(channels, size=tokens)] -= 1.0
    p[3::10] = 0.0
    return (64.0 * p).astype(np.float32)


def check_gradients(dout, x, w, dtype, dx_dtype=None):
    tokens, channels = dout.shape
    depth = x.q.shape[1]
    g = f64(dout)
    xq, xs, wq, ws = x.q.cpu().numpy(), f64(x.scale), w.q.cpu().numpy(), f64(w.scale)
    st = gs.status_tensor()
    dx_dtype = dtype if dx_dtype is None else dx_dtype
    dx, buf = laid(np.zeros((tokens, depth)), TYPES[dx_dtype], stride=depth + 1)
    gs.linear_q8_grad_input(dout, w, out=dx, d_status=st)
    even = gs.linear_q8_grad_input(dout, w, dtype=TYPES[dx_dtype], d_status=st)
    dw, wbuf = laid(np.zeros((channels, depth)), torch.float32, stride=depth + 1, first=1)
    gs.linear_q8_grad_weight(dout, x, out=dw, d_status=st)
    flat = gs.linear_q8_grad_weight(dout, x, d_status=st)
    status_ok(st)
    assert torch.equal(dx, even) and torch.equal(dw, flat) and flat.is_contiguous()
    untouched(dx, buf, float("nan"))
    untouched(dw, wbuf, float("nan"))
    planes = {"bf16": 1, "fp16": 2, "fp32": 3}[dtype]
    want = layer.linear_grad_input(g, wq, ws)
    assert (np.abs(want) < overflow(dx_dtype)).all()
    close(dx, want, sums_tolerance(layer.linear_grad_input(np.abs(g), np.abs(wq.astype(float)), ws), planes * channels, dx_dtype, want, dtype), "dx")
    want = layer.linear_grad_weight(g, xq, xs)
    close(dw, want, sums_tolerance(layer.linear_grad_weight(np.abs(g), np.abs(xq.astype(float)), xs), planes * tokens, "fp32", want, dtype), "dweight")
    return flat


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,depth", [s for s in SIZES if s[2] < 32768] + [(1, 5000, 64), (2100, 100, 80), (700, 3000, 40)])
def test_gradient_sizes(dtype, tokens, channels, depth):
    x, w = quants(41, tokens, depth, spread=3), quants(42, channels, depth, pad=16, spread=3)
    values = gradient(43, tokens, channels)
    if dtype == "fp16":
        values /= 256                                  # results within the type
    for stride, first in ((-(-channels // 8) * 8, 0), (channels + 3, 1)):
        dout, _ = laid(values, TYPES[dtype], stride, first)
        check_gradients(dout, x, w, dtype)


@pytest.mark.parametrize("tokens,channels,depth", [(2500, 2700, 96), (2300, 2900, 8192), (5000, 700, 300), (700, 5000, 520)])
def test_product_of_many_tiles(tokens, channels, depth):
    """More tiles than pairs of SMs, in several bands either way, the last ones split or not: against 64 bits on the GPU."""
    x, w = quants(63, tokens, depth, spread=2), quants(64, channels, depth, spread=2)
    st = gs.status_tensor()
    out = gs.linear_q8(x, w, torch.float32, d_status=st)
    status_ok(st)
    want = (x.q.double() * x.scale.double()[:, None]) @ (w.q.double() * w.scale.double()[:, None]).t()
    assert bool(((out.double() - want).abs() <= 1.01 * U * want.abs()).all())      # powers of two: one rounding


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,channels,depth", [(2500, 2700, 2816), (1500, 5000, 700), (5000, 1500, 264)])
def test_gradients_of_many_tiles(dtype, tokens, channels, depth):
    x, w = quants(65, tokens, depth, spread=2), quants(66, channels, depth, spread=2)
    dout = dev(gradient(67, tokens, channels) / 64, TYPES[dtype])
    st = gs.status_tensor()
    dx, dw = gs.linear_q8_grad_input(dout, w, dtype=torch.float32, d_status=st), gs.linear_q8_grad_weight(dout, x, d_status=st)
    status_ok(st)
    g, xv, wv = dout.double(), x.q.double() * x.scale.double()[:, None], w.q.double() * w.scale.double()[:, None]
    planes = {"bf16": 1, "fp16": 2, "fp32": 3}[dtype]
    for got, want, size, terms in ((dx, g @ wv, g.abs() @ wv.abs(), channels), (dw, g.t() @ xv, g.t().abs() @ xv.abs(), tokens)):
        close(got, f64(want), sums_tolerance(f64(size), planes * terms, "fp32", f64(want), dtype), "gradient")


@pytest.mark.parametrize("dtype,dx_dtype", [("bf16", "fp32"), ("fp32", "bf16"), ("fp16", "fp32")])
def test_gradient_input_types(dtype, dx_dtype):
    x, w = quants(44, 140, 300), quants(45, 90, 300)
    check_gradients(dev(gradient(46, 140, 90), TYPES[dtype]), x, w, dtype, dx_dtype)


def test_gradient_fp32_is_whole():
    """fp32 gradients keep their 24 bits: entries that bf16 and two of it would cut."""
    dout = dev(np.array([[1.0 + 2.0 ** -23, 1.0 + 2.0 ** -16], [-(1.0 + 2.0 ** -8), 2.0 ** -30]]))
    q, _ = laid([[1], [0]], torch.int8, stride=16, fill=7)
    x = w = gs.QuantRows(q, torch.ones(2, device="cuda"))
    assert gs.linear_q8_grad_weight(dout, x).flatten().tolist() == [1.0 + 2.0 ** -23, 1.0 + 2.0 ** -16]
    assert gs.linear_q8_grad_input(dout, w).flatten().tolist() == [1.0 + 2.0 ** -23, -(1.0 + 2.0 ** -8)]


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_infinities(dtype):
    """An infinite or NaN gradient reaches what it is multiplied with, and nothing else."""
    dout = dev(gradient(47, 20, 30), TYPES[dtype])
    dout[2, 4], dout[5, 7] = float("inf"), float("nan")
    x, w = quants(48, 20, 70), quants(49, 30, 70)
    x.q[2, :], w.q[4, :] = 3, -5
    dx, dw = gs.linear_q8_grad_input(dout, w, dtype=torch.float32), gs.linear_q8_grad_weight(dout, x)
    assert (dx[2] == -float("inf")).all() and torch.isnan(dx[5]).all() and torch.isfinite(dx[[0, 1, 3, 4] + list(range(6, 20))]).all()
    assert (dw[4] == float("inf")).all() and torch.isnan(dw[7]).all() and torch.isfinite(dw[[0, 1, 2, 3, 5, 6] + list(range(8, 30))]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_rows_without_values(dtype):
    """A checkpoint's row of NaN (it held an infinity) is NaN in every weight; zeros and the smallest scale add nothing."""
    x = dev(normal(50, 40, 65))
    x[3] = 0.0
    x8, w8 = gs.quantize_rows(x), quants(51, 30, 65)
    dout = dev(gradient(52, 40, 30) / 16, TYPES[dtype])
    check_gradients(dout, x8, w8, dtype, "fp32")
    x[7, 2] = float("inf")
    assert torch.isnan(gs.linear_q8_grad_weight(dout, gs.quantize_rows(x))).all()


def test_gradient_scales_that_are_no_powers_of_two():
    """The 8-bit operand's values are rounded to bf16: half a step of it, 2^-8... of each product's second factor."""
    x = quants(53, 50, 64)
    x = gs.QuantRows(x.q, dev(np.random.default_rng(5).uniform(0.5, 2.0, 50)))
    g = gradient(54, 50, 40)
    dout = dev(g)
    want = layer.linear_grad_weight(g.astype(np.float64), x.q.cpu().numpy(), f64(x.scale))
    size = layer.linear_grad_weight(np.abs(g.astype(np.float64)), np.abs(x.q.cpu().numpy().astype(float)), f64(x.scale))
    # q * scale is rounded to fp32 and to bf16: u + 2^-8
    close(gs.linear_q8_grad_weight(dout, x), want, (2.0 ** -8 + 100 * U) * size, "dweight")


def test_gradient_shares_rows():
    """dout with a stride of 0: the gradient of a sum over tokens."""
    g = dev(gradient(55, 1, 60), torch.bfloat16)
    x, w = quants(56, 300, 48), quants(57, 60, 48)
    check_gradients(g.expand(300, 60), x, w, "bf16", "fp32")


def test_no_tokens():
    w, x = quants(58, 9, 40), quants(59, 0, 40)
    dout = torch.empty((0, 9), device="cuda")
    out = torch.full((9, 40), 3.0, device="cuda")
    assert (gs.linear_q8_grad_weight(dout, x, out=out) == 0).all()
    assert gs.linear_q8_grad_input(dout, w).shape == (0, 40) and gs.linear_q8(x, w).shape == (0, 9)


def test_products_beyond_32_bits():
    """2.4e9 results and gradients: places past 2^31."""
    tokens, channels, depth = 60001, 40008, 32
    x, w = quants(60, tokens, depth), quants(61, channels, depth)
    out = gs.linear_q8(x, w)
    for rows in (slice(0, 3), slice(tokens - 3, tokens)):
        part = gs.QuantRows(x.q[rows].contiguous(), x.scale[rows].contiguous())
        assert torch.equal(out[rows], gs.linear_q8(part, w))
    dout = out
    dx = gs.linear_q8_grad_input(dout, w, dtype=torch.float32)
    last = gs.linear_q8_grad_input(dout[-3:], w, dtype=torch.float32)
    size = f64(dout[-3:].abs()) @ np.abs(w.q.cpu().numpy().astype(float) * f64(w.scale)[:, None])
    close(dx[-3:], f64(last), 2 * (64 + 34 + channels / 512 + 13) * U * size, "dx")
    dw = gs.linear_q8_grad_weight(dout, x)
    cols = slice(channels - 4, channels)
    g = f64(dout[:, cols])
    want = layer.linear_grad_weight(g, x.q.cpu().numpy(), f64(x.scale))
    size = layer.linear_grad_weight(np.abs(g), np.abs(x.q.cpu().numpy().astype(float)), f64(x.scale))
    close(dw[cols], want, sums_tolerance(size, tokens, "fp32", want), "dweight")


# together, and the ways of calling ------------------------------------------------------------------------

def test_a_training_step_of_the_output_layer():
    """Stream, norm in 8 bits, logits, loss with its gradient, the layer's gradients from the 8 bits, the norm's gradient, and
    the compression of the weights' gradient, twice over one residual."""
    tokens, channels, depth = 150, 1001, 256
    rng = np.random.default_rng(62)
    weight = rng.normal(size=(channels, depth)).astype(np.float32) / 16
    gain = 1 + 0.1 * normal(63, depth)
    residual = torch.zeros(channels * depth, device="cuda")
    for step in range(2):
        stream, branch = (dev(normal(64 + step + 10 * i, tokens, depth), torch.bfloat16) for i in (0, 1))
        targets = dev(rng.integers(-1, channels, tokens), torch.int32)
        w8 = gs.quantize_rows(dev(weight))
        n = gs.rms_norm(branch, dev(gain), stream, want_q=True, want_rstd=True)
        logits = gs.linear_q8(n.q, w8)
        coefficient = torch.full((tokens,), -1.0, device="cuda")
        r = gs.token_logprobs(logits, targets, want_grad=True, grad_logprob=coefficient)
        assert r.dlogits.stride() == logits.stride()          # rows that the gradients take as they are
        dw = gs.linear_q8_grad_weight(r.dlogits, n.q)
        dhidden = gs.linear_q8_grad_input(r.dlogits, w8)
        back = gs.rms_norm_backward(n.h, dev(gain), n.rstd, dhidden)
        # the same in 64 bits from each link's own inputs
        q, s = layer.quantize_rows(weight.astype(np.float64))
        assert np.array_equal(w8.q.cpu().numpy(), q)
        xq, xs = n.q.q.cpu().numpy(), f64(n.q.scale)
        z = layer.linear(xq, xs, q, s)
        close(logits, z, (2.0 ** -8 + 4 * U) * np.abs(z), "logits")
        g = f64(r.dlogits)
        want = layer.linear_grad_weight(g, xq, xs)
        close(dw, want, sums_tolerance(layer.linear_grad_weight(np.abs(g), np.abs(xq.astype(float)), xs), tokens, "fp32", want), "dw")
        want = layer.linear_grad_input(g, q, s)
        close(dhidden, want, sums_tolerance(layer.linear_grad_input(np.abs(g), np.abs(q.astype(float)), s), channels, "bf16", want), "dhidden")
        want, _ = layer.rms_norm_grad(f64(n.h), gain.astype(np.float64), float(np.float32(1e-6)), f64(dhidden))
        tol, _ = grad_tolerance(f64(n.h), gain.astype(np.float64), float(np.float32(1e-6)), f64(dhidden), None, "bf16", 0)
        close(back.dx, want, tol, "dx")
        before = residual + dw.reshape(-1)
        idx, val, off = gs.residual_topk(dw.reshape(-1), residual, (1, 100))
        k = int(off[-1].item())
        assert k == gs.k_for(channels * depth, (1, 100))
        sent = torch.zeros_like(before)
        sent[idx[:k].long()] = val[:k]
        assert torch.equal(sent + residual, before)
        weight = weight - 0.1 * f64(sent).reshape(channels, depth).astype(np.float32)


def chain(x, res, gain, w, target):
    n = gs.rms_norm(x, gain, res, want_q=True, want_rstd=True)
    w8 = gs.quantize_rows(w)
    logits = gs.linear_q8(n.q, w8)
    r = gs.token_logprobs(logits, target, want_grad=True, grad_logprob=torch.ones(x.shape[0], device="cuda"))
    dw = gs.linear_q8_grad_weight(r.dlogits, n.q)
    dx = gs.linear_q8_grad_input(r.dlogits, w8)
    return [n.h, n.q.q, logits, r.logprob, dw, *gs.rms_norm_backward(n.h, gain, n.rstd, dx)]


def inputs(seed, tokens=130, channels=700, depth=320):
    return [dev(normal(seed, tokens, depth), torch.bfloat16), dev(normal(seed + 1, tokens, depth), torch.bfloat16),
            dev(1 + 0.1 * normal(seed + 2, depth)), dev(normal(seed + 3, channels, depth, scale=0.05)),
            dev(np.random.default_rng(seed).integers(0, channels, tokens), torch.int32)]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_same_call_gives_the_same_bits():
    args = inputs(70)
    want = chain(*args)
    for _ in range(5):
        assert same(chain(*args), want)


def test_two_streams():
    a, b = inputs(71), inputs(81, 90, 500, 512)
    want_a, want_b = chain(*a), chain(*b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(s):
            p = chain(*a)
        with torch.cuda.stream(t):
            q = chain(*b)
        got.append((p, q))
    torch.cuda.synchronize()
    assert all(same(p, want_a) and same(q, want_b) for p, q in got)


def test_two_host_threads():
    args = [inputs(72), inputs(82, 300, 257, 128)]
    want = [chain(*a) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                r = chain(*args[i])
                torch.cuda.current_stream().synchronize()
                if not same(r, want[i]):
                    wrong.append(i)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_captured_and_replayed():
    """Two graphs that live at once, replayed on new inputs in turn."""
    graphs = []
    for seed, sizes in ((73, (130, 700, 320)), (83, (5, 999, 96))):
        args = inputs(seed, *sizes)
        chain(*args)                                     # the first calls load the kernels
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(*args)
        graphs.append((g, args, out, sizes))
    for turn in range(3):
        for k, (g, args, out, sizes) in enumerate(graphs):
            new = inputs(90 + turn * 7 + k, *sizes)
            want = chain(*new)
            for a, n in zip(args, new):
                a.copy_(n)
            g.replay()
            torch.cuda.synchronize()
            assert same(out, want)


def test_calls_after_one_another_share_a_workspace():
    x, w = quants(74, 150, 200), quants(75, 900, 200)
    g = dev(gradient(76, 150, 900))
    size = max(gs.lib().gsparse_linear_q8_workspace_size(150, 900, 200),
               gs.lib().gsparse_linear_q8_grad_input_workspace_size(g.data_ptr(), 0, 900, 150, 900, 200),
               gs.lib().gsparse_linear_q8_grad_weight_workspace_size(g.data_ptr(), 0, 900, 150, 900, 200))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    want = gs.linear_q8(x, w), gs.linear_q8_grad_input(g, w), gs.linear_q8_grad_weight(g, x)
    for _ in range(3):
        got = gs.linear_q8(x, w, workspace=ws), gs.linear_q8_grad_input(g, w, workspace=ws), gs.linear_q8_grad_weight(g, x, workspace=ws)
        assert same(got, want)


def test_arguments_of_the_binding():
    x, w = quants(77, 4, 32), quants(78, 6, 32)
    bad = [
        lambda: gs.linear_q8(x, quants(78, 6, 48)), lambda: gs.linear_q8(x, w, torch.int8),
        lambda: gs.linear_q8(x, w, out=torch.empty((4, 7), device="cuda")),
        lambda: gs.linear_q8(gs.QuantRows(x.q, x.scale[:3]), w), lambda: gs.linear_q8(gs.QuantRows(x.q.float(), x.scale), w),
        lambda: gs.linear_q8_grad_input(torch.empty((4, 7), device="cuda"), w),
        lambda: gs.linear_q8_grad_weight(torch.empty((5, 6), device="cuda"), x),
        lambda: gs.linear_q8_grad_weight(torch.empty((4, 6), device="cuda"), x, out=torch.empty((6, 32), device="cuda", dtype=torch.float16)),
        lambda: gs.quantize_rows(torch.empty((4, 7), device="cuda", dtype=torch.float64)),
        lambda: gs.quantize_rows(torch.empty((4, 32), device="cuda"), out=w),
        lambda: gs.rms_norm(torch.empty((4, 32), device="cuda"), torch.empty(31, device="cuda")),
        lambda: gs.rms_norm(torch.empty((4, 32), device="cuda"), torch.empty(32, device="cuda"), torch.empty((4, 31), device="cuda")),
        lambda: gs.rms_norm(torch.empty((4, 32), device="cuda"), torch.empty(32, device="cuda"), q=w),
        lambda: gs.rms_norm(torch.empty((4, 32), device="cuda"), torch.empty(32, device="cuda"), eps=0.0),
        lambda: gs.rms_norm_backward(torch.empty((4, 32), device="cuda"), torch.empty(32, device="cuda"), torch.empty(5, device="cuda"),
                                     torch.empty((4, 32), device="cuda")),
        lambda: gs.linear_q8_grad_input(torch.empty((4, 6), device="cuda"), w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(gs.GsparseError):
            call()
