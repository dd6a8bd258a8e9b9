"""Losses over vocabulary rows on the GPU against their formulas in 64 bits (oracle/vocab.py), at the
sizes, types, masks, layouts and lists where a row kernel can go wrong.

Tolerances count roundings, u = 2^-24 (half a step of fp32):
 - an exponential 2^q, q = (x - M) c: the hardware's 2^q is within 4 u (its documented 2^-22), and q carries
   the roundings of c and of the product, 2 |q| u, in the exponent: ln2 * 2 |q| u relative. The entries that
   carry a softmax's weight have sum p |q| <= log2 V + entropy <= 2 log2 V.
 - a CTA's seven warps hold 7 * 32 * 2 = 448 fp32 sums, of V / 448 entries each and whole chunks of up to 16, and six
   more additions join them before 64 bits do: n u with n = max(64, V / 448 + 22).
 So log S, and with it a log probability, is within LSE(V) = (4 + 2 * 2 log2 V + n) u, plus u |result| for the
 result's own rounding; the entropy log S - T / S within LSE (2 + ln V) as T weighs the same errors by |q|.
 - a gradient p (A + B log p) + a: p is off by the exponential's error at its own q' = log2 p and by log S's,
   P(p) = (4 + 3 |log2 p| + 4 log2 V) u + LSE (the exponent is the sum of three rounded terms), the products
   and the bracket by 4 u each, a by 2 u; it is rounded once to its type (half a step, eps / 2, and where that
   type's smallest steps begin half of one).
 - a loss is summed in 64 bits: LSE (mass of q + rest <= 2) + u |loss|."""
import math

import numpy as np
import pytest
import torch

import compressed_sgd_b200 as gs
from oracle import vocab

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"fp32": 2.0 ** -126, "bf16": 2.0 ** -126, "fp16": 2.0 ** -25}   # fp32 results below 2^-126 may be flushed


def lse_tol(V):
    return (4 + 4 * math.log2(V + 1) + max(64, V / 448 + 22)) * U


def close(got, want, tol, what):
    got = got.detach().float().cpu().numpy().astype(np.float64) if torch.is_tensor(got) else got
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), what
    fine = ~nan & ~inf
    off = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert off.size == 0 or off.max() <= 0, (what, off.max(), np.abs(got - want)[fine].max())


def grad_tol(x, it, want, dtype, A, B, extra):
    """A, B, extra: sizes of the bracket's parts and of the added entries, by row, already with it."""
    V = x.shape[1]
    lp = vocab.log_softmax(x, it)
    p = np.where(np.isfinite(lp), np.exp(lp), 0.0)
    l2 = np.where(np.isfinite(lp), np.abs(lp) / math.log(2), 0.0)
    rel = (4 + 3 * l2 + 4 * math.log2(V + 1)) * U + lse_tol(V)
    size = np.abs(A)[:, None] + np.abs(B)[:, None] * (l2 * math.log(2))
    # the bracket itself: the entropy and log p carry LSE's error into it
    body = p * (size * (rel + 8 * U) + np.abs(B)[:, None] * (rel + lse_tol(V) * (2 + math.log(V + 1))))
    half = torch.finfo(TYPES[dtype]).eps / 2
    body = body + 2 * U * np.abs(extra)[:, None] * (want != 0)
    return body + half * (np.abs(want) + body) + TINY[dtype]


def make(rows, V, dtype, seed=0, scale=3.0, stride=None, first=0):
    """Logits with rows `stride` apart, the first `first` elements into a buffer whose other elements are NaN."""
    rng = np.random.default_rng([seed, rows, V])
    x = torch.from_numpy(rng.normal(size=(rows, V)).astype(np.float32) * scale).to(TYPES[dtype])
    stride = V if stride is None else stride
    buf = torch.full((first + max(rows, 1) * stride + 16,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = buf.as_strided((rows, V), (stride, 1), first)
    view.copy_(x)
    return view, buf


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a, dtype=torch.float32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def weights(rows, seed=1):
    rng = np.random.default_rng([seed, rows])
    w = rng.normal(size=(2, rows)).astype(np.float32)
    w[:, 3::7] = 0.0
    return w


def check_tokens(x, dtype, temperature=1.0, targets=None, top_k=0, grad=True, dlogits=None):
    rows, V = x.shape
    it = float(np.float32(1.0 / temperature))
    h = f64(x)
    if targets is None:
        targets = np.random.default_rng([5, rows, V]).integers(-1, V, size=rows)
    t = dev(targets, torch.int32)
    w = weights(rows)
    g, e = dev(w[0]), dev(w[1])
    st = gs.status_tensor()
    r = gs.token_logprobs(x, t, top_k=top_k, want_entropy=True, want_stats=True, temperature=temperature, want_grad=grad,
                          grad_logprob=g if grad else None, grad_entropy=e if grad else None, dlogits=dlogits, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    lp, ent, idx, val = vocab.token_logprobs(h, it, targets, top_k)
    tol = lse_tol(V)
    close(r.logprob, lp, tol + 4 * U * np.abs(np.where(np.isfinite(lp), lp, 0)), "logprob")
    close(r.entropy, ent, tol * (2 + math.log(V + 1)) + U * np.abs(np.nan_to_num(ent)), "entropy")
    if top_k:
        assert np.array_equal(r.top_idx.cpu().numpy(), idx)
        close(r.top_logprob, val, tol + 4 * U * np.abs(np.where(np.isfinite(val), val, 0)), "top_logprob")
    if grad:
        want = vocab.token_logprobs_grad(h, it, targets, w[0].astype(np.float64), w[1].astype(np.float64))
        want[(np.where(targets < 0, 0, w[0]) == 0) & (w[1] == 0)] = 0.0
        ent0 = np.nan_to_num(ent)
        tolg = grad_tol(h, it, want, dtype, it * (np.abs(w[0]) + np.abs(w[1]) * ent0), it * w[1], it * w[0])
        close(r.dlogits, want, tolg, "dlogits")
    return r


MANY = [(301, 1), (160, 3), (200, 7), (333, 9), (170, 130), (1000, 1000), (449, 1031), (300, 4099), (160, 12347), (150, 70001)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,V", MANY)
def test_tokens_many_rows(rows, V, dtype):
    """More rows than the GPU holds at once; rows at every offset from 16 bytes."""
    x, buf = make(rows, V, dtype, stride=V + 1, first=1)
    before = buf.clone()
    check_tokens(x, dtype, temperature=1.25)
    check_tokens(x, dtype, grad=False)
    other, _ = make(rows, V, dtype, stride=V + 3)            # a gradient out of step with the logits
    check_tokens(x, dtype, dlogits=other)
    assert torch.equal(torch.nan_to_num(buf.float(), 7.0), torch.nan_to_num(before.float(), 7.0))
    t = dev(np.arange(rows) % V, torch.int32)
    kw = dict(grad_logprob=dev(weights(rows)[0]), grad_entropy=dev(weights(rows)[1]))
    want = gs.token_logprobs(x, t, want_grad=True, **kw)
    got = gs.token_logprobs(x, t, dlogits=x, **kw)
    assert torch.equal(got.dlogits, want.dlogits) and torch.equal(got.logprob, want.logprob)


SIZES = [(1, 1), (3, 2), (2, 3), (5, 7), (2, 8), (3, 9), (2, 31), (1, 64), (4, 65), (2, 255), (3, 1000), (2, 1001),
         (2, 4099), (1, 16385), (2, 50021)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,V", SIZES)
def test_tokens_sizes(rows, V, dtype):
    x, _ = make(rows, V, dtype)
    check_tokens(x, dtype, top_k=min(V, 5))


@pytest.mark.parametrize("rows", [0, 1, 37, 150, 700])
def test_tokens_rows(rows):
    x, _ = make(rows, 4200, "bf16")
    check_tokens(x, "bf16", top_k=3) if rows else gs.token_logprobs(x, dev(np.zeros(0), torch.int32), top_k=3)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("stride,first", [(1003, 0), (1003, 3), (1040, 5), (1004, 1)])
def test_tokens_layouts_and_what_stands_between_rows(stride, first, dtype):
    V = 1003
    x, buf = make(5, V, dtype, stride=stride, first=first)
    before = buf.clone()
    check_tokens(x, dtype, top_k=4)
    assert torch.equal(torch.nan_to_num(buf.float(), 7.0), torch.nan_to_num(before.float(), 7.0))
    # a gradient laid out in another way, and one in the logits' place
    other, obuf = make(5, V, dtype, stride=1050, first=2)
    outside = torch.ones(obuf.numel(), dtype=torch.bool, device="cuda")
    outside.as_strided((5, V), (1050, 1), 2).fill_(False)
    check_tokens(x, dtype, dlogits=other)
    assert bool(torch.isnan(obuf[outside]).all())
    w = weights(5)
    t = dev([0, V - 1, 500, -1, 7], torch.int32)
    kw = dict(grad_logprob=dev(w[0]), grad_entropy=dev(w[1]))
    want = gs.token_logprobs(x, t, top_k=4, want_grad=True, **kw)
    got = gs.token_logprobs(x, t, top_k=4, dlogits=x, **kw)
    assert got.dlogits.data_ptr() == x.data_ptr() and torch.equal(got.dlogits, want.dlogits)
    assert torch.equal(got.top_idx, want.top_idx) and torch.equal(got.logprob, want.logprob)


def test_tokens_of_one_row_for_all():
    x, _ = make(1, 777, "bf16")
    # (rows that start at other offsets from 16 bytes add in another order: compared by the tolerance)
    r = check_tokens(x.expand(6, 777), "bf16", targets=np.array([0, 5, 776, -1, 8, 9]), top_k=3)
    assert bool((r.top_idx == r.top_idx[0]).all()) and r.dlogits.stride(0) == 777


@pytest.mark.parametrize("temperature", [0.25, 1.25, 3.0])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_tokens_temperature(dtype, temperature):
    x, _ = make(4, 2003, dtype, scale=2.0)
    check_tokens(x, dtype, temperature=temperature, top_k=9)


@pytest.mark.parametrize("times", [1, 20])     # few rows, and enough for every CTA to take several
@pytest.mark.parametrize("dtype", list(TYPES))
def test_tokens_masks(dtype, times):
    V = 1200
    x, _ = make(9, V, dtype)
    low = torch.finfo(TYPES[dtype]).min
    x[0] = float("-inf")                                  # nothing left
    x[1, :] = float("-inf"); x[1, 700] = 2.0              # one token left
    x[2, 1:] = float("-inf")
    x[3, torch.arange(V) % 2 == 0] = float("-inf")
    x[4, 5:] = low                                        # the type's lowest value as a mask
    x[5] = low                                            # all of it: a uniform row
    x[6, 3] = float("nan")
    x[7, 1100] = float("inf")
    x[8, :40] = float("-inf")
    x = x.repeat(times, 1)
    check_tokens(x, dtype, targets=np.tile([3, 700, 1, 4, 2, 9, 8, 8, 39], times), top_k=7)
    check_tokens(x, dtype, targets=np.tile([-1, 5, 0, -1, 6, 1199, -1, 1100, 41], times), top_k=128, grad=False)
    check_tokens(x, dtype, targets=np.tile([-1, 700, 0, 4, 6, 1199, 8, 1100, 41], times))
    check_tokens(x, dtype, targets=np.tile([-1, 700, 0, 4, 6, 1199, 8, 1100, 41], times), grad=False)


@pytest.mark.parametrize("times", [1, 25])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_tokens_far_apart(dtype, times):
    """Entries far above those before them, finite masks, values at the ends of the types."""
    V = 9000
    x, _ = make(8, V, dtype)
    big = 6.0e4 if dtype == "fp16" else 3.0e38
    x[0, 1500:] += 300.0                                  # far above the first chunk
    x[1] += (torch.arange(V, device="cuda") // 1024 * 90).to(x.dtype)   # rising from chunk to chunk
    x[2, :4000] = -1.0e4                                  # a finite mask over whole chunks
    x[3, ::2] = -6.0e4
    x[4, 8000] = big                                      # one entry that is everything
    x[5] = -big; x[5, 40] = -big / 2; x[5, 41] = -big / 2  # all below what sums are taken from
    x[6, :8999] = torch.finfo(TYPES[dtype]).min           # the last entry alone is more than the mask
    x[7] = big
    x = x.repeat(times, 1)
    t = np.tile([1600, 8999, 20, 1, 8000, 40, 8999, 3], times)
    check_tokens(x, dtype, targets=t, top_k=5)
    check_tokens(x, dtype, targets=t, grad=False, temperature=4.0)
    idx = np.tile(np.array([[1600, 8999, 20, 40]], np.int32), (8 * times, 1))
    val = np.tile(np.log(np.array([[0.4, 0.3, 0.1, 0.05]], np.float32)), (8 * times, 1))
    keep = np.tile([True, True, True, True, False, True, True, True], times)   # row 4 has losses of 1e38
    check_distill(x[torch.from_numpy(keep).cuda()], dtype, idx[keep], val[keep], False, w=np.ones(keep.sum(), np.float32))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,V", [(2, 9000), (1, 40000), (300, 2100)])
@pytest.mark.parametrize("k", [1, 20, 256])
def test_alternatives_with_ties(rows, V, k, dtype):
    rng = np.random.default_rng(3)
    a = rng.integers(0, 6, size=(rows, V)).astype(np.float32)     # many equal entries
    a[0] = 1.5                                                    # one value
    if rows > 1:
        a[1] = np.where(np.arange(V) % 512 == 7, 100.0 + np.arange(V) / V, 0.0)   # large entries in step
    if rows > 2:
        a[2] = -np.arange(V) / 64.0                               # large entries side by side
        a[3] = np.where(np.arange(V) < V - 300, 0.0, -0.0)
    x = torch.from_numpy(a).to(TYPES[dtype]).cuda()
    r = gs.token_logprobs(x, top_k=k)
    want = np.argsort(-f64(x), axis=1, kind="stable")[:, :k]
    assert np.array_equal(r.top_idx.cpu().numpy(), want)
    lp = vocab.log_softmax(f64(x), 1.0)
    val = np.take_along_axis(lp, want, 1)
    close(r.top_logprob, val, lse_tol(V) + 4 * U * np.abs(val), "top_logprob")
    assert r.logprob is None and r.entropy is None and r.dlogits is None


def test_alternatives_few_left_and_many_asked():
    V = 30000
    x = torch.full((3, V), float("-inf"), device="cuda")
    x[0, [5, 29999, 17]] = torch.tensor([1.0, 2.0, 1.0], device="cuda")
    x[1, 100:100 + 2000] = 0.25
    x[2, ::3] = torch.arange(10000, device="cuda").float()
    r = gs.token_logprobs(x, top_k=200)
    want = vocab.token_logprobs(f64(x), 1.0, None, 200)
    assert np.array_equal(r.top_idx.cpu().numpy(), want[2])
    close(r.top_logprob, want[3], lse_tol(V) + 4 * U * np.abs(np.nan_to_num(want[3], neginf=0.0)), "top_logprob")


def test_tokens_outside_the_vocabulary_are_reported_and_left_out():
    x, _ = make(4, 100, "fp32")
    for bad in ([100, 1, 2, 3], [0, -2, 2, 3], [0, 1, 2, 2 ** 31 - 1]):
        st = gs.status_tensor()
        ok = [t if 0 <= t < 100 else -1 for t in bad]
        g = dev(np.ones(4))
        a = gs.token_logprobs(x, dev(bad, torch.int64).to(torch.int32), want_grad=True, grad_logprob=g, d_status=st)
        b = gs.token_logprobs(x, dev(ok, torch.int32), want_grad=True, grad_logprob=g)
        assert int(st.item()) == gs.DERR_INDEX_RANGE
        assert torch.equal(a.logprob, b.logprob) and torch.equal(a.dlogits, b.dlogits)


def test_zero_weights_give_zeros_whatever_the_row_holds():
    x, _ = make(3, 500, "bf16")
    x[1] = float("nan")
    r = gs.token_logprobs(x, dev([1, 2, 3], torch.int32), want_grad=True, grad_logprob=dev([1.0, 0.0, 1.0]))
    assert bool((r.dlogits[1] == 0).all()) and bool(torch.isnan(r.logprob[1])) and bool((r.dlogits[0] != 0).any())
    r = gs.token_logprobs(x, dev([1, 2, 3], torch.int32), want_grad=True)
    assert bool((r.dlogits == 0).all())


def test_same_bits_every_time():
    x, _ = make(5, 60001, "bf16", scale=1.0)
    idx = torch.randint(0, 60001, (5, 100), device="cuda", dtype=torch.int32)
    val = torch.randn(5, 100, device="cuda")
    a = gs.token_logprobs(x, idx[:, 0].contiguous(), top_k=100, want_entropy=True, want_grad=True,
                          grad_logprob=val[:, 0].contiguous())
    d = gs.distill_topk(x, idx, val - 6, tail=True, want_grad=True, grad_loss=val[:, 0].contiguous())
    for _ in range(3):
        b = gs.token_logprobs(x, idx[:, 0].contiguous(), top_k=100, want_entropy=True, want_grad=True,
                              grad_logprob=val[:, 0].contiguous())
        e = gs.distill_topk(x, idx, val - 6, tail=True, want_grad=True, grad_loss=val[:, 0].contiguous())
        for u, v in zip([a.logprob, a.entropy, a.top_idx, a.top_logprob, a.dlogits, d.loss, d.dlogits],
                        [b.logprob, b.entropy, b.top_idx, b.top_logprob, b.dlogits, e.loss, e.dlogits]):
            assert torch.equal(u, v)


# ---- backward pass of its own ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (3, 9, 4), (4, 1000, 0), (3, 4099, 20), (2, 50021, 256), (400, 2100, 3)])
def test_tokens_backward(rows, V, k, dtype):
    x, _ = make(rows, V, dtype, stride=V + 3, first=2)
    if rows > 2:
        x[2, : V // 2] = float("-inf")
    h = f64(x)
    it = float(np.float32(1 / 1.25))
    rng = np.random.default_rng([9, rows, V])
    t = rng.integers(-1, V, size=rows)
    w = weights(rows)
    r = gs.token_logprobs(x, dev(t, torch.int32), top_k=k, want_entropy=True, want_stats=True, temperature=1.25)
    gt = rng.normal(size=(rows, k)).astype(np.float32)
    gt[3::7] = 0.0
    got = gs.token_logprobs_backward(x, r.stats, dev(t, torch.int32), dev(w[0]), r.entropy, dev(w[1]),
                                     r.top_idx, dev(gt) if k else None, temperature=1.25)
    want = vocab.token_logprobs_grad(h, it, t, w[0].astype(np.float64), w[1].astype(np.float64),
                                     r.top_idx.cpu().numpy() if k else None, gt.astype(np.float64) if k else None)
    ent = vocab.token_logprobs(h, it)[1]
    extra = np.abs(w[0]) + np.abs(gt).sum(1)
    tol = grad_tol(h, it, want, dtype, it * (extra + np.abs(w[1]) * ent), it * w[1], it * extra)
    close(got, want, tol, "dlogits")
    # in the logits' place
    if k:
        again = gs.token_logprobs_backward(x, r.stats, dev(t, torch.int32), dev(w[0]), r.entropy, dev(w[1]), r.top_idx,
                                           dev(gt), temperature=1.25, dlogits=x)
        assert torch.equal(again, got)


def test_alternatives_whose_gradients_cancel():
    x, _ = make(1, 50, "fp32")
    s = gs.token_logprobs(x, top_k=2, want_stats=True)
    g = gs.token_logprobs_backward(x, s.stats, top_idx=s.top_idx, grad_top=dev([[0.5, -0.5]]))
    i = s.top_idx.cpu().numpy()[0]
    want = np.zeros(50)
    want[i] = [0.5, -0.5]
    assert np.array_equal(f64(g)[0], want)
    twice = gs.token_logprobs_backward(x, s.stats, targets=s.top_idx[:, 0].contiguous(), grad_logprob=dev([1.0]),
                                       top_idx=s.top_idx[:, :1].repeat(1, 3), grad_top=dev([[0.25, 0.5, 0.25]]))
    once = gs.token_logprobs_backward(x, s.stats, targets=s.top_idx[:, 0].contiguous(), grad_logprob=dev([2.0]))
    assert torch.equal(twice, once)


# ---- distillation -----------------------------------------------------------------------------------

def lists(x, k, it, tail, seed=0, ragged=True):
    rows, V = x.shape
    rng = np.random.default_rng([seed, rows, V, k])
    y = f64(x) + rng.normal(size=x.shape) * 0.7
    lp = vocab.log_softmax(np.where(np.isfinite(y), y, -50.0), it)
    idx = np.argsort(-lp, axis=1, kind="stable")[:, :k].astype(np.int32)
    if idx.shape[1] < k:                                  # more places than tokens
        idx = np.concatenate([idx, np.full((rows, k - idx.shape[1]), -1, np.int32)], 1)
    val = np.take_along_axis(lp, np.maximum(idx, 0), 1).astype(np.float32)
    if ragged:
        idx[:, k // 2:][rng.random((rows, k - k // 2)) < 0.3] = -1
        if rows > 2:
            idx[1] = -1
    for r in range(rows):
        p = rng.permutation(k)
        idx[r], val[r] = idx[r, p], val[r, p]
    return idx, val


def check_distill(x, dtype, idx, val, tail, temperature=1.0, val_dtype="fp32", w=None):
    rows, V = x.shape
    it = float(np.float32(1.0 / temperature))
    h = f64(x)
    tv = torch.from_numpy(val).to(TYPES[val_dtype]).cuda()
    ti = dev(idx, torch.int32)
    w = weights(rows)[0] if w is None else w
    st = gs.status_tensor()
    r = gs.distill_topk(x, ti, tv, tail=tail, temperature=temperature, grad_loss=dev(w), want_grad=True, want_stats=True,
                        d_status=st)
    assert int(st.item()) == 0
    v64 = f64(tv)
    want = vocab.distill(h, it, idx, v64, tail)
    close(r.loss, want, 2 * lse_tol(V) + 2 * U * np.abs(np.where(np.isfinite(want), want, 0)), "loss")
    grad = vocab.distill_grad(h, it, idx, v64, tail, w.astype(np.float64))
    grad[w == 0] = 0.0
    q = vocab.teacher(idx, v64, it, tail)[1].sum(1)
    size = it * np.abs(w) * np.maximum(q, 1.0)
    # with the tail, an entry outside the list has (mass + rest) p - rest p / R: two terms of p's accuracy
    tol = grad_tol(h, it, grad, dtype, size, 0 * size, size)
    if tail:
        lp = vocab.log_softmax(h, it)
        for row in range(rows):
            lr = vocab._log_rest(lp[row], idx[row]) if np.isfinite(lp[row]).any() else -np.inf
            if np.isfinite(lr):
                l2 = np.abs(np.where(np.isfinite(lp[row]), lp[row] - lr, 0)) / math.log(2)
                pt = np.exp(np.where(np.isfinite(lp[row]), lp[row] - lr, -np.inf))
                tol[row] += 2 * size[row] * pt * ((8 + 3 * l2 + 4 * math.log2(V + 1)) * U + lse_tol(V)) * max(0.0, 1 - q[row])
    close(r.dlogits, grad, tol, "dlogits")
    back = gs.distill_topk_backward(x, r.stats, ti, tv, dev(w), tail=tail, temperature=temperature)
    # the statistics were rounded to fp32 on the way: the tolerance has room for it (LSE holds 64 u)
    close(back, grad, tol, "backward")
    # without the gradient the row may be added in another order: the loss to the same tolerance
    plain = gs.distill_topk(x, ti, tv, tail=tail, temperature=temperature)
    close(plain.loss, want, 2 * lse_tol(V) + 2 * U * np.abs(np.where(np.isfinite(want), want, 0)), "loss alone")
    return r


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (3, 2, 2), (3, 9, 4), (4, 65, 13), (5, 1000, 8), (3, 1001, 64),
                                      (3, 4099, 32), (2, 50021, 256), (1, 40000, 100), (350, 2100, 5), (3, 5, 9),
                                      (301, 1, 1), (200, 9, 4), (1000, 1000, 8), (449, 1031, 40), (160, 12347, 256),
                                      (150, 70001, 64)])
def test_distill_sizes(rows, V, k, dtype, tail):
    x, _ = make(rows, V, dtype, stride=V + 5, first=3)
    idx, val = lists(x, k, 1.0, tail)
    check_distill(x, dtype, idx, val, tail)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature,val_dtype", [(0.5, "fp32"), (2.0, "bf16"), (1.25, "fp16"), (4.0, "fp32")])
def test_distill_temperature_and_value_types(temperature, val_dtype, tail):
    x, _ = make(4, 3001, "bf16")
    idx, val = lists(x, 24, float(np.float32(1 / temperature)), tail)
    check_distill(x, "bf16", idx, val, tail, temperature, val_dtype)


@pytest.mark.parametrize("times", [1, 50])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_a_confident_student(tail, times):
    # the list holds all but 1e-9 of the student's mass: what it leaves must not be a difference of sums
    V = 3000
    x = torch.zeros(4, V, device="cuda")
    x[:, 7] = 30.0
    x[1, 8] = 29.0
    x[2, 9] = 80.0
    x[3, 7] = 200.0
    idx = np.array([[7, 8], [8, 7], [9, 7], [7, 3]], np.int32)
    val = np.log(np.array([[0.9, 0.05], [0.3, 0.6], [0.5, 0.25], [0.99, 0.001]])).astype(np.float32)
    check_distill(x.repeat(times, 1), "fp32", np.tile(idx, (times, 1)), np.tile(val, (times, 1)), tail,
                  w=np.ones(4 * times, np.float32))


@pytest.mark.parametrize("times", [1, 20])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_distill_masks_and_lists(dtype, tail, times):
    V = 1100
    x, _ = make(10, V, dtype)
    idx = np.tile(np.array([[3, 900, 14, 15]], np.int32), (10, 1))
    val = np.tile(np.log(np.array([[0.4, 0.3, 0.1, 0.05]], np.float32)), (10, 1))
    x[0] = float("-inf")                                  # nothing left, and a list: no probability for it
    x[1] = float("-inf"); idx[1] = -1                     # nothing left and nothing wanted
    x[2, [i for i in range(V) if i not in (3, 900, 14, 15)]] = float("-inf")   # the list is all there is
    x[3, 900] = float("-inf")                             # a wanted token is ruled out
    val[4, 1] = -np.inf                                   # an entry without mass on a token ruled out
    x[4, 900] = float("-inf")
    val[5] = -np.inf                                      # no mass in the list at all
    idx[6] = [3, 3, 14, 3]                                # an index several times
    idx[7] = [-1, -1, 5, -1]
    val[8] += 0.3                                         # with the tail: more mass than one
    x[9, 40] = float("nan")
    check_distill(x.repeat(times, 1), dtype, np.tile(idx, (times, 1)), np.tile(val, (times, 1)), tail,
                  w=np.tile(np.linspace(0.5, 1.5, 10), times).astype(np.float32))


@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_empty_lists_give_zeros_whatever_the_row_holds(dtype, tail, rows):
    """Padding: rows without a list and with anything for logits."""
    x, _ = make(rows, 3000, dtype)
    x[0] = float("nan")
    x[1, 2999] = float("inf")
    idx = np.full((rows, 5), -1, np.int32)
    idx[2] = [4, 7, -1, 1, 2000]
    ti, tv, w = dev(idx, torch.int32), dev(np.log(np.full((rows, 5), 0.1))), dev(np.ones(rows))
    r = gs.distill_topk(x, ti, tv, tail=tail, want_grad=True, want_stats=True, grad_loss=w)
    back = gs.distill_topk_backward(x, r.stats, ti, tv, w, tail=tail)
    plain = gs.distill_topk(x, ti, tv, tail=tail)
    empty = torch.arange(rows, device="cuda") != 2
    for out in (r.loss, plain.loss, r.dlogits, back):
        assert bool((out[empty] == 0).all()) and bool(torch.isfinite(out[2]).all()) and bool((out[2] != 0).any())


def test_distill_bad_indices_are_reported_and_left_out():
    x, _ = make(2, 100, "fp32")
    val = dev(np.log([[0.5, 0.2, 0.1], [0.5, 0.2, 0.1]]))
    for tail in (False, True):
        for bad in ([[1, 100, 3], [4, 5, 6]], [[1, 2, -5], [4, 5, 6]], [[1, 2 ** 31 - 1, 3], [-2 ** 31, 5, 6]]):
            ok = [[i if 0 <= i < 100 else -1 for i in row] for row in bad]
            st = gs.status_tensor()
            g = dev(np.ones(2))
            a = gs.distill_topk(x, dev(bad, torch.int64).to(torch.int32), val, tail=tail, grad_loss=g, want_grad=True, d_status=st)
            b = gs.distill_topk(x, dev(ok, torch.int32), val, tail=tail, grad_loss=g, want_grad=True, want_stats=True)
            assert int(st.item()) == gs.DERR_INDEX_RANGE
            assert torch.equal(a.loss, b.loss) and torch.equal(a.dlogits, b.dlogits)
            st.zero_()
            gs.distill_topk_backward(x, b.stats, dev(bad, torch.int64).to(torch.int32), val, g, tail=tail, d_status=st)
            assert int(st.item()) == gs.DERR_INDEX_RANGE


@pytest.mark.parametrize("tail", [False, True])
def test_distill_in_place(tail):
    for rows, V in [(3, 2000), (1, 40001), (400, 1500)]:
        x, _ = make(rows, V, "bf16", first=1)
        idx, val = lists(x, 17, 1.0, tail)
        ti, tv, w = dev(idx, torch.int32), dev(val), dev(weights(rows)[0])
        want = gs.distill_topk(x, ti, tv, tail=tail, grad_loss=w, want_grad=True, want_stats=True)
        y = x.clone()
        gs.distill_topk_backward(y, want.stats, ti, tv, w, tail=tail, dlogits=y)
        got = gs.distill_topk(x, ti, tv, tail=tail, grad_loss=w, dlogits=x)
        assert torch.equal(got.dlogits, want.dlogits) and torch.equal(got.loss, want.loss)
        half = torch.finfo(torch.bfloat16).eps
        assert bool(((y.float() - want.dlogits.float()).abs() <= half * want.dlogits.float().abs() + 1e-6).all())


@pytest.mark.parametrize("dtype,V", [("bf16", 900_001), ("fp32", 450_003)])
def test_rows_longer_than_eight_slices(dtype, V):
    """Rows that shared memory cannot hold between the sums and the gradient are read twice."""
    x, _ = make(2, V, dtype, stride=V + 3, first=1)
    check_tokens(x, dtype, targets=np.array([V - 1, 17]), top_k=20)
    idx, val = lists(x, 40, 1.0, True, ragged=False)
    for tail in (False, True):
        check_distill(x, dtype, idx, val, tail)
    ti, tv, w = dev(idx, torch.int32), dev(val), dev(weights(2)[0])
    want = gs.distill_topk(x, ti, tv, tail=True, grad_loss=w, want_grad=True)
    got = gs.distill_topk(x, ti, tv, tail=True, grad_loss=w, dlogits=x)
    assert torch.equal(got.dlogits, want.dlogits) and torch.equal(got.loss, want.loss)


# ---- references far from 0 ------------------------------------------------------------------------
#
# The exponent (x - m) c of an entry far from 0 must be 0 at the reference m itself: the rounding of the product
# m c alone, half a step of it, is more than an exponent may be off by once |m c| is beyond about 2^20.

MASKS = [-1e6, -1e7, -1e8, -1e9, -1e10, -1e11, -1e12, -1e15, -1e18, -1e20, -1e30]


def rounded_out(want, dtype):
    """What rounding makes of values beyond the type's range: infinities (fp16 from 65520 on, fp32 from 2^128 - 2^103)."""
    end = 65520.0 if dtype == "fp16" else 2.0 ** 128 - 2.0 ** 103
    return np.where(np.abs(want) >= end, np.copysign(np.inf, want), want)


def check_all(x, dtype, temperature, targets, idx, val):
    """Both losses in every form: alone, with the gradient, the gradient from statistics."""
    rows, V = x.shape
    it = float(np.float32(1.0 / temperature))
    h = f64(x)
    w, t, k = weights(rows), dev(targets, torch.int32), 4 if rows < 100 else 0
    r = gs.token_logprobs(x, t, top_k=k, want_entropy=True, temperature=temperature)
    lp, ent, idx4, val4 = vocab.token_logprobs(h, it, targets, k)

    def logs(want):
        return lse_tol(V) + 4 * U * np.abs(np.where(np.isfinite(want), want, 0))

    def losses(r):
        close(r.logprob, rounded_out(lp, "fp32"), logs(lp), "logprob")
        close(r.entropy, ent, lse_tol(V) * (2 + math.log(V + 1)) + U * np.abs(ent), "entropy")

    losses(r)
    if k:
        assert np.array_equal(r.top_idx.cpu().numpy(), idx4)
        close(r.top_logprob, rounded_out(val4, "fp32"), logs(val4), "top_logprob")
    kw = dict(grad_logprob=dev(w[0]), grad_entropy=dev(w[1]), temperature=temperature)
    r = gs.token_logprobs(x, t, want_entropy=True, want_stats=True, want_grad=True, **kw)
    back = gs.token_logprobs_backward(x, r.stats, t, entropy=r.entropy, **kw)
    losses(r)
    want = vocab.token_logprobs_grad(h, it, targets, w[0].astype(np.float64), w[1].astype(np.float64))
    want[(np.where(targets < 0, 0, w[0]) == 0) & (w[1] == 0)] = 0.0
    tol = grad_tol(h, it, want, dtype, it * (np.abs(w[0]) + np.abs(w[1]) * ent), it * w[1], it * w[0])
    close(r.dlogits, rounded_out(want, dtype), tol, "dlogits")
    close(back, rounded_out(want, dtype), tol, "backward")
    small = min(1.0, 1.0e4 * temperature) if dtype == "fp16" else 1.0
    for tail in (False, True):
        check_distill(x, dtype, idx, val, tail, temperature, w=np.full(rows, small, np.float32))


def some_lists(rows, V):
    idx = np.tile(np.array([[V - 3, 7, V // 2, -1]], np.int32), (rows, 1))
    val = np.tile(np.log(np.array([[0.4, 0.3, 0.1, 0.05]], np.float32)), (rows, 1))
    return idx, val


# once: a row over several CTAs; six times: a CTA for each row
@pytest.mark.parametrize("temperature,times", [(0.5, 1), (1.0, 1), (1.25, 1), (2.0, 1), (4.0, 1), (1.0, 6), (2.0, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_finite_masks_of_any_size(dtype, temperature, times):
    V, n = 9000, len(MASKS)
    x, _ = make(5 * n, V, dtype)
    m = torch.tensor(MASKS, device="cuda").to(x.dtype)[:, None]
    x[:n] = m                                             # nothing but the mask
    x[n:2 * n, :2048] = m                                 # the first entries of a vocabulary
    x[2 * n:3 * n, :V - 1] = m                            # all entries but one
    x[3 * n:4 * n] = -m                                   # far above 0
    x[4 * n:, ::2] = m
    x[4 * n:, 4096:8192] = m                              # whole chunks after ordinary ones
    x = x.repeat(times, 1)
    t = np.tile([3, V - 1, 2050, -1, 5], n * times)
    check_all(x, dtype, temperature, t, *some_lists(len(t), V))


@pytest.mark.parametrize("temperature", [1e-3, 1e-4, 1e-5, 1e-6, 1e-7, 1e-8, 1e-9])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_low_temperatures(dtype, temperature):
    V = 9000
    x, _ = make(12, V, dtype)
    x[0, [20, 8000]] = 9.1                                # two equal maxima
    x[1, [8000, 8001]] = 21.5
    x[2] = 7.3
    x[3] = -7.3
    x[4, :4500] = -1.0e4
    x[5] = float("-inf"); x[5, 4000:4002] = 3.3
    x[6] = torch.linspace(1.0, 1.0 + 40 * temperature, V, device="cuda").to(x.dtype)
    x[7] = 1.7 + torch.linspace(0.0, 40 * temperature, V, device="cuda").flip(0).to(x.dtype)
    t = np.array([20, 8001, 5, 6, 8000, 4001, V - 1, 0, -1, 7, 8, 9])
    check_all(x, dtype, temperature, t, *some_lists(12, V))


@pytest.mark.parametrize("at", [45426.0, -45426.0, 726817.0, -726817.0, 3.0e6, -3.0e6])
@pytest.mark.parametrize("times", [1, 40])
def test_references_on_both_sides_of_the_border(at, times):
    """Logits around the size where the difference is taken first (2^20 bits) and beyond, spread as ordinary ones are."""
    V = 9000
    x, _ = make(6, V, "fp32")
    x += at
    x[0, :4000] += 8.0
    x[1, 4000:] += 8.0
    x[2] += (torch.arange(V, device="cuda") // 512).float()
    x[3] -= (torch.arange(V, device="cuda") // 512).float()
    x[4, :3000] = 0.0 if at < 0 else -1e9
    x = x.repeat(times, 1)
    t = np.tile([3, V - 1, 2050, 17, 5, 4000], times)
    check_all(x, "fp32", 1.0, t, *some_lists(len(t), V))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_entropy_of_rows_with_a_peak_far_above_what_came_before(dtype):
    """The entropy log S - T / S of a row with one likely token: taken from a reference far below the peak, T / S
    alone carries |q| u.

    From a reference at the peak (36 bits or more above the rest, so that sums are moved to it) S is 1 and a rest
    below 2^-22, with the 4 u of 2^q at the peak; |T / S| is below 2^-16, its roundings nothing; the result
    is rounded to fp32. Together less than 8 u, where a reference 36 to 50 bits below the peak has up to 35 u."""
    rows, V = 300, 20000
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.uniform(0.0, 1.0, size=(rows, V)).astype(np.float32)).to(TYPES[dtype]).cuda()
    at = rng.integers(8000, V, size=rows)
    x[torch.arange(rows), torch.from_numpy(at).cuda()] = dev(rng.uniform(26.5, 35.0, size=rows)).to(x.dtype)
    t = dev(at, torch.int32)
    h = f64(x)
    ent = vocab.token_logprobs(h, 1.0)[1]
    one = torch.ones(rows, device="cuda")
    for r in (gs.token_logprobs(x, t, want_entropy=True),
              gs.token_logprobs(x, t, want_entropy=True, want_grad=True, grad_logprob=one)):
        close(r.entropy, ent, 8 * U, "entropy")
        close(r.logprob, vocab.token_logprobs(h, 1.0, at)[0], 8 * U, "logprob")


@pytest.mark.parametrize("dtype,V,rows", [("bf16", 1000000, 300), ("fp32", 300000, 300), ("bf16", 1 << 24, 2)])
def test_many_small_entries_beside_a_large_one(dtype, V, rows):
    """One entry of 1 and V - 1 entries e of 0.9 u (u = 2^-24): added one by one to 1 each of them would be lost, V / 448
    of them in the sum that holds the 1. A chunk's entries are added up first (of 7 warps, 128 vectors of N entries each):
    at most a lane's own 2 N there are lost, and each of the warp's V / (7 * 128 N) chunks adds one rounding, u; then
    2^q (4 u), the join of the lanes (6 u), the result (2 u)."""
    peak = torch.tensor(-math.log(0.9 * U), device="cuda").to(TYPES[dtype])
    x = torch.zeros(rows, V, dtype=TYPES[dtype], device="cuda")
    at = dev(np.random.default_rng(12).integers(0, V, size=rows), torch.int32)
    x[torch.arange(rows, device="cuda"), at.long()] = peak
    e = math.exp(-float(peak))
    N = 4 if dtype == "fp32" else 8
    tol = (2 * N + V / (7 * 128 * N) + 12) * U
    one = torch.ones(rows, device="cuda")
    for r in (gs.token_logprobs(x, at, want_stats=True),
              gs.token_logprobs(x, at, want_stats=True, want_grad=True, grad_logprob=one)):
        close(r.logprob, np.full(rows, -math.log1p((V - 1) * e)), tol, "logprob")


@pytest.mark.parametrize("rows,V", [(3, 1 << 24), (9, 128001), (330, 40003)])
def test_infinite_and_huge_entries_with_long_lists(rows, V):
    """Rows with +inf or entries near the types' ends cost no more than others: the largest vocabulary, a list of 256."""
    k = 256
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    x = torch.randn(rows, V, device="cuda", generator=gen).to(torch.bfloat16)
    x[0, V - 5] = float("inf")
    x[1, 4000] = 1.0e38
    x[2, ::2] = -1.0e38
    idx = np.tile((np.arange(k, dtype=np.int64) * 7919 * 2 + 1) % V, (rows, 1)).astype(np.int32)
    idx[1, 5] = 4000
    val = np.tile(np.log(np.full(k, 0.9 / k)).astype(np.float32), (rows, 1))
    w = np.ones(rows, np.float32)
    ti, tv, st = dev(idx, torch.int32), dev(val), gs.status_tensor()
    n = min(rows, 9)                                      # the rows that are compared
    h, v64 = f64(x[:n]), val[:n].astype(np.float64)
    for tail in (True, False):
        a = gs.distill_topk(x, ti, tv, tail=tail, d_status=st)
        b = gs.distill_topk(x, ti, tv, tail=tail, want_grad=True, grad_loss=dev(w), d_status=st)
        want = vocab.distill(h, 1.0, idx[:n], v64, tail)
        tol = 2 * lse_tol(V) + 2 * U * np.abs(np.nan_to_num(want))
        close(a.loss[:n], want, tol, "loss")
        close(b.loss[:n], want, tol, "loss with the gradient")
        grad = vocab.distill_grad(h, 1.0, idx[:n], v64, tail, w[:n].astype(np.float64))
        # (mass + rest) p - rest p / R: terms of p's accuracy that cancel at most where R is near 1 (four times p), the
        # second alone (the gradient itself; log2 of p / R within 64) where p vanishes beside the list; rounded to bf16
        l2 = np.abs(np.nan_to_num(np.maximum(vocab.log_softmax(h, 1.0), -100.0))) / math.log(2)
        rel = (16 + 8 * math.log2(V + 1)) * U + 2 * lse_tol(V)
        body = 4 * np.exp2(-l2) * (rel + 3 * l2 * U) + np.abs(np.nan_to_num(grad)) * (rel + 3 * 64 * U)
        close(b.dlogits[:n], grad, body + 2.0 ** -8 * (np.abs(np.nan_to_num(grad)) + body) + TINY["bf16"], "dlogits")
    r = gs.token_logprobs(x, ti[:, 0].contiguous(), top_k=20, want_entropy=True, d_status=st)
    lp, ent, top, _ = vocab.token_logprobs(h[:3], 1.0, idx[:3, 0], 0 if V > 1 << 20 else 20)
    close(r.logprob[:3], lp, lse_tol(V) + 4 * U * np.abs(np.nan_to_num(lp)), "logprob")
    close(r.entropy[:3], ent, lse_tol(V) * (2 + math.log(V + 1)), "entropy")
    if V <= 1 << 20:
        assert np.array_equal(r.top_idx[:3].cpu().numpy(), top)
    assert int(st.item()) == 0


# ---- as a run ---------------------------------------------------------------------------------------

def test_teacher_to_student_to_compressed_gradient():
    """A teacher's alternatives are the student's lists, and the student's gradient is what the residual
    top-k compresses."""
    rows, V, k, T = 24, 3001, 16, 2.0
    teacher, _ = make(rows, V, "fp32", seed=1)
    student = teacher + 0.3 * make(rows, V, "fp32", seed=2)[0]
    top = gs.token_logprobs(teacher, top_k=k, temperature=T)
    same = gs.distill_topk(teacher, top.top_idx, top.top_logprob, tail=True, temperature=T, want_grad=True,
                           grad_loss=dev(np.ones(rows)))
    # the list's values were rounded to fp32 (u |log q| each) and carry log S's error
    assert float(same.loss.abs().max()) < 4 * lse_tol(V) and float(same.dlogits.abs().max()) < 16 * U * 10 + lse_tol(V)
    w = np.full(rows, T * T / rows, np.float32)
    r = gs.distill_topk(student, top.top_idx, top.top_logprob, tail=True, temperature=T, want_grad=True, grad_loss=dev(w))
    it = 1.0 / T
    want = vocab.distill(f64(student), it, top.top_idx.cpu().numpy(), f64(top.top_logprob), True)
    close(r.loss, want, 2 * lse_tol(V) + 2 * U * np.abs(want), "loss")
    flat = r.dlogits.reshape(-1)
    pad = (-flat.numel()) % 4
    g = torch.nn.functional.pad(flat, (0, pad))
    residual = torch.zeros_like(g)
    idx, val, off = gs.residual_topk(g, residual, (1, 100))
    K = int(off[-1])
    order = torch.argsort(g.abs(), descending=True, stable=True)[:K]
    assert torch.equal(idx[:K].long(), order.sort().values) and torch.equal(val[:K], g[idx[:K].long()])
    # moving the student against its gradient lowers the loss by about the gradient's square
    step = 0.05
    after = gs.distill_topk(student - step * r.dlogits, top.top_idx, top.top_logprob, tail=True, temperature=T)
    down = float((dev(w) * (r.loss - after.loss)).sum())
    square = float((r.dlogits.double() ** 2).sum())
    assert 0.9 * step * square < down < 1.0 * step * square + 1e-6


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_output_layers_gradient_over_steps(dtype, pad):
    """Three steps of a student: the gradient of its output layer, made from that of the logits, goes through the
    residual top-k; what was sent and what is carried add up to the gradients of all steps."""
    rows, V, D, k, T = 20, 1001, 16, 8, 2.0
    rng = np.random.default_rng(21)
    weight = dev(rng.normal(size=(V, D)) * 0.3).requires_grad_()
    residual = torch.zeros(V * D, device="cuda")
    sent, total = np.zeros(V * D), np.zeros(V * D)
    w = np.full(rows, 1.0 / rows, np.float32)
    for step in range(3):
        hidden = dev(rng.normal(size=(rows, D)))
        teacher, _ = make(rows, V, dtype, seed=50 + step, stride=V + pad)
        top = gs.token_logprobs(teacher, top_k=k, temperature=T)
        out = (hidden @ weight.t()).to(TYPES[dtype])
        logits, _ = make(rows, V, dtype, stride=V + pad)      # rows of a padded buffer
        logits.copy_(out.detach())
        r = gs.distill_topk(logits, top.top_idx, top.top_logprob, tail=True, temperature=T, want_grad=True, grad_loss=dev(w))
        assert r.dlogits.stride(0) == V + pad and not r.loss.requires_grad
        grad = (r.dlogits.float().t() @ hidden).reshape(-1)
        weight.grad = None
        out.backward(r.dlogits)                               # the same through autograd: fp32 sums of 20 products
        size = (r.dlogits.abs().double().t() @ hidden.abs().double()).reshape(-1)
        assert bool(((grad - weight.grad.reshape(-1)).abs() <= 2 * (rows + 1) * U * size).all())
        before = residual.clone()
        idx, val, off = gs.residual_topk(grad, residual, (1, 100))
        K = int(off[-1])
        assert K == gs.k_for(V * D, (1, 100))
        acc = before + grad
        at = idx[:K].long()
        assert torch.equal(val[:K], acc[at]) and bool((residual[at] == 0).all())
        keep = torch.ones(V * D, dtype=torch.bool, device="cuda")
        keep[at] = False
        assert torch.equal(residual[keep], acc[keep])
        sent[at.cpu().numpy()] += f64(val[:K])
        total += f64(grad)
    # two fp32 additions per place
    assert np.abs(sent + f64(residual) - total).max() <= 2 * U * 3 * np.abs(total).max() + 1e-12


@pytest.mark.parametrize("temperature", [2.0 ** -64, 2.0 ** 64])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_temperatures_at_the_ends(dtype, temperature):
    V = 9000
    x, _ = make(8, V, dtype)
    x[0] = 0.0
    x[1, 5000:] = 1.0e38
    x[2] = -1.0e38; x[2, 4500] = 3.0e38
    x[3] = torch.linspace(1.0, 2.0, V, device="cuda").to(x.dtype) * 2.0 ** -63
    x[4] = torch.linspace(-1.0, 1.0, V, device="cuda").to(x.dtype) * 2.0 ** 63
    x[5, 100:] = float("-inf")
    t = np.array([3, V - 1, 4500, V - 1, 0, 99, -1, 17])
    if temperature < 1:                                    # (the losses of rows 1, 2 and 4 are beyond fp32)
        with_losses = [0, 3, 5, 6, 7]
        r = gs.token_logprobs(x, dev(t, torch.int32), top_k=1, want_entropy=True, temperature=temperature)
        assert r.logprob[4].item() == -math.inf and r.top_idx[2].item() == 4500 and r.logprob[2].item() == 0.0
        assert abs(r.entropy[4].item() - math.log((x[4] == x[4].max()).sum().item())) < 1e-6
        x, t = x[with_losses].contiguous(), t[with_losses]
    check_all(x, dtype, temperature, t, *some_lists(len(t), V))


def test_streams_and_two_calls_at_once():
    sets = []
    for s in range(2):
        x, _ = make(200, 20001, "bf16", seed=10 + s)
        idx, val = lists(x[:4], 8, 1.0, True)
        sets.append((x, dev(np.tile(idx, (50, 1)), torch.int32), dev(np.tile(val, (50, 1)))))
    want = [gs.distill_topk(x, i, v, tail=True, want_grad=True, grad_loss=torch.ones(200, device="cuda")) for x, i, v in sets]
    tops = [gs.token_logprobs(x, top_k=50) for x, _, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got, gtops = [None, None], [None, None]
    ones = torch.ones(200, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (x, i, v) in enumerate(sets):
            with torch.cuda.stream(streams[s]):
                got[s] = gs.distill_topk(x, i, v, tail=True, want_grad=True, grad_loss=ones)
                gtops[s] = gs.token_logprobs(x, top_k=50)
    torch.cuda.synchronize()
    for s in range(2):
        assert torch.equal(got[s].loss, want[s].loss) and torch.equal(got[s].dlogits, want[s].dlogits)
        assert torch.equal(gtops[s].top_idx, tops[s].top_idx) and torch.equal(gtops[s].top_logprob, tops[s].top_logprob)


@pytest.mark.parametrize("rows", [6, 330])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_far_references_in_the_logits_place_and_in_graphs(dtype, rows):
    """Rows whose sums and gradient take the difference first: the gradient over the logits, captured and replayed."""
    V, T = 9001, 1e-4                                     # (rows at every offset from 16 bytes)
    x, _ = make(rows, V, dtype)
    if dtype != "fp16":
        x[0] = -1.0e12
        x[1, :5000] = -1.0e12
        x[2, 4000:] = 1.0e12
    t = dev(np.arange(rows) % V, torch.int32)
    idx, val = some_lists(rows, V)
    ti, tv, w = dev(idx, torch.int32), dev(val), dev(np.full(rows, 1e-4))

    def forms(x, place):
        y = [x.clone() if place else None for _ in range(4)]
        a = gs.token_logprobs(x if y[0] is None else y[0], t, want_entropy=True, want_stats=True, temperature=T, grad_logprob=w,
                              grad_entropy=w, want_grad=True, dlogits=y[0])
        b = gs.token_logprobs_backward(x if y[1] is None else y[1], a.stats, t, w, a.entropy, w, temperature=T, dlogits=y[1])
        c = gs.distill_topk(x if y[2] is None else y[2], ti, tv, tail=True, temperature=T, grad_loss=w, want_grad=True,
                            want_stats=True, dlogits=y[2])
        d = gs.distill_topk_backward(x if y[3] is None else y[3], c.stats, ti, tv, w, tail=True, temperature=T, dlogits=y[3])
        return [a.logprob, a.entropy, a.dlogits, b, c.loss, c.dlogits, d]

    want = forms(x, False)
    for u, v in zip(forms(x, True), want):
        assert torch.equal(u, v) and not bool(torch.isnan(v).any())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = forms(x, False)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_calls_of_two_threads():
    """Host threads that call one operator with other vocabularies and lists: each launch gets the memory it asks for."""
    import threading
    one = torch.ones(1, device="cuda")
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    sets = []
    for V, k in [(110000, 3), (400000, 250)]:
        x = make(1, V, "fp32", seed=40)[0]
        r = gs.token_logprobs(x, t, top_k=k, want_stats=True, want_grad=True, grad_logprob=one)
        g_top = torch.ones(1, k, device="cuda")
        sets.append((x, k, r, g_top, gs.token_logprobs_backward(x, r.stats, t, one, top_idx=r.top_idx, grad_top=g_top)))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def work(x, k, want, g_top, back):
        try:
            V, out, back_out = x.shape[1], torch.empty_like(x), torch.empty_like(x)
            logprob, stream = torch.empty_like(want.logprob), torch.cuda.Stream()
            fused = (x.data_ptr(), 0, 1, V, V, 1.0, t.data_ptr(), logprob.data_ptr(), None, None, 0, None, None,
                     out.data_ptr(), V, one.data_ptr(), None, None, stream.cuda_stream)
            backward = (x.data_ptr(), 0, 1, V, V, 1.0, want.stats.data_ptr(), t.data_ptr(), one.data_ptr(), None, None, k,
                        want.top_idx.data_ptr(), g_top.data_ptr(), back_out.data_ptr(), V, None, stream.cuda_stream)
            for f, args in [(gs.lib().gsparse_token_logprobs, fused), (gs.lib().gsparse_token_logprobs_backward, backward)]:
                start.wait(60)
                refused = sum(f(*args) != 0 for _ in range(10000))
                if refused:
                    wrong.append((f.__name__, V, refused))
            stream.synchronize()
            if not (torch.equal(logprob, want.logprob) and torch.equal(out, want.dlogits) and torch.equal(back_out, back)):
                wrong.append(("results", V))
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            start.abort()
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong


def test_captured_and_replayed():
    x, _ = make(3, 30000, "bf16", seed=20)
    idx, val = lists(x, 9, 1.0, True)
    ti, tv, w = dev(idx, torch.int32), dev(val), dev(np.ones(3))
    t = ti[:, 0].clamp_min(0).contiguous()

    def step():
        a = gs.token_logprobs(x, t, top_k=6, want_entropy=True, want_stats=True)
        b = gs.token_logprobs_backward(x, a.stats, t, w, a.entropy, w)
        c = gs.distill_topk(x, ti, tv, tail=True, want_grad=True, want_stats=True, grad_loss=w)
        d = gs.distill_topk_backward(x, c.stats, ti, tv, w, tail=True)
        return [a.logprob, a.entropy, a.top_idx, a.top_logprob, b, c.loss, c.dlogits, d]

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for s in range(3):
        x.copy_(make(3, 30000, "bf16", seed=30 + s)[0])
        want = step()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_rows_beyond_32_bits_of_elements():
    V, stride = 1000, (1 << 31) + 24
    buf = torch.zeros(stride + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, V), (stride, 1), 0)
    x.copy_(make(2, V, "bf16")[0])
    t = dev([5, 999], torch.int32)
    got = gs.token_logprobs(x, t, top_k=5, dlogits=x, grad_logprob=dev([1.0, 2.0]))
    y = make(2, V, "bf16")[0].clone()
    want = gs.token_logprobs(y, t, top_k=5, want_grad=True, grad_logprob=dev([1.0, 2.0]))
    assert torch.equal(got.top_idx, want.top_idx) and torch.equal(got.logprob, want.logprob)
    assert torch.equal(got.dlogits, want.dlogits)
    assert bool((buf[V:stride] == 0).all())


def test_the_binding_refuses():
    x, _ = make(2, 10, "fp32")
    i, v = dev([[1], [2]], torch.int32), dev([[0.0], [0.0]])
    E = gs.GsparseError
    for call in (lambda: gs.token_logprobs(x.double()), lambda: gs.token_logprobs(x.t()), lambda: gs.token_logprobs(x[0]),
                 lambda: gs.token_logprobs(x, dev([1, 2], torch.int64)), lambda: gs.token_logprobs(x, dev([1], torch.int32)),
                 lambda: gs.token_logprobs(x, temperature=0.0), lambda: gs.token_logprobs(x, temperature=-1.0),
                 lambda: gs.token_logprobs(x, top_k=11), lambda: gs.token_logprobs(x, grad_logprob=v[:, 0].contiguous()),
                 lambda: gs.token_logprobs(x, dlogits=x.half()), lambda: gs.token_logprobs(x, dlogits=x[:1]),
                 lambda: gs.token_logprobs_backward(x, v), lambda: gs.token_logprobs_backward(x, dev(np.ones((2, 2))), top_idx=i),
                 lambda: gs.distill_topk(x, i, v[:1]), lambda: gs.distill_topk(x, i[:, 0], v), lambda: gs.distill_topk(x, i, i),
                 lambda: gs.distill_topk(x, i, v, want_grad=True),
                 lambda: gs.distill_topk_backward(x, dev(np.ones((2, 2))), i, v, v[:, 0].contiguous(), tail=True)):
        with pytest.raises(E):
            call()
