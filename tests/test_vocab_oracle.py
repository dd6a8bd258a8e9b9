"""CPU checks of the losses over vocabulary rows: the 64-bit formulas against hand-worked cases and
differences, and the refusals of the C entry points and of the binding. No kernel runs."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import vocab


@pytest.fixture(scope="module")
def gs():
    from compressed_sgd_b200 import build
    build.build()
    import compressed_sgd_b200
    return compressed_sgd_b200


def _difference(f, x, h=1e-5):
    """Central differences of the scalar f by every finite entry of x."""
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        if np.isfinite(x[i]):
            a, b = x.copy(), x.copy()
            a[i] += h
            b[i] -= h
            out[i] = (f(a) - f(b)) / (2 * h)
    return out


# a central difference with h = 1e-5 is off by h^2 / 6 times the third derivative (below about 10 times the
# weights for these sizes) and by the rounding of the loss, 2^-53 * 10 / h = 1e-10
DIFF = 2e-8


def test_hand_worked_rows():
    x = np.log(np.array([[1.0, 2.0, 5.0], [4.0, 4.0, 0.0 + 1e-300]]))
    x[1, 2] = -np.inf
    lp, ent, idx, val = vocab.token_logprobs(x, 1.0, [2, -1], 2)
    assert np.allclose(lp, [np.log(5 / 8), 0.0])
    assert np.allclose(ent, [-(1 / 8 * np.log(1 / 8) + 1 / 4 * np.log(1 / 4) + 5 / 8 * np.log(5 / 8)), np.log(2)])
    assert idx.tolist() == [[2, 1], [0, 1]] and np.allclose(val, np.log([[5 / 8, 1 / 4], [1 / 2, 1 / 2]]))
    # a list of two against p = (1, 2, 5) / 8: renormalised (1/3, 2/3); with the tail (1/8, 2/8) and 5/8
    i, v = np.array([[0, 1]]), np.log([[1.0, 2.0]])
    assert np.allclose(vocab.distill(x[:1], 1.0, i, v, False), np.log((1 / 3) / (1 / 8)))
    assert np.allclose(vocab.distill(x[:1], 1.0, i, v - np.log(8.0), True), 0.0)
    q = np.array([[0.5, 0.25]])
    want = 0.5 * np.log(0.5 / (1 / 8)) + 0.25 * np.log(0.25 / 0.25) + 0.25 * np.log(0.25 / (5 / 8))
    assert np.allclose(vocab.distill(x[:1], 1.0, i, np.log(q), True), want)


def test_rows_with_nothing_left():
    x = np.full((2, 4), -np.inf)
    lp, ent, idx, val = vocab.token_logprobs(x, 1.0, [1, -1], 2)
    assert np.isneginf(lp[0]) and lp[1] == 0 and (ent == 0).all() and (idx == -1).all() and np.isneginf(val).all()
    assert (vocab.token_logprobs_grad(x, 1.0, [1, -1], [1.0, 1.0], [1.0, 1.0]) == 0).all()
    empty = np.full((2, 3), -1)
    assert (vocab.distill(x, 1.0, empty, np.zeros((2, 3)), True) == 0).all()


@pytest.mark.parametrize("it", [1.0, 0.5, 1.25])
def test_logprob_gradient_against_differences(it):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 7)) * 2
    x[1, 3] = -np.inf
    t = np.array([2, 5, -1])
    g, h = rng.normal(size=3), rng.normal(size=3)
    top = np.array([[0, 3], [1, 1], [6, -1]])
    gt = rng.normal(size=(3, 2))
    gt[top == 3] = 0.0

    def f(y):
        lp = vocab.log_softmax(y, it)
        logprob, ent, _, _ = vocab.token_logprobs(y, it, t)
        s = (g * logprob).sum() + (h * ent).sum()
        for r in range(3):
            for i, w in zip(top[r], gt[r]):
                if i >= 0 and w:
                    s += w * lp[r, i]
        return s

    got = vocab.token_logprobs_grad(x, it, t, g, h, top, gt)
    assert np.abs(got - _difference(f, x)).max() < DIFF


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("it", [1.0, 0.5, 1.25])
def test_distillation_gradient_against_differences(it, tail):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(4, 8)) * 2
    idx = np.array([[0, 3, 5], [7, -1, -1], [2, 2, 6], [-1, -1, -1]])
    val = np.log(rng.uniform(0.05, 0.3, size=(4, 3)))
    g = rng.normal(size=4)
    got = vocab.distill_grad(x, it, idx, val, tail, g)
    assert np.abs(got - _difference(lambda y: (g * vocab.distill(y, it, idx, val, tail)).sum(), x)).max() < DIFF
    assert (got[3] == 0).all()


def test_the_rest_of_a_row_keeps_its_shares_beside_a_huge_entry():
    # beside 1e38 the others have p = 0, but the mass the list leaves still goes to them by their own softmax
    x = np.array([[1e38, np.log(1.0), np.log(3.0)]])
    got = vocab.distill_grad(x, 1.0, np.array([[0]]), np.log([[0.75]]), True, np.ones(1))
    assert np.allclose(got, [[1.0 - 0.75, -0.25 * 0.25, -0.25 * 0.75]])


def test_a_student_like_its_teacher_has_no_loss():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(2, 9))
    _, _, idx, val = vocab.token_logprobs(x, 0.5, None, 4)
    assert np.abs(vocab.distill(x, 0.5, idx, val, True)).max() < 1e-14
    assert np.abs(vocab.distill_grad(x, 0.5, idx, val, True, np.ones(2))).max() < 1e-14


# ---- refusals: found on the host before any launch ---------------------------------------------

INVALID, UNSUPPORTED = 1, 4
BUF = ctypes.create_string_buffer(64)
P = (ctypes.addressof(BUF) + 15) // 16 * 16      # a pointer that no refused call follows
ROWS = dict(logits=P, dtype=1, rows=2, vocab=16, stride=16, it=1.0)


def _score(gs, **kw):
    a = dict(ROWS, targets=P, logprob=P, entropy=None, stats=None, top_k=0, top_idx=None, top_val=None, dlogits=None,
             dstride=0, g=None, h=None)
    a.update(kw)
    return gs.lib().gsparse_token_logprobs(a["logits"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["it"],
                                           a["targets"], a["logprob"], a["entropy"], a["stats"], a["top_k"],
                                           a["top_idx"], a["top_val"], a["dlogits"], a["dstride"], a["g"], a["h"],
                                           None, None)


def _score_backward(gs, **kw):
    a = dict(ROWS, stats=P, targets=P, g=P, entropy=None, h=None, top_k=0, top_idx=None, top_g=None, dlogits=P,
             dstride=16)
    a.update(kw)
    return gs.lib().gsparse_token_logprobs_backward(a["logits"], a["dtype"], a["rows"], a["vocab"], a["stride"],
                                                    a["it"], a["stats"], a["targets"], a["g"], a["entropy"], a["h"],
                                                    a["top_k"], a["top_idx"], a["top_g"], a["dlogits"], a["dstride"],
                                                    None, None)


def _distill(gs, **kw):
    a = dict(ROWS, idx=P, val=P, val_dtype=0, k=4, mode=0, loss=P, stats=None, dlogits=None, dstride=0, g=None)
    a.update(kw)
    return gs.lib().gsparse_distill_topk(a["logits"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["it"],
                                         a["idx"], a["val"], a["val_dtype"], a["k"], a["mode"], a["loss"], a["stats"],
                                         a["dlogits"], a["dstride"], a["g"], None, None)


def _distill_backward(gs, **kw):
    a = dict(ROWS, stats=P, idx=P, val=P, val_dtype=0, k=4, mode=0, g=P, dlogits=P, dstride=16)
    a.update(kw)
    return gs.lib().gsparse_distill_topk_backward(a["logits"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["it"],
                                                  a["stats"], a["idx"], a["val"], a["val_dtype"], a["k"], a["mode"],
                                                  a["g"], a["dlogits"], a["dstride"], None, None)


CALLS = [_score, _score_backward, _distill, _distill_backward]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__[1:])
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(stride=-1), INVALID), (dict(logits=None), INVALID), (dict(logits=P + 1), INVALID),
    (dict(it=0.0), INVALID), (dict(it=-1.0), INVALID), (dict(it=float("nan")), INVALID),
    (dict(it=float("inf")), INVALID), (dict(it=3e38), UNSUPPORTED), (dict(it=1e-45), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1, stride=1 << 25, dstride=1 << 25), UNSUPPORTED), (dict(rows=1 << 28), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED),
])
def test_common_refusals(gs, call, kw, want):
    assert call(gs, **kw) == want


@pytest.mark.parametrize("call,kw,want", [
    (_score, dict(targets=None), INVALID),
    (_score, dict(top_k=-1), INVALID), (_score, dict(top_k=17, top_idx=P, top_val=P), INVALID),
    (_score, dict(top_k=2), INVALID), (_score, dict(top_k=257, vocab=300, stride=300, top_idx=P, top_val=P), UNSUPPORTED),
    (_score, dict(g=P), INVALID), (_score, dict(h=P), INVALID),
    (_score, dict(dlogits=P, dstride=15, g=P), INVALID), (_score, dict(dlogits=P + 1, dstride=16, g=P), INVALID),
    (_score, dict(dlogits=P, stride=20, dstride=16, g=P), INVALID),
    (_score, dict(dlogits=P + 16, dstride=16, g=P, targets=None, logprob=None), INVALID),
    (_score_backward, dict(stats=None), INVALID), (_score_backward, dict(dlogits=None), INVALID),
    (_score_backward, dict(targets=None), INVALID), (_score_backward, dict(h=P), INVALID),
    (_score_backward, dict(top_k=2), INVALID), (_score_backward, dict(top_k=2, top_idx=P), INVALID),
    (_score_backward, dict(dstride=15), INVALID),
    (_distill, dict(val_dtype=5), INVALID), (_distill, dict(k=0), INVALID), (_distill, dict(k=257), UNSUPPORTED),
    (_distill, dict(mode=2), INVALID), (_distill, dict(idx=None), INVALID), (_distill, dict(val=None), INVALID),
    (_distill, dict(loss=None), INVALID), (_distill, dict(g=P), INVALID), (_distill, dict(dlogits=P, dstride=16), INVALID),
    (_distill_backward, dict(g=None), INVALID), (_distill_backward, dict(stats=None), INVALID),
    (_distill_backward, dict(dlogits=None), INVALID), (_distill_backward, dict(mode=-1), INVALID),
    (_distill_backward, dict(k=0), INVALID), (_distill_backward, dict(dstride=1), INVALID),
])
def test_refusals(gs, call, kw, want):
    assert call(gs, **kw) == want


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__[1:])
def test_no_rows_is_no_work(gs, call):
    assert call(gs, rows=0, logits=None, dlogits=None, g=None) == 0


def test_the_binding_takes_device_tensors_only(gs):
    x, i, v = torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    for call in (lambda: gs.token_logprobs(x), lambda: gs.token_logprobs_backward(x, torch.zeros(2, 2)),
                 lambda: gs.distill_topk(x, i, v), lambda: gs.distill_topk_backward(x, torch.zeros(2, 2), i, v, v[:, 0])):
        with pytest.raises(gs.GsparseError, match="CUDA"):
            call()
