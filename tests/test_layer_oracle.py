"""The layer in 8 bits without a GPU: the 64-bit formulas (oracle/layer.py) against hand-worked values and differences, and
every refusal of the entry points and of the binding. No kernel runs."""
import numpy as np
import pytest
import torch

from oracle import layer

INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 4
P = 1 << 20        # a well-aligned address that no call may follow: the refusal comes first
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def gs():
    from compressed_sgd_b200 import build
    build.build()
    import compressed_sgd_b200
    return compressed_sgd_b200


def test_scales_by_hand():
    assert layer.scale_of(127.0) == 1.0 and layer.scale_of(np.nextafter(127.0, 128.0)) == 2.0
    assert layer.scale_of(1.0) == 2.0 ** -6 and layer.scale_of(63.5) == 0.5 and layer.scale_of(0.0) == 2.0 ** -126
    assert layer.scale_of(2.0 ** -149) == 2.0 ** -126 and layer.scale_of(float(np.finfo(np.float32).max)) == 2.0 ** 121


def test_rows_by_hand():
    q, s = layer.quantize_rows(np.array([[1.0, -0.5, 1.5, 2.5, 127.0], [254.0, 1.0, 3.0, -5.0, 0.0], [0.0] * 5,
                                         [1.0, np.inf, 0, 0, 0], [np.nan, 1, 1, 1, 1]]))
    assert q.tolist() == [[1, 0, 2, 2, 127], [127, 0, 2, -2, 0], [0] * 5, [0] * 5, [0] * 5]   # to even at the half
    assert s[:3].tolist() == [1.0, 2.0, 2.0 ** -126] and np.isnan(s[3:]).all()


def test_norm_by_hand():
    y, r = layer.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(r, np.sqrt(2) / 5) and np.allclose(y, [[3 * np.sqrt(2) / 5, 8 * np.sqrt(2) / 5]])


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w, dy, dh = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    f = lambda h, w: np.sum(layer.rms_norm(h, w, 0.1)[0] * dy) + np.sum(h * dh)   # noqa: E731
    dx, dw = layer.rms_norm_grad(h, w, 0.1, dy, dh)
    step = 1e-6
    for at in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[at] = step
        assert abs((f(h + e, w) - f(h - e, w)) / (2 * step) - dx[at]) < 1e-7
    for k in range(7):
        e = np.zeros(7)
        e[k] = step
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * step) - dw[k]) < 1e-7


def test_product_and_its_gradients_against_differences():
    rng = np.random.default_rng(1)
    xq, wq = rng.integers(-127, 128, (3, 5)), rng.integers(-127, 128, (4, 5))
    xs, ws = 2.0 ** rng.integers(-3, 3, 3), 2.0 ** rng.integers(-3, 3, 4)
    out = layer.linear(xq, xs, wq, ws)
    x, w = xq * xs[:, None], wq * ws[:, None]
    assert np.array_equal(out, x @ w.T)
    dout = rng.normal(size=(3, 4))
    f = lambda x, w: np.sum(dout * (x @ w.T))   # noqa: E731
    dx, dw = layer.linear_grad_input(dout, wq, ws), layer.linear_grad_weight(dout, xq, xs)
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = 1.0
        assert abs(f(x + e, w) - f(x - e, w) - 2 * dx[at]) < 1e-8 * (1 + abs(f(x, w)))
    for at in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[at] = 1.0
        assert abs(f(x, w + e) - f(x, w - e) - 2 * dw[at]) < 1e-8 * (1 + abs(f(x, w)))


# refusals -------------------------------------------------------------------------------------------

def _quantize(gs, **kw):
    a = dict(x=P, dtype=F32, rows=3, depth=40, stride=40, q=P, q_stride=48, scale=P) | kw
    return gs.lib().gsparse_quantize_rows(a["x"], a["dtype"], a["rows"], a["depth"], a["stride"], a["q"], a["q_stride"], a["scale"], None)


def _dequantize(gs, **kw):
    a = dict(q=P, q_stride=48, scale=P, rows=3, depth=40, x=P, dtype=F32, stride=40) | kw
    return gs.lib().gsparse_dequantize_rows(a["q"], a["q_stride"], a["scale"], a["rows"], a["depth"], a["x"], a["dtype"], a["stride"], None)


def _norm(gs, **kw):
    a = dict(x=P, stride=40, residual=2 * P, residual_stride=40, weight=P, weight_dtype=F32, dtype=F32, rows=3, depth=40, eps=1e-6,
             h=3 * P, h_stride=40, y=4 * P, y_stride=40, q=P, q_stride=48, scale=P, rstd=P) | kw
    return gs.lib().gsparse_rms_norm(a["x"], a["stride"], a["residual"], a["residual_stride"], a["weight"], a["weight_dtype"], a["dtype"],
                                     a["rows"], a["depth"], a["eps"], a["h"], a["h_stride"], a["y"], a["y_stride"], a["q"], a["q_stride"],
                                     a["scale"], a["rstd"], None)


def _norm_backward(gs, **kw):
    a = dict(x=P, stride=40, weight=P, weight_dtype=F32, rstd=P, dy=2 * P, dy_stride=40, dh=3 * P, dh_stride=40, dtype=F32, rows=3,
             depth=40, dx=4 * P, dx_stride=40, dweight=P, workspace=P, bytes=1 << 20) | kw
    return gs.lib().gsparse_rms_norm_backward(a["x"], a["stride"], a["weight"], a["weight_dtype"], a["rstd"], a["dy"], a["dy_stride"],
                                              a["dh"], a["dh_stride"], a["dtype"], a["rows"], a["depth"], a["dx"], a["dx_stride"],
                                              a["dweight"], a["workspace"], a["bytes"], None)


ROW_CALLS = [_quantize, _dequantize, _norm, _norm_backward]


@pytest.mark.parametrize("call", ROW_CALLS, ids=lambda f: f.__name__[1:])
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(depth=0), INVALID), (dict(x=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(stride=-1), INVALID), (dict(depth=(1 << 15) + 1, stride=1 << 16, q_stride=1 << 16), UNSUPPORTED),
    (dict(rows=(1 << 26) + 1), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
])
def test_common_refusals_of_rows(gs, call, kw, want):
    assert call(gs, **kw) == want


@pytest.mark.parametrize("call", [_quantize, _dequantize, _norm], ids=lambda f: f.__name__[1:])
@pytest.mark.parametrize("kw", [dict(q=None), dict(scale=None), dict(q=P + 8), dict(q_stride=40), dict(q_stride=32), dict(scale=P + 2)])
def test_refusals_of_8_bits(gs, call, kw):
    assert call(gs, **kw) == INVALID


@pytest.mark.parametrize("call,kw,want", [
    (_dequantize, dict(stride=39), INVALID),
    (_norm, dict(depth=(1 << 14) + 1), UNSUPPORTED), (_norm, dict(weight=None), INVALID), (_norm, dict(weight=P + 2), INVALID),
    (_norm, dict(weight_dtype=3), INVALID), (_norm, dict(eps=0.0), INVALID), (_norm, dict(eps=-1.0), INVALID),
    (_norm, dict(eps=float("nan")), INVALID), (_norm, dict(eps=float("inf")), INVALID), (_norm, dict(eps=1e-39), INVALID),
    (_norm, dict(residual=P + 1), INVALID), (_norm, dict(h_stride=39), INVALID), (_norm, dict(y_stride=39), INVALID),
    (_norm, dict(h=P, h_stride=44), INVALID), (_norm, dict(h=2 * P, h_stride=44), INVALID), (_norm, dict(rstd=P + 1), INVALID),
    (_norm_backward, dict(depth=(1 << 14) + 1), UNSUPPORTED), (_norm_backward, dict(weight=None), INVALID),
    (_norm_backward, dict(weight_dtype=7), INVALID), (_norm_backward, dict(rstd=None), INVALID), (_norm_backward, dict(rstd=P + 1), INVALID),
    (_norm_backward, dict(dy=None), INVALID), (_norm_backward, dict(dh=P + 2), INVALID), (_norm_backward, dict(dx=None), INVALID),
    (_norm_backward, dict(dx_stride=39), INVALID), (_norm_backward, dict(dx=P, dx_stride=44), INVALID),
    (_norm_backward, dict(dx=2 * P, dx_stride=44), INVALID), (_norm_backward, dict(dx=3 * P, dx_stride=44), INVALID),
    (_norm_backward, dict(dweight=P + 1), INVALID), (_norm_backward, dict(workspace=None), WORKSPACE),
    (_norm_backward, dict(workspace=P + 16), WORKSPACE), (_norm_backward, dict(bytes=100), WORKSPACE),
])
def test_refusals_of_rows(gs, call, kw, want):
    assert call(gs, **kw) == want


@pytest.mark.parametrize("call", ROW_CALLS, ids=lambda f: f.__name__[1:])
def test_no_rows_is_no_work(gs, call):
    nothing = dict(rows=0, x=None, q=None, scale=None, dy=None, dx=None, h=None, y=None)
    if call is _norm_backward:
        nothing["dweight"] = None
    assert call(gs, **nothing) == 0


def _product(gs, **kw):
    a = dict(x=P, x_stride=48, xs=P, w=P, w_stride=48, ws=P, tokens=30, channels=5, depth=40, out=P, out_dtype=F32, out_stride=5,
             workspace=P, bytes=1 << 40) | kw
    return gs.lib().gsparse_linear_q8(a["x"], a["x_stride"], a["xs"], a["w"], a["w_stride"], a["ws"], a["tokens"], a["channels"],
                                      a["depth"], a["out"], a["out_dtype"], a["out_stride"], a["workspace"], a["bytes"], None, None)


def _grad_input(gs, **kw):
    a = dict(dout=P, dtype=F32, dout_stride=5, w=P, w_stride=48, ws=P, tokens=30, channels=5, depth=40, out=P, out_dtype=F32, out_stride=40,
             workspace=P, bytes=1 << 40) | kw
    return gs.lib().gsparse_linear_q8_grad_input(a["dout"], a["dtype"], a["dout_stride"], a["w"], a["w_stride"], a["ws"], a["tokens"],
                                                 a["channels"], a["depth"], a["out"], a["out_dtype"], a["out_stride"], a["workspace"],
                                                 a["bytes"], None, None)


def _grad_weight(gs, **kw):
    a = dict(dout=P, dtype=F32, dout_stride=5, x=P, x_stride=48, xs=P, tokens=30, channels=5, depth=40, out=P, out_stride=40,
             workspace=P, bytes=1 << 40) | kw
    return gs.lib().gsparse_linear_q8_grad_weight(a["dout"], a["dtype"], a["dout_stride"], a["x"], a["x_stride"], a["xs"], a["tokens"],
                                                  a["channels"], a["depth"], a["out"], a["out_stride"], a["workspace"], a["bytes"],
                                                  None, None)


PRODUCTS = [_product, _grad_input, _grad_weight]


@pytest.mark.parametrize("call", PRODUCTS, ids=lambda f: f.__name__[1:])
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(channels=0), INVALID), (dict(depth=0), INVALID), (dict(depth=(1 << 15) + 1), UNSUPPORTED),
    (dict(tokens=(1 << 26) + 1), UNSUPPORTED), (dict(channels=(1 << 26) + 1), UNSUPPORTED), (dict(out=None), INVALID),
    (dict(out=P + 1), INVALID), (dict(out_stride=4), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace=P + 128), WORKSPACE),
    (dict(bytes=100), WORKSPACE),
])
def test_common_refusals_of_products(gs, call, kw, want):
    assert call(gs, **kw) == want


@pytest.mark.parametrize("call,kw", [
    (c, k) for c in PRODUCTS for k in (dict(x=None), dict(x=P + 8), dict(x_stride=40), dict(x_stride=32), dict(xs=None), dict(xs=P + 2))
    if c is not _grad_input
] + [
    (c, k) for c in PRODUCTS for k in (dict(w=None), dict(w=P + 8), dict(w_stride=40), dict(w_stride=32), dict(ws=None), dict(ws=P + 2))
    if c is not _grad_weight
] + [
    (c, k) for c in (_grad_input, _grad_weight) for k in (dict(dout=None), dict(dout=P + 2), dict(dout_stride=-1), dict(dtype=3))
] + [(_product, dict(out_dtype=3)), (_grad_input, dict(out_dtype=-1))])
def test_refusals_of_products(gs, call, kw):
    assert call(gs, **kw) == INVALID


def test_no_tokens_is_no_work(gs):
    assert _product(gs, tokens=0, x=None, out=None, workspace=None) == 0
    assert _grad_input(gs, tokens=0, dout=None, out=None, workspace=None) == 0


@pytest.mark.parametrize("tokens,channels,depth", [(0, 5, 40), (1, 1, 1), (1 << 26, 1, 1), (1, 1 << 26, 1), (1 << 20, 1 << 20, 1 << 15)])
def test_workspace_queries_of_any_size(gs, tokens, channels, depth):
    """A size, or 0 where the call is refused or needs nothing; never an error of arithmetic."""
    lib = gs.lib()
    assert 0 <= lib.gsparse_linear_q8_workspace_size(tokens, channels, depth) < 1 << 50
    for f in (lib.gsparse_linear_q8_grad_input_workspace_size, lib.gsparse_linear_q8_grad_weight_workspace_size):
        for dtype in (F32, BF16, F16):
            assert 0 <= f(P, dtype, channels, tokens, channels, depth) < 1 << 50
    assert 0 <= lib.gsparse_rms_norm_backward_workspace_size(tokens, depth) < 1 << 50


def test_workspace_queries_refuse_what_the_calls_refuse(gs):
    lib = gs.lib()
    assert lib.gsparse_rms_norm_backward_workspace_size(1000, 512) >= 512 * 4
    assert lib.gsparse_rms_norm_backward_workspace_size(-1, 512) == 0 and lib.gsparse_rms_norm_backward_workspace_size(1, 0) == 0
    assert lib.gsparse_linear_q8_workspace_size(30, 5, 40) > 0 and lib.gsparse_linear_q8_workspace_size(3, 0, 40) == 0
    for f in (lib.gsparse_linear_q8_grad_input_workspace_size, lib.gsparse_linear_q8_grad_weight_workspace_size):
        assert f(P, F32, 5, 30, 5, 40) > 0 and f(P, 3, 5, 3, 5, 40) == 0 and f(P, F32, 5, 3, 5, 0) == 0


def test_the_binding_takes_device_tensors_only(gs):
    x, w = torch.zeros(2, 16), torch.ones(16)
    q = gs.QuantRows(torch.zeros(2, 16, dtype=torch.int8), torch.ones(2))
    for call in (lambda: gs.quantize_rows(x), lambda: gs.dequantize_rows(q), lambda: gs.rms_norm(x, w),
                 lambda: gs.rms_norm_backward(x, w, torch.ones(2), x), lambda: gs.linear_q8(q, q),
                 lambda: gs.linear_q8_grad_input(torch.zeros(3, 2), q), lambda: gs.linear_q8_grad_weight(torch.zeros(2, 3), q)):
        with pytest.raises(gs.GsparseError, match="CUDA"):
            call()


class _Device:
    """A stand-in for the switch of the current device."""
    current = 0

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.before, _Device.current = _Device.current, self.index

    def __exit__(self, *_):
        _Device.current = self.before


def test_workspace_sizes_are_those_of_the_tensors_device(gs, monkeypatch):
    """Two devices with other numbers of SMs: each call gets its own device's size, whichever was asked first."""
    class Lib:
        @staticmethod
        def gsparse_linear_q8_workspace_size(tokens, channels, depth):
            return 1000 * (1 + _Device.current) + tokens

    monkeypatch.setattr(gs, "lib", lambda: Lib)
    monkeypatch.setattr(gs, "_current_device", lambda: _Device.current)
    monkeypatch.setattr(gs.torch.cuda, "device", _Device)
    gs._layer_workspace_size.cache_clear()
    try:
        class Like:
            def __init__(self, index):
                self.device = torch.device("cuda", index)

            def new_empty(self, size, dtype):
                return torch.empty(size, dtype=dtype)

        for _ in range(2):
            for index in (0, 1, 0):
                assert gs._scratch(None, Like(index), "gsparse_linear_q8_workspace_size", 30, 5, 40)[2] == 1000 * (1 + index) + 30
                assert _Device.current == 0
    finally:
        gs._layer_workspace_size.cache_clear()


def test_workspaces_of_another_device_or_with_shared_entries_are_refused(gs):
    class Like:
        device = torch.device("cuda", 0)

    class Workspace:                       # as torch shows one
        def __init__(self, device, t):
            self.device, self.t = torch.device(device), t

        def __getattr__(self, name):
            return getattr(self.t, name)

    t = torch.empty(64, dtype=torch.float32)
    for bad in (t, Workspace("cuda:1", t), Workspace("cuda:0", t[:1].expand(1 << 20)), Workspace("cuda:0", t[::2])):
        with pytest.raises(gs.GsparseError, match="workspace"):
            gs._scratch(bad, Like, "gsparse_linear_q8_workspace_size", 30, 5, 40)
    assert gs._scratch(Workspace("cuda:0", t), Like, "gsparse_linear_q8_workspace_size", 30, 5, 40)[1:] == (t.data_ptr(), 256)
