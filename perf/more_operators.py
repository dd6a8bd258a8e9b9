"""A layer in 8 bits and its gradient: what is timed, and the plain forms.

norm: the residual's addition and the root-mean-square norm, its output in 8 bits with a scale per row.
norm_backward: its gradient by the input and by the weight.
quantize: rows in 8 bits with a scale each, and read back.
product: the product in 8-bit integers with scales for each token and channel.
grad_input, grad_weight, grad_both: the product's gradients, read from the 8-bit weights and activations.

Rows in 8 bits: scale = 2^e with the smallest e >= -126 for which no entry exceeds 127 * 2^e, value =
round-half-even(y / 2^e) * 2^e, which bf16 holds exactly.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-6


def listed():
    return [
        # one token between two layers while a sentence is decoded: latency
        dict(name="norm_1x512", op="norm", dtype="bf16", rows=1, depth=512, residual=True),
        # a training batch of long sequences before a wide layer
        dict(name="norm_8192x4096", op="norm", dtype="bf16", rows=8192, depth=4096, residual=True),
        # the 80 x 50 tokens of a translation batch, on the way back
        dict(name="norm_backward_4000x512", op="norm_backward", dtype="bf16", rows=4000, depth=512, residual=True),
        # odd sizes in fp32, a norm without a stream beside it
        dict(name="norm_backward_2047x1001_fp32", op="norm_backward", dtype="fp32", rows=2047, depth=1001, residual=False),
        # activations of an odd width kept in 8 bits, fp16
        dict(name="quantize_777x1001_fp16", op="quantize", dtype="fp16", rows=777, depth=1001),
        # the weights of the vocabulary's matrix after an optimiser's step
        dict(name="quantize_85000x512_fp32", op="quantize", dtype="fp32", rows=85000, depth=512),
        # the output layer for one token of decoding
        dict(name="product_1x85000x512", op="product", dtype="bf16", tokens=1, channels=85000, depth=512),
        # the output layer over a translation batch
        dict(name="product_4000x85000x512", op="product", dtype="bf16", tokens=4000, channels=85000, depth=512),
        # the largest: a wide layer, an odd vocabulary, fp16 out
        dict(name="product_8192x32003x4096", op="product", dtype="fp16", tokens=8192, channels=32003, depth=4096),
        # the gradient that goes on into the layers below
        dict(name="grad_input_4000x85000x512", op="grad_input", dtype="bf16", tokens=4000, channels=85000, depth=512),
        # the gradient of the vocabulary's matrix, which is what is compressed
        dict(name="grad_weight_4000x85000x512", op="grad_weight", dtype="bf16", tokens=4000, channels=85000, depth=512),
        # a classifier of 1000 classes over 2048 features, fp32 gradients
        dict(name="grad_both_256x1000x2048_fp32", op="grad_both", dtype="fp32", tokens=256, channels=1000, depth=2048),
    ]


_MOST_FLOPS = 2 * 8192 * 32003 * 4096


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "quantize", "product", "product", "grad_input", "grad_weight", "grad_both"])
    depth = _spread(rng, 64, 8192)
    if rng.random() < 0.6:
        depth = (depth + 31) // 32 * 32
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_backward", "quantize"):
        rows = _spread(rng, 1, min(85000, (1 << 25) // depth))
        case = dict(op=op, dtype=dtype, rows=rows, depth=depth)
        if op != "quantize":
            case["residual"] = rng.random() < 0.7
        return case
    channels = _spread(rng, 100, 128000)
    # fp32 gradients are three times the products
    most = min(8192, (1 << 28) // channels, _MOST_FLOPS // (8 * channels * depth))
    tokens = _spread(rng, 1, max(2, most))
    return dict(op=op, dtype=dtype, tokens=tokens, channels=channels, depth=depth)


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return gen


def _activations(gen, rows, depth):
    """A stream of activations: channels of different sizes, a few of them much larger than the others."""
    size = torch.exp(0.4 * torch.randn(depth, device="cuda", generator=gen))
    size = torch.where(torch.rand(depth, device="cuda", generator=gen) < 0.01, size * 12.0, size)
    return torch.randn(rows, depth, device="cuda", generator=gen) * size


def _held(x):
    """fp32 rows in 8 bits as the framework keeps them: int8 rows that start at multiples of 16 bytes, and scales."""
    q, scale = _rows_in_8_bits(x)
    stride = (x.shape[1] + 15) // 16 * 16
    held = torch.zeros(x.shape[0], stride, dtype=torch.int8, device="cuda")
    held[:, :x.shape[1]] = q
    return held[:, :x.shape[1]], scale


def prepare(case, seed):
    gen = _generator(seed)
    dtype = _TYPES[case["dtype"]]
    op = case["op"]
    state = dict(case=dict(case))
    depth = case["depth"]
    if op in ("norm", "norm_backward", "quantize"):
        rows = case["rows"]
        x = _activations(gen, rows, depth)
        if rows > 8:
            x[7::64] = 0.0   # padding
        if op == "quantize":
            state["x"] = x.to(dtype)
            return state
        state["weight"] = 1.0 + 0.1 * torch.randn(depth, device="cuda", generator=gen)
        state["residual"] = (2.0 * _activations(gen, rows, depth)).to(dtype) if case["residual"] else None
        if op == "norm":
            state["x"] = x.to(dtype)
            return state
        # what the forward pass has left, and the gradients that come in
        state["h"] = (x + state["residual"].float()).to(dtype) if case["residual"] else x.to(dtype)
        state["rstd"] = torch.rsqrt(state["h"].double().square().mean(-1) + _EPS).float()
        state["dy"] = (0.01 * torch.randn(rows, depth, device="cuda", generator=gen)).to(dtype)
        state["dh"] = (0.01 * torch.randn(rows, depth, device="cuda", generator=gen)).to(dtype) if case["residual"] else None
        state["residual"] = None
        return state
    tokens, channels = case["tokens"], case["channels"]
    if op != "grad_input":
        state["x"], state["x_scale"] = _held(_activations(gen, tokens, depth))
    if op != "grad_weight":
        w = torch.randn(channels, depth, device="cuda", generator=gen) * depth ** -0.5
        w *= torch.exp(0.5 * torch.randn(channels, 1, device="cuda", generator=gen))
        state["w"], state["w_scale"] = _held(w)
        del w
    if op != "product":
        # the gradient of a loss over the channels: probabilities, less one at each target; a tenth of the tokens is padding. Rows as
        # the framework lays logits out, at multiples of 16 bytes
        size = 4 if case["dtype"] == "fp32" else 2
        stride = (channels + 16 // size - 1) // (16 // size) * (16 // size)
        dout = torch.zeros(tokens, stride, dtype=dtype, device="cuda")
        step = max(1, (1 << 28) // channels)
        for a in range(0, tokens, step):
            b = min(tokens, a + step)
            p = torch.softmax(2.0 * torch.randn(b - a, channels, device="cuda", generator=gen), -1)
            target = torch.randint(channels, (b - a, 1), device="cuda", generator=gen)
            p.scatter_add_(1, target, torch.full((b - a, 1), -1.0, device="cuda"))
            live = torch.rand(b - a, 1, device="cuda", generator=gen) < 0.9
            dout[a:b, :channels] = p * torch.where(live, 64.0, 0.0)   # a loss scaled up, as fp16 needs it
        state["dout"] = dout[:, :channels]
    return state


# plain forms --------------------------------------------------------------------------------

def _rows_in_8_bits(y):
    """(q, scale) of fp32 or fp64 rows. frexp: y = m 2^e with 1/2 <= m < 1; 127/128 is the border of m."""
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True))
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp_min(-126)
    one = torch.ones_like(m, dtype=torch.float64)
    q = torch.round(y.double() * torch.ldexp(one, -e))
    return q.to(torch.int8), torch.ldexp(one, e).float().squeeze(-1)


def _plain_norm(state):
    x, residual = state["x"], state["residual"]
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    # values next to a border between two steps of the 8 bits: 64
    wide = h.double()
    rstd = torch.rsqrt(wide.square().mean(-1, keepdim=True) + _EPS)
    q, scale = _rows_in_8_bits(wide * rstd * state["weight"].double())
    out = {"y": (q.float() * scale[:, None]).to(torch.bfloat16), "rstd": rstd.float().squeeze(-1)}
    if residual is not None:
        out["h"] = h
    return out


def _plain_norm_backward(state):
    h, dy, r = state["h"].float(), state["dy"].float(), state["rstd"][:, None]
    g = dy * state["weight"]
    dx = r * (g - h * (r * r * (g * h).mean(-1, keepdim=True)))
    if state["dh"] is not None:
        dx = dx + state["dh"].float()
    return {"dx": dx.to(state["h"].dtype), "dweight": (dy * h * r).sum(0)}


def _plain_quantize(state):
    q, scale = _rows_in_8_bits(state["x"].float())
    return {"y": (q.float() * scale[:, None]).to(torch.bfloat16)}


def run(state):
    case = state["case"]
    op = case["op"]
    dtype = _TYPES[case["dtype"]]
    if own:
        import compressed_sgd_b200 as gs
        if op == "norm":
            r = gs.rms_norm(state["x"], state["weight"], state["residual"], eps=_EPS, want_q=True, want_rstd=True)
            out = {"y": gs.dequantize_rows(r.q, torch.bfloat16), "rstd": r.rstd}
            if state["residual"] is not None:
                out["h"] = r.h
            return out
        if op == "norm_backward":
            r = gs.rms_norm_backward(state["h"], state["weight"], state["rstd"], state["dy"], state["dh"])
            return {"dx": r.dx, "dweight": r.dweight}
        if op == "quantize":
            return {"y": gs.dequantize_rows(gs.quantize_rows(state["x"]), torch.bfloat16)}
        if op == "product":
            return {"out": gs.linear_q8(gs.QuantRows(state["x"], state["x_scale"]), gs.QuantRows(state["w"], state["w_scale"]), dtype)}
        out = {}
        if op != "grad_weight":
            out["dx"] = gs.linear_q8_grad_input(state["dout"], gs.QuantRows(state["w"], state["w_scale"]))
        if op != "grad_input":
            out["dweight"] = gs.linear_q8_grad_weight(state["dout"], gs.QuantRows(state["x"], state["x_scale"]))
        return out
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_backward":
        return _plain_norm_backward(state)
    if op == "quantize":
        return _plain_quantize(state)
    if op == "product":
        sums = state["x"].float() @ state["w"].float().t()
        return {"out": (sums * state["x_scale"][:, None] * state["w_scale"]).to(dtype)}
    out = {}
    dout = state["dout"].float()
    if op != "grad_weight":
        out["dx"] = (dout @ (state["w"].float() * state["w_scale"][:, None])).to(dtype)
    if op != "grad_input":
        out["dweight"] = dout.t() @ (state["x"].float() * state["x_scale"][:, None])
    return out


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    op, depth = case["op"], case["depth"]
    if op in ("norm", "norm_backward", "quantize"):
        rows = case["rows"]
        entries = rows * depth
        if op == "quantize":       # read, held in 8 bits, read back
            return {"bytes": entries * (size + 1 + 1 + 2) + 8 * rows, "flops": 4 * entries}
        both = 2 if case["residual"] else 1
        if op == "norm":           # x, residual; h, the 8 bits, read back
            return {"bytes": entries * (size * (both + both - 1) + 1 + 1 + 2) + 4 * depth + 12 * rows, "flops": 8 * entries}
        return {"bytes": entries * size * (2 + both) + 8 * depth + 4 * rows, "flops": 10 * entries}
    tokens, channels = case["tokens"], case["channels"]
    x, w, dout = tokens * depth + 4 * tokens, channels * depth + 4 * channels, size * tokens * channels
    once = 2 * tokens * channels * depth
    if op == "product":
        return {"bytes": x + w + dout, "flops": once}
    if op == "grad_input":
        return {"bytes": dout + w + size * tokens * depth, "flops": once}
    if op == "grad_weight":
        return {"bytes": dout + x + 4 * channels * depth, "flops": once}
    return {"bytes": dout + w + x + size * tokens * depth + 4 * channels * depth, "flops": 2 * once}


# the definition in 64 bits ------------------------------------------------------------------

def _exact_8_bits(y):
    """The values that rows in 8 bits stand for, by counting up from the smallest scale's exponent."""
    top = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / 127.0)) - 1.0
    e = torch.where(torch.exp2(e) * 127.0 < top, e + 1.0, e)
    e = torch.where(torch.exp2(e) * 127.0 < top, e + 1.0, e).clamp_min(-126.0)
    scale = torch.exp2(e)
    return torch.round(y / scale) * scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"y": _exact_8_bits(s["x"].double())}
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            # the sum as it is held: its type is part of the definition
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        r = (h.pow(2).sum(-1) / case["depth"] + _EPS) ** -0.5
        out = {"y": _exact_8_bits(h * r[:, None] * s["weight"].double()), "rstd": r}
        if s["residual"] is not None:
            out["h"] = s["x"].double() + s["residual"].double()
        return out
    if op == "norm_backward":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        inner = torch.einsum("tk,tk,k->t", dy, h, s["weight"].double()) / case["depth"]
        dx = r[:, None] * dy * s["weight"].double() - (r ** 3 * inner)[:, None] * h
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("tk,tk,t->k", dy, h, r)}
    if op == "product":
        x = s["x"].double() * s["x_scale"].double()[:, None]
        return {"out": x @ (s["w"].double() * s["w_scale"].double()[:, None]).t()}
    out = {}
    dout = s["dout"].double()
    if op != "grad_weight":
        out["dx"] = torch.einsum("tn,nk->tk", dout * s["w_scale"].double(), s["w"].double())
    if op != "grad_input":
        out["dweight"] = torch.einsum("tn,tk->nk", dout * s["x_scale"].double()[:, None], s["x"].double())
    return out
