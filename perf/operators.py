"""The operators over vocabulary rows: what is timed, and their plain forms.

token_logprobs: log probabilities of given tokens, the entropy of each row and its most likely
tokens; with the gradient in the same call, or as a backward pass from saved row statistics.
distill_topk: the loss of a student against the (index, value) list of a teacher's most likely
tokens, with the gradient in the same call, or as a backward pass.

Logits are rows over a vocabulary, in fp32, bf16 or fp16, their row stride at least the vocabulary.
z = x * it with it = fp32(1 / temperature); p = softmax(z).
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_LOWEST = torch.finfo(torch.float32).min


def listed():
    return [
        # one step of decoding one sentence, with the alternatives shown to a user: latency
        dict(name="score_1x85000_top5", op="score", dtype="bf16", rows=1, vocab=85000, pad=0, top_k=5, entropy=False,
             temperature=1.0, masked=False),
        # one step of decoding a batch, fp16 logits, alternatives and entropy kept with the tokens
        dict(name="score_64x32000_top20", op="score", dtype="fp16", rows=64, vocab=32000, pad=0, top_k=20, entropy=True,
             temperature=1.25, masked=False),
        # constrained decoding: part of the vocabulary ruled out by -inf, an odd vocabulary, many alternatives
        dict(name="score_777x50021_top64_masked", op="score", dtype="bf16", rows=777, vocab=50021, pad=0, top_k=64,
             entropy=True, temperature=0.5, masked=True),
        # scoring the 80 x 50 tokens of a translation batch
        dict(name="score_4000x85000", op="score", dtype="bf16", rows=4000, vocab=85000, pad=0, top_k=0, entropy=True,
             temperature=1.0, masked=False),
        # the training step of the same batch: log probabilities and the logits' gradient in one call
        dict(name="train_4000x85000", op="train", dtype="bf16", rows=4000, vocab=85000, pad=0, top_k=0, entropy=True,
             temperature=1.0, masked=False),
        # backward pass of a policy step: weights known only after the log probabilities, entropy bonus, alternatives
        dict(name="backward_2048x32003_fp32", op="backward", dtype="fp32", rows=2048, vocab=32003, pad=0, top_k=8,
             entropy=True, temperature=1.0, masked=False),
        # a small classifier distilled in fp32: latency of a training call
        dict(name="distill_16x1000_fp32", op="distill", dtype="fp32", rows=16, vocab=1000, pad=0, k=8, tail=False,
             temperature=4.0, values="fp32"),
        # distillation on the translation batch, the teacher's list renormalised
        dict(name="distill_4000x85000_k32", op="distill", dtype="bf16", rows=4000, vocab=85000, pad=0, k=32, tail=False,
             temperature=2.0, values="fp16"),
        # fp16, odd vocabulary in padded rows, the teacher's remaining mass kept as one more class
        dict(name="distill_2048x50021_k64_tail", op="distill", dtype="fp16", rows=2048, vocab=50021, pad=27, k=64, tail=True,
             temperature=1.0, values="fp32"),
        # validation loss of a large vocabulary, long lists, no gradient
        dict(name="distill_loss_1024x128000_k128", op="distill_loss", dtype="bf16", rows=1024, vocab=128000, pad=0, k=128,
             tail=True, temperature=1.0, values="fp32"),
        # the largest training call
        dict(name="distill_8192x128000_k64", op="distill", dtype="bf16", rows=8192, vocab=128000, pad=0, k=64, tail=False,
             temperature=1.0, values="bf16"),
        # backward pass of its own, fp32 logits
        dict(name="distill_backward_4096x32000_fp32", op="distill_backward", dtype="fp32", rows=4096, vocab=32000, pad=0,
             k=32, tail=True, temperature=2.0, values="fp32"),
    ]


def draw(rng):
    op = rng.choice(["score", "score", "train", "backward", "distill", "distill", "distill_loss", "distill_backward"])
    vocab = int(round(math.exp(rng.uniform(math.log(1000), math.log(160000)))))
    most = min(8192, (1 << 28) // vocab)
    rows = int(round(math.exp(rng.uniform(0.0, math.log(most)))))
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows=rows, vocab=vocab,
                pad=rng.choice([0, 0, 1, 8, 61]), temperature=rng.choice([0.5, 1.0, 1.0, 1.25, 2.0, 4.0]))
    if op in ("score", "train", "backward"):
        case.update(top_k=0 if op == "train" else rng.choice([0, 1, 5, 20, 64, 128]), entropy=rng.random() < 0.6,
                    masked=rng.random() < 0.3)
    else:
        case.update(k=rng.choice([1, 8, 13, 32, 64, 128, 200]), tail=rng.random() < 0.5,
                    values=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
        if case["tail"]:
            case["values"] = "fp32"
    return case


def _it(case):
    """The factor of the logits, as the operators take it: 1 / temperature in fp32."""
    return torch.tensor(1.0 / case["temperature"], dtype=torch.float32).item()


def _in_rows(rows, vocab, bytes_per=4 << 28):
    step = max(1, bytes_per // (4 * vocab))
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def prepare(case, seed):
    dev = "cuda"
    rows, vocab, stride = case["rows"], case["vocab"], case["vocab"] + case["pad"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    # a vocabulary sorted by frequency: the early tokens are the likely ones, every row has its own scores
    # on top, and the token that follows stands out by a margin that differs from row to row
    logits = torch.empty(rows, stride, dtype=_TYPES[case["dtype"]], device=dev)
    prior = -1.1 * torch.log(torch.arange(1, vocab + 1, device=dev, dtype=torch.float32) + 2.7)
    targets = torch.clamp((torch.rand(rows, device=dev, generator=gen) ** 4 * vocab).to(torch.int64), max=vocab - 1)
    margin = torch.rand(rows, device=dev, generator=gen) * 12.0
    lists = "k" in case
    idx, val = [], []
    for a, b in _in_rows(rows, vocab):
        x = torch.randn(b - a, vocab, device=dev, generator=gen).mul_(1.7).add_(prior).add_(8.0)
        x[torch.arange(b - a, device=dev), targets[a:b]] += margin[a:b]
        logits[a:b, :vocab] = x
        if lists:  # the teacher: near the student, its k largest
            x = x.add_(torch.randn(x.shape, device=dev, generator=gen).mul_(0.5))
            v, i = torch.topk(x, min(case["k"], vocab), dim=-1)
            if case["tail"]:
                it = _it(case)
                v = v * it - torch.logsumexp(x * it, -1, keepdim=True)
            idx.append(i)
            val.append(v)
        del x
    if case["pad"]:
        logits[:, vocab:] = float("nan")  # what stands behind a row's last token is not part of it
    if case.get("masked"):  # half of the tokens ruled out; every sixteenth row is padding with nothing left
        keep = torch.rand(vocab, device=dev, generator=gen) < 0.5
        logits[:, :vocab].masked_fill_(~keep, float("-inf"))
        logits[15::16, :vocab] = float("-inf")
    logits = logits[:, :vocab]
    state = dict(case=dict(case), logits=logits, targets=targets.to(torch.int32))
    live = torch.rand(rows, device=dev, generator=gen) < 0.9  # the others are padding
    weight = torch.where(live, 1.0, 0.0) * (0.5 + torch.rand(rows, device=dev, generator=gen))
    if lists:
        i = torch.cat(idx).to(torch.int32)
        v = torch.cat(val)
        mass = torch.softmax(v, -1).cumsum(-1)
        past = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], -1) > 0.999
        i = torch.where(past | ~live[:, None], -1, i)  # lists end where the mass does; padding has none
        v = torch.where(i < 0, 0.0, v)
        state.update(idx=i.contiguous(), val=v.to(_TYPES[case["values"]]).contiguous())
        state["weight"] = weight * case["temperature"] ** 2
    else:
        state["targets"] = torch.where(live, state["targets"], torch.full_like(state["targets"], -1))
        state["weight"] = -weight
        state["weight_entropy"] = 0.01 * weight if case["entropy"] else None
    if case["op"] in ("backward", "distill_backward"):
        # what the forward pass has left: row statistics, entropy, alternatives, each in the type it has there
        d, e, s = _softmax32(logits, _it(case))
        state["stats"] = torch.cat([logits.float().amax(-1, keepdim=True).clamp_min(_LOWEST), s], -1).contiguous()
        if case["op"] == "backward":
            state["entropy"] = _entropy32(d, e, s) if case["entropy"] else None
            state["top_idx"] = state["weight_top"] = None
            if case["top_k"]:
                top = torch.topk(logits.float(), min(case["top_k"], vocab), dim=-1)
                state["top_idx"] = torch.where(top.values > float("-inf"), top.indices, -1).to(torch.int32).contiguous()
                state["weight_top"] = torch.rand(rows, state["top_idx"].shape[1], device=dev, generator=gen) * 0.1
        else:
            out = logits.float()
            if case["tail"]:
                out = out.masked_fill(_member(state["idx"], vocab), float("-inf"))
            d, e, s = _softmax32(out, _it(case))
            rest = torch.cat([out.amax(-1, keepdim=True).clamp_min(_LOWEST), s], -1)
            state["stats"] = torch.cat([state["stats"], rest], -1).contiguous()
    return state


# plain forms --------------------------------------------------------------------------------

def _softmax32(logits, it):
    """(z - max z, its exp, the sum of those), in 32 bits; a row with nothing in it has the sum 0."""
    x = logits.float()
    d = (x - x.amax(-1, keepdim=True).clamp_min(_LOWEST)) * it
    e = torch.exp(d)
    return d, e, e.sum(-1, keepdim=True)


def _entropy32(d, e, s):
    h = s.log() - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / s
    return torch.where(s > 0, h, 0.0).squeeze(-1)


def _member(idx, vocab):
    """Which tokens of each row are in its list (absent entries, -1, go to a column of their own)."""
    at = torch.where(idx < 0, vocab, idx).long()
    return torch.zeros(idx.shape[0], vocab + 1, dtype=torch.bool, device=idx.device).scatter_(1, at, True)[:, :vocab]


def _plain_rows(state, gradient):
    case, logits = state["case"], state["logits"]
    it, vocab = _it(case), case["vocab"]
    d, e, s = _softmax32(logits, it)
    log_s = s.log()
    at = state["targets"].long()
    has = at >= 0
    lp = torch.where(s > 0, d.gather(1, at.clamp_min(0)[:, None]) - log_s, float("-inf")).squeeze(1)
    out = {"logprob": torch.where(has, lp, 0.0)}
    h = _entropy32(d, e, s) if case["entropy"] else None
    if case["entropy"]:
        out["entropy"] = h
    if case["top_k"] and not gradient:
        k = min(case["top_k"], vocab)
        order = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
        left = order.values[:, :k] > float("-inf")
        i = order.indices[:, :k]
        out["top_idx"] = torch.where(left, i, -1).to(torch.int32)
        out["top_logprob"] = torch.where(left, d.gather(1, i) - log_s, float("-inf"))
    if gradient:
        out["dlogits"] = _plain_gradient(state, d, e, s, h)
    return out


def _plain_gradient(state, d, e, s, h):
    case, it = state["case"], _it(state["case"])
    p = torch.where(s > 0, e / s, 0.0)
    at = state["targets"].long()
    g = torch.where(at >= 0, state["weight"], 0.0)[:, None]
    coefficient = g
    if state["weight_entropy"] is not None:
        log_p = torch.where(p > 0, d - s.log(), 0.0)
        coefficient = coefficient + state["weight_entropy"][:, None] * (log_p + h[:, None])
    w_top = state.get("weight_top")
    if w_top is not None:
        w_top = torch.where(state["top_idx"] >= 0, w_top, 0.0)
        coefficient = coefficient + w_top.sum(-1, keepdim=True)
    grad = -p * coefficient
    grad.scatter_add_(1, at.clamp_min(0)[:, None], g)
    if w_top is not None:
        grad.scatter_add_(1, state["top_idx"].long().clamp_min(0), w_top)
    grad = torch.where(s > 0, grad * it, 0.0)
    return grad.to(_TYPES[case["dtype"]])


def _plain_distill(state, loss, gradient):
    case, logits = state["case"], state["logits"]
    it, vocab = _it(case), case["vocab"]
    _, e, s = _softmax32(logits, it)
    there = state["idx"] >= 0
    at = state["idx"].long().clamp_min(0)
    # over the list and in long sums 64 bits: the loss is a small difference, and so is the mass that the list leaves
    v = torch.where(there, state["val"].double(), float("-inf"))
    if case["tail"]:
        log_q = v
    else:
        v = (v - v.amax(-1, keepdim=True).clamp_min(_LOWEST)) * it
        log_q = v - torch.exp(v).sum(-1, keepdim=True).log()
    q = torch.where(there, torch.exp(log_q), 0.0)
    mass = q.sum(-1, keepdim=True)
    rest = torch.clamp(1.0 - mass, min=0.0)
    high = logits.amax(-1, keepdim=True).double().clamp_min(_LOWEST)
    d = (logits.gather(1, at).double() - high) * it
    if case["tail"]:
        # the tokens outside the list by themselves: their sum as the difference of two others would lose its digits
        outside = logits.float().masked_fill(_member(state["idx"], vocab), float("-inf"))
        _, eo, so = _softmax32(outside, it)
        top = outside.amax(-1, keepdim=True).double().clamp_min(_LOWEST)
        log_r = (top - high) * it + eo.sum(-1, keepdim=True, dtype=torch.float64).log()
        log_s = (torch.where(there, d.exp(), 0.0).sum(-1, keepdim=True) + log_r.exp()).log()
        log_r = log_r - log_s
        rest = torch.where(so > 0, rest, 0.0)
    else:
        log_s = e.sum(-1, keepdim=True, dtype=torch.float64).log()
    out = {}
    if loss:
        terms = torch.where(q > 0, q * (log_q - (d - log_s)), 0.0).sum(-1)
        if case["tail"]:
            terms = terms + torch.where(rest > 0, rest * (rest.log() - log_r), 0.0).squeeze(1)
        out["loss"] = terms.float()
    if gradient:
        if case["tail"]:
            grad = (mass + rest).float() * (e / s) - rest.float() * torch.where(so > 0, eo / so, 0.0)
        else:
            grad = mass.float() * (e / s)
        grad.scatter_add_(1, at, -q.float())
        grad = torch.where(s > 0, grad * (it * state["weight"][:, None]), 0.0)
        out["dlogits"] = grad.to(_TYPES[case["dtype"]])
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import compressed_sgd_b200 as gs
        if op == "score":
            r = gs.token_logprobs(state["logits"], state["targets"], top_k=case["top_k"], want_entropy=case["entropy"],
                                  temperature=case["temperature"])
            out = {"logprob": r.logprob, "entropy": r.entropy, "top_idx": r.top_idx, "top_logprob": r.top_logprob}
            return {k: v for k, v in out.items() if v is not None}
        if op == "train":
            r = gs.token_logprobs(state["logits"], state["targets"], want_entropy=case["entropy"],
                                  temperature=case["temperature"], grad_logprob=state["weight"],
                                  grad_entropy=state["weight_entropy"], want_grad=True)
            out = {"logprob": r.logprob, "entropy": r.entropy, "dlogits": r.dlogits}
            return {k: v for k, v in out.items() if v is not None}
        if op == "backward":
            return {"dlogits": gs.token_logprobs_backward(
                state["logits"], state["stats"], state["targets"], grad_logprob=state["weight"], entropy=state["entropy"],
                grad_entropy=state["weight_entropy"], top_idx=state["top_idx"], grad_top=state["weight_top"],
                temperature=case["temperature"])}
        if op == "distill":
            r = gs.distill_topk(state["logits"], state["idx"], state["val"], tail=case["tail"],
                                temperature=case["temperature"], grad_loss=state["weight"], want_grad=True)
            return {"loss": r.loss, "dlogits": r.dlogits}
        if op == "distill_loss":
            return {"loss": gs.distill_topk(state["logits"], state["idx"], state["val"], tail=case["tail"],
                                            temperature=case["temperature"]).loss}
        # the renormalised loss leaves the first two statistics of each row
        stats = state["stats"] if case["tail"] else state["stats"][:, :2].contiguous()
        return {"dlogits": gs.distill_topk_backward(state["logits"], stats, state["idx"], state["val"], state["weight"],
                                                    tail=case["tail"], temperature=case["temperature"])}
    if op == "score":
        return _plain_rows(state, gradient=False)
    if op == "train":
        return _plain_rows(state, gradient=True)
    if op == "backward":
        d, e, s = _softmax32(state["logits"], _it(case))
        return {"dlogits": _plain_gradient(state, d, e, s, state["entropy"])}
    return _plain_distill(state, loss=op != "distill_backward", gradient=op != "distill_loss")


def work(case):
    rows, vocab, size = case["rows"], case["vocab"], 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    forward = op in ("score", "train", "distill", "distill_loss")
    gradient = op not in ("score", "distill_loss")
    entries = rows * vocab
    small = 8  # a target and a result, or a weight and a result, for each row
    if "k" in case:
        small += min(case["k"], vocab) * (4 + (4 if case["values"] == "fp32" else 2)) + 8
        per = 4 * forward + 5 * gradient
    else:
        small += min(case["top_k"], vocab) * 8 + (4 if case["entropy"] else 0) + 8 * gradient
        per = (6 if case["entropy"] else 4) * forward + (7 if case["entropy"] else 4) * gradient
    return {"bytes": entries * size * (2 if gradient else 1) + rows * small, "flops": entries * per}


# the definition in 64 bits ------------------------------------------------------------------

def _exact_rows(case, state, a, b):
    z = state["logits"][a:b].double() * _it(case)
    nothing = torch.isneginf(z).all(-1)
    log_p = torch.log_softmax(torch.where(nothing[:, None], 0.0, z), -1)
    log_p[nothing] = float("-inf")
    p = log_p.exp()
    t = state["targets"][a:b].long()
    ent = -torch.special.xlogy(p, p).sum(-1)
    out = {}
    if case["op"] != "backward":
        out["logprob"] = torch.where(t < 0, 0.0, log_p.gather(1, t.clamp_min(0)[:, None])[:, 0])
        if case["entropy"]:
            out["entropy"] = ent
    if case["op"] == "score":
        if case["top_k"]:
            out["top_logprob"] = torch.topk(log_p, min(case["top_k"], case["vocab"]), dim=-1).values
        return out
    g = torch.where(t < 0, 0.0, state["weight"][a:b].double())
    one = torch.nn.functional.one_hot(t.clamp_min(0), case["vocab"])
    grad = g[:, None] * (one - p)
    if state["weight_entropy"] is not None:
        grad -= state["weight_entropy"][a:b].double()[:, None] * (torch.special.xlogy(p, p) + p * ent[:, None])
    if state.get("weight_top") is not None:
        i = state["top_idx"][a:b].long()
        w = torch.where(i < 0, 0.0, state["weight_top"][a:b].double())
        grad += torch.zeros_like(p).scatter_add_(1, i.clamp_min(0), w) - p * w.sum(-1, keepdim=True)
    grad[nothing] = 0.0
    out["dlogits"] = grad * _it(case)
    return out


def _exact_distill(case, state, a, b):
    z = state["logits"][a:b].double() * _it(case)
    log_p = torch.log_softmax(z, -1)
    i = state["idx"][a:b].long()
    v = state["val"][a:b].double()
    v[i < 0] = float("-inf")
    if not case["tail"]:
        v = torch.where((i < 0).all(-1, keepdim=True), float("-inf"), torch.log_softmax(v * _it(case), -1))
        v[i < 0] = float("-inf")
    q = v.exp()
    student = torch.where(i < 0, 0.0, log_p.gather(1, i.clamp_min(0)))
    loss = (torch.special.xlogy(q, q) - q * student).sum(-1)
    grad = q.sum(-1, keepdim=True) * log_p.exp()
    if case["tail"]:
        rho = (1 - q.sum(-1)).clamp_min(0)
        hit = torch.zeros(b - a, case["vocab"] + 1, dtype=torch.bool, device=z.device)
        hit.scatter_(1, torch.where(i < 0, case["vocab"], i), True)
        outside = log_p.masked_fill(hit[:, :-1], float("-inf"))
        log_r = torch.logsumexp(outside, -1)
        rho = torch.where(torch.isneginf(log_r), 0.0, rho)
        loss += torch.special.xlogy(rho, rho) - torch.where(rho > 0, rho * log_r, 0.0)
        grad += rho[:, None] * (log_p.exp() - torch.softmax(outside, -1).nan_to_num(0.0))
    grad.scatter_add_(1, i.clamp_min(0), -q)
    out = {}
    if case["op"] != "distill_backward":
        out["loss"] = loss
    if case["op"] != "distill_loss":
        out["dlogits"] = grad * (state["weight"][a:b].double()[:, None] * _it(case))
    return out


def exact(case, seed):
    state = prepare(case, seed)
    one = _exact_distill if "k" in case else _exact_rows
    parts = [one(case, state, a, b) for a, b in _in_rows(case["rows"], case["vocab"], 1 << 28)]
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "score" and case["top_k"]:
        out["top_idx"] = None
    return out
