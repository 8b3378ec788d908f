"""Cases of the operators around a trained layer: layer norm with the residual's sum (``norm``:
forward alone, or forward and backward), log probabilities of given tokens with entropy and top
alternatives (``logprob``: forward alone, or with the gradient of the scores), and the global norm
of many gradients with clipping (``clip``, or the norm alone).

``run`` computes a case in plain torch operations of 32 bits (sums of squares in 64), or with the
framework's kernels when ``own`` is true; ``exact`` computes it from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-5          # under the root of the norm's variance
CLIP_EPS = 1e-6     # beside the norm that clipping divides by
MOST_SCORES = 8192 * 131072      # of a drawn training pass
MOST_TOP_SCORES = 1024 * 131072  # of a drawn pass with alternatives
MOST_GRADS = 600_000_000         # elements of a drawn list of gradients


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one user before the Pangu-shaped layer: nothing but latency
        _norm("norm_token", "fwd", "bf16", "bf16", M=1, N=7680, residual=True, bias=True),
        # training step of a small fp32 model, odd sizes
        _norm("norm_train_f32", "train", "f32", "f32", M=777, N=1001, residual=False, bias=True),
        # training step before the mid-size layer, fp32 weights beside bf16 activations
        _norm("norm_train_mid", "train", "bf16", "f32", M=4096, N=2048, residual=True, bias=False),
        # training step before the Pangu-shaped layer, 8K tokens
        _norm("norm_train_large", "train", "bf16", "bf16", M=8192, N=7680, residual=True, bias=True),
        # the answer's next token with twenty alternatives, large vocabulary
        _logprob("logprob_token", "fwd", "f32", M=1, V=131072, top=20, entropy=True, masked=False),
        # the drafted tokens of several users, odd vocabulary, constrained answers (masked scores)
        _logprob("logprob_masked", "fwd", "bf16", M=48, V=50001, top=8, entropy=False, masked=True),
        # policy training: log probability and entropy of given answers, padded batch
        _logprob("logprob_train_mid", "train", "f32", M=4096, V=32000, top=0, entropy=True, masked=False),
        # pre-training loss over 8K tokens and a large vocabulary
        _logprob("logprob_train_large", "train", "bf16", M=8192, V=131072, top=0, entropy=False, masked=False),
        # gradients of the tiny fp32 layer (E=8, d=512, f=256): the smallest step
        _clip("clip_tiny", "clip", "f32", layer="tiny", count=3, seed=0),
        # a model's many small tensors of odd sizes and both types
        _clip("clip_many", "clip", "mixed", layer="", count=300, seed=1),
        # gradients of the mid-size layer (E=64, d=2048, f=1408, two shared experts)
        _clip("clip_mid", "clip", "bf16", layer="mid", count=5, seed=0),
        # the same, the norm alone (logged every step)
        _clip("norm_only_mid", "norm", "bf16", layer="mid", count=5, seed=0),
    ]


def _norm(name, direction, dtype, w_dtype, **sizes):
    return dict(name=name, op="norm", dir=direction, dtype=dtype, w_dtype=w_dtype, **sizes)


def _logprob(name, direction, dtype, **sizes):
    return dict(name=name, op="logprob", dir=direction, dtype=dtype, **sizes)


def _clip(name, direction, dtype, **sizes):
    return dict(name=name, op="clip", dir=direction, dtype=dtype, **sizes)


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("norm", "logprob", "clip"))
    while True:
        case = {"norm": _draw_norm, "logprob": _draw_logprob, "clip": _draw_clip}[op](rng)
        if _allowed(case):
            case.pop("name")
            return case


def _draw_norm(rng):
    dtype, w_dtype = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")))
    direction = rng.choice(("fwd", "train", "train"))
    unit = rng.choice((1, 8, 64, 64))
    N = unit * _log(rng, max(1, 64 // unit), 8192 // unit)
    return _norm("", direction, dtype, w_dtype, M=_log(rng, 1 if direction == "fwd" else 64, 16384), N=N,
                 residual=rng.random() < 0.5, bias=rng.random() < 0.7)


def _draw_logprob(rng):
    direction = rng.choice(("fwd", "train"))
    V = rng.choice((32000, 131072, _log(rng, 1000, 131072), _log(rng, 1000, 131072)))
    if direction == "train":
        return _logprob("", direction, rng.choice(("bf16", "f32")), M=_log(rng, 64, 8192), V=V, top=0,
                        entropy=rng.random() < 0.5, masked=rng.random() < 0.3)
    return _logprob("", direction, rng.choice(("bf16", "f32")), M=_log(rng, 1, 1024), V=V, top=rng.choice((0, 1, 5, 20, 32)),
                    entropy=rng.random() < 0.5, masked=rng.random() < 0.3)


def _draw_clip(rng):
    return _clip("", rng.choice(("clip", "clip", "norm")), rng.choice(("f32", "bf16", "mixed")), layer="",
                 count=_log(rng, 1, 400), seed=rng.randrange(1 << 30))


def _allowed(c):
    """A drawn case costs no more than the largest listed one of its operator."""
    if c["op"] == "norm":
        return c["M"] * c["N"] * _size(c["dtype"]) <= 8192 * 7680 * 2
    if c["op"] == "logprob":
        most = MOST_SCORES * 2 if c["dir"] == "train" else MOST_TOP_SCORES * 2
        return c["M"] * c["V"] * _size(c["dtype"]) <= most
    return sum(n for n, _ in _grad_sizes(c)) <= MOST_GRADS


def _size(dtype):
    return 2 if dtype == "bf16" else 4


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    """Inputs on the GPU, and with ``own`` the operator's handle (its buffers)."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"norm": _prepare_norm, "logprob": _prepare_logprob, "clip": _prepare_clip}[case["op"]](case, g, int(seed))
    state["case"] = case
    if own:
        from dropless_token_routing_gb300 import api
        state["handle"] = _handle(api, case, state)
    return state


def _normal(g, dtype, std, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _prepare_norm(c, g, seed):
    """Hidden states: channels of unequal size, a few of them large."""
    dt, wt, M, N = _dtype(c["dtype"]), _dtype(c["w_dtype"]), c["M"], c["N"]
    channel = torch.exp(0.5 * _normal(g, torch.float32, 1.0, N))
    channel[torch.randint(0, N, (max(1, N // 1000),), generator=g, device="cuda")] *= 20
    s = dict(x=_normal(g, dt, 1.0, M, N).mul_(channel.to(dt)),
             weight=(1 + 0.2 * _normal(g, torch.float32, 1.0, N)).to(wt),
             bias=_normal(g, wt, 0.1, N) if c["bias"] else None,
             residual=_normal(g, dt, 1.0, M, N).mul_(channel.to(dt)) if c["residual"] else None)
    if c["dir"] == "train":
        s["dy"] = _normal(g, dt, 1.0, M, N)
        s["d_sum"] = _normal(g, dt, 1.0, M, N) if c["residual"] else None
    return s


def _prepare_logprob(c, g, seed):
    """Scores of a trained head; a constrained answer's masked ones are -inf, a padded row's token is -1."""
    dt, M, V = _dtype(c["dtype"]), c["M"], c["V"]
    scores = _normal(g, dt, 2.5, M, V)
    tokens = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int64)
    if c["masked"]:
        at = scores.gather(1, tokens[:, None])
        hidden = torch.rand(M, V, generator=g, device="cuda") < 0.3
        hidden[:, V - V // 50:] = True       # the vocabulary's padding
        scores.masked_fill_(hidden, -math.inf)
        scores.scatter_(1, tokens[:, None], at)
    s = dict(scores=scores, tokens=tokens.to(torch.int32))
    if c["dir"] == "train":
        pad = torch.rand(M, generator=g, device="cuda") < 0.1
        s["tokens"][pad] = -1
        s["d_logprob"] = _normal(g, torch.float32, 1.0, M)
        s["d_entropy"] = _normal(g, torch.float32, 0.1, M).masked_fill_(pad, 0.0) if c["entropy"] else None
    return s


def _grad_sizes(c):
    """(elements, type) of every gradient."""
    if c["layer"]:
        d, E, f, S, f_s = dict(tiny=(512, 8, 256, 0, 0), mid=(2048, 64, 1408, 2, 1408))[c["layer"]]
        sizes = [(E * 2 * f * d, c["dtype"]), (E * d * f, c["dtype"]), (d * E, "f32")]
        return sizes + ([(S * 2 * f_s * d, c["dtype"]), (S * d * f_s, c["dtype"])] if S else [])
    rng = random.Random(c["seed"])
    return [(_log(rng, 1, 4_000_000), rng.choice(("f32", "bf16")) if c["dtype"] == "mixed" else c["dtype"])
            for _ in range(c["count"])]


def _prepare_clip(c, g, seed):
    """Gradients of a step, each tensor of its own size of values, and flat buffers that the optimizer
    reads them from once they are clipped, one for each type; the limit is below their norm, at times above."""
    rng = random.Random(seed)
    sizes = _grad_sizes(c)
    std = [math.exp(rng.uniform(math.log(1e-6), math.log(1e-2))) for _ in sizes]
    norm = math.sqrt(sum(s * s * n for (n, _), s in zip(sizes, std)))
    grads = [_normal(g, _dtype(t), s, n) for (n, t), s in zip(sizes, std)]
    s = dict(grads=grads, max_norm=norm * (2.0 if seed % 5 == 3 else 0.37))
    if c["dir"] == "clip":
        s["places"], length = [], {}
        for n, t in sizes:
            at = length.get(t, 0)
            s["places"].append((t, at, at + n))
            length[t] = -(-(at + n) // 64) * 64
        s["flat"] = {t: torch.zeros(n, dtype=_dtype(t), device="cuda") for t, n in length.items()}
        s["out"] = [s["flat"][t][a:b] for t, a, b in s["places"]]
    return s


def _handle(api, c, s):
    """What a program makes once and keeps."""
    if c["op"] == "norm":
        return api.LayerNorm(s["weight"], s["bias"], eps=EPS, max_rows=c["M"], dtype=_dtype(c["dtype"]))
    if c["op"] == "logprob":
        return api.TokenLogprobs(c["M"], c["V"], top=c["top"], dtype=_dtype(c["dtype"]))
    return api.GradClipper(s["grads"], out=s.get("out"))


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "logprob": _own_logprob, "clip": _own_clip}[c["op"]](c, state)
    return {"norm": _plain_norm, "logprob": _plain_logprob, "clip": _plain_clip}[c["op"]](c, state)


def _own_norm(c, s):
    ln, train = s["handle"], c["dir"] == "train"
    out = {}
    if c["residual"]:
        out["y"], out["sum"] = ln.forward(s["x"], residual=s["residual"], save=train)
    else:
        out["y"] = ln.forward(s["x"], save=train)
    if train:
        grads = ln.backward(s["dy"], d_sum=s["d_sum"])
        out.update(dx=grads["dx"], dw=grads["dw"])
        if c["bias"]:
            out["db"] = grads["db"]
    return out


def _own_logprob(c, s):
    lp, train = s["handle"], c["dir"] == "train"
    out = dict(lp.forward(s["scores"], s["tokens"], entropy=c["entropy"], save=train))
    if train:
        out["d_scores"] = lp.backward(s["d_logprob"], d_entropy=s["d_entropy"])
    return out


def _own_clip(c, s):
    if c["dir"] == "norm":
        return {"norm": s["handle"].norm()}
    return {"norm": s["handle"].clip(s["max_norm"]), "grads": s["flat"]}


def _plain_norm(c, s):
    dt, wt = _dtype(c["dtype"]), _dtype(c["w_dtype"])
    x = s["x"].float()
    if c["residual"]:
        x = x + s["residual"].float()
    centred = x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((centred * centred).mean(-1, keepdim=True) + EPS)
    xh = centred * rstd
    w = s["weight"].float()
    y = xh * w
    if c["bias"]:
        y = y + s["bias"].float()
    out = {"y": y.to(dt)}
    if c["residual"]:
        out["sum"] = x.to(dt)
    if c["dir"] == "train":
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        if c["residual"]:
            dx = dx + s["d_sum"].float()
        out.update(dx=dx.to(dt), dw=(dy * xh).sum(0).to(wt))
        if c["bias"]:
            out["db"] = dy.sum(0).to(wt)
    return out


def _alternatives(x, n):
    """The n largest of each row, equal ones by the lowest index: whole numbers that order as
    (score, -index) do. -inf is no alternative: -1."""
    V = x.shape[1]
    bits = (x + 0.0).contiguous().view(torch.int32)   # -0 is +0
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    key = order * 2 ** 32 + torch.arange(V - 1, -1, -1, device=x.device)
    top = torch.topk(key, n, dim=1, sorted=True).values
    idx = V - 1 - (top & 0xFFFFFFFF)
    return torch.where(torch.isinf(x.gather(1, idx)), torch.full_like(idx, -1), idx)


def _plain_logprob(c, s):
    x, tokens = s["scores"].float(), s["tokens"].long()
    m = x.amax(1, keepdim=True)
    logp = x - m
    log_sum = torch.log(torch.exp(logp).sum(1, keepdim=True))
    logp = logp - log_sum
    given = tokens >= 0
    at = tokens.clamp(min=0)[:, None]
    out = {"logprob": torch.where(given, logp.gather(1, at)[:, 0], torch.zeros_like(logp[:, 0]))}
    if c["top"]:
        idx = _alternatives(x, c["top"])
        out["top_idx"] = idx.to(torch.int32)
        out["top_logprob"] = torch.where(idx >= 0, logp.gather(1, idx.clamp(min=0)), torch.full_like(logp[:, :1], -math.inf))
    p = torch.exp(logp) if c["entropy"] or c["dir"] == "train" else None
    if c["entropy"]:
        plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
        out["entropy"] = -plogp.sum(1)
    if c["dir"] == "train":
        g = torch.where(given, s["d_logprob"], torch.zeros_like(s["d_logprob"]))[:, None]
        d = -g * p
        d.scatter_add_(1, at, g)
        if c["entropy"]:
            d -= s["d_entropy"][:, None] * (plogp + p * out["entropy"][:, None])
        out["d_scores"] = d.to(_dtype(c["dtype"]))
    return out


def _plain_clip(c, s):
    total = sum((t.float() ** 2).sum(dtype=torch.float64) for t in s["grads"])
    norm = torch.sqrt(total)
    if c["dir"] == "norm":
        return {"norm": norm.float()}
    scale = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0).float()
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * scale)
    return {"norm": norm.float(), "grads": s["flat"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    return {"norm": _work_norm, "logprob": _work_logprob, "clip": _work_clip}[case["op"]](case)


def _work_norm(c):
    M, N, size, w_size = c["M"], c["N"], _size(c["dtype"]), _size(c["w_dtype"])
    weights = N * (2 if c["bias"] else 1)
    rows = 4 if c["residual"] else 2           # x, residual -> sum, y
    if c["dir"] == "fwd":
        return {"bytes": rows * M * N * size + weights * w_size, "flops": 8 * M * N}
    rows += 3 if c["residual"] else 2          # dy, d_sum -> dx
    return {"bytes": rows * M * N * size + 2 * weights * w_size, "flops": 20 * M * N}


def _work_logprob(c):
    M, V, size = c["M"], c["V"], _size(c["dtype"])
    rows = M * (8 + (4 if c["entropy"] else 0) + 8 * c["top"])
    if c["dir"] == "fwd":
        return {"bytes": M * V * size + rows, "flops": 5 * M * V}
    return {"bytes": 2 * M * V * size + rows + M * (8 if c["entropy"] else 4), "flops": 10 * M * V}


def _work_clip(c):
    sizes = _grad_sizes(c)
    read = sum(n * _size(t) for n, t in sizes)
    n = sum(n for n, _ in sizes)
    return {"bytes": read + 4, "flops": 2 * n} if c["dir"] == "norm" else {"bytes": 2 * read + 4, "flops": 3 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"norm": _exact_norm, "logprob": _exact_logprob, "clip": _exact_clip}[case["op"]](case, s)


def _exact_norm(c, s):
    M, N = c["M"], c["N"]
    w = s["weight"].double()
    b = s["bias"].double() if c["bias"] else None
    out = {"y": []}
    for name in (("sum",) if c["residual"] else ()) + (("dx",) if c["dir"] == "train" else ()):
        out[name] = []
    dw = torch.zeros(N, dtype=torch.float64, device="cuda")
    db = torch.zeros_like(dw)
    for i in range(0, M, 2048):        # rows at a time
        at = slice(i, min(M, i + 2048))
        x = s["x"][at].double()
        if c["residual"]:
            x = x + s["residual"][at].double()
            out["sum"].append(x)
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        sigma = torch.sqrt(var + EPS)
        xh = (x - mean) / sigma
        out["y"].append(torch.addcmul(b, xh, w) if c["bias"] else xh * w)
        if c["dir"] == "train":
            dy = s["dy"][at].double()
            dw += torch.einsum("mn,mn->n", dy, xh)
            db += dy.sum(0)
            u = dy * w
            # the part of u that is neither constant nor along xh
            dx = (u - u.sum(1, keepdim=True) / N - xh * ((u * xh).sum(1, keepdim=True) / N)) / sigma
            out["dx"].append(dx + s["d_sum"][at].double() if c["residual"] else dx)
    out = {k: torch.cat(v) for k, v in out.items()}
    if c["dir"] == "train":
        out["dw"] = dw
        if c["bias"]:
            out["db"] = db
    return out


def _exact_logprob(c, s):
    M, V, top = c["M"], c["V"], c["top"]
    out = {"logprob": []}
    step = max(1, (1 << 27) // V)
    for i in range(0, M, step):
        at = slice(i, min(M, i + step))
        logp = torch.log_softmax(s["scores"][at].double(), 1)
        tokens = s["tokens"][at].long()
        rows = torch.arange(tokens.shape[0], device="cuda")
        lp = logp[rows, tokens.clamp(min=0)]
        lp[tokens < 0] = 0.0
        out["logprob"].append(lp)
        if top:
            values, idx = torch.sort(s["scores"][at].double(), dim=1, descending=True, stable=True)
            idx = torch.where(values[:, :top] > -math.inf, idx[:, :top], -1)
            out.setdefault("top_idx", []).append(idx.to(torch.int32))
            out.setdefault("top_logprob", []).append(logp.gather(1, idx.clamp(min=0)).masked_fill(idx < 0, -math.inf))
        if c["entropy"] or c["dir"] == "train":
            p = torch.exp(logp)
        if c["entropy"]:
            h = torch.special.entr(p).sum(1)
            out.setdefault("entropy", []).append(h)
        if c["dir"] == "train":
            g = s["d_logprob"][at].double().masked_fill(tokens < 0, 0.0)
            d = p * -g[:, None]
            d[rows, tokens.clamp(min=0)] += g
            if c["entropy"]:
                # dH/dx_j = -p_j (ln p_j + H), 0 where p_j is
                d += s["d_entropy"][at].double()[:, None] * (torch.special.entr(p) - p * h[:, None])
            out.setdefault("d_scores", []).append(d)
    return {k: torch.cat(v) for k, v in out.items()}


def _exact_clip(c, s):
    norm = math.sqrt(math.fsum(float((t.double() * t.double()).sum()) for t in s["grads"]))
    value = torch.tensor(norm, dtype=torch.float64)
    if c["dir"] == "norm":
        return {"norm": value}
    scale = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    flat = {t: torch.zeros(b.shape, dtype=torch.float64, device="cuda") for t, b in s["flat"].items()}
    for (t, a, b), grad in zip(s["places"], s["grads"]):
        flat[t][a:b] = grad.double() * scale
    return {"norm": value, "grads": flat}
