"""Cases of the few-token operators: the whole MoE layer for a few tokens (``decode``), the
linear layer with bias, activation and residual (``linear``: forward alone, or forward and
backward) and the verification of drafted tokens (``verify``).

``run`` computes a case in plain fp32 torch operations, or with the framework's kernels when
``own`` is true; ``exact`` computes it from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

WEIGHT_STD = 0.02
MASS_BITS = 40      # sampling weights are whole multiples of 2^-40
UNIFORM_BITS = 24   # of a uniform number in [0, 1)
MAX_DECODE_BYTES = 25e9    # expert weights of a drawn layer
MAX_DECODE_COPIES = 9e9    # gathered fp32 expert weights (elements) of a drawn pass
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a single token through the small fp32 layer: nothing but latency
        _decode("decode_tiny_t1", "f32", T=1, d=512, E=8, k=2, f=256, S=0, f_s=0, zipf=0.0),
        # a short draft through the mid-size layer with two shared experts
        _decode("decode_mid_t5", "bf16", T=5, d=2048, E=64, k=6, f=1408, S=2, f_s=1408, zipf=0.0),
        # one token of one user through the Pangu-shaped layer: 9 experts' weights
        _decode("decode_pangu_t1", "bf16", T=1, d=7680, E=256, k=8, f=2048, S=1, f_s=2048, zipf=0.8),
        # drafts of several users through the DeepSeek-shaped layer: most experts are read
        _decode("decode_dsv3_t32", "bf16", T=32, d=7168, E=256, k=8, f=2048, S=1, f_s=2048, zipf=1.1),
        # the projection back to the hidden size for one token
        _linear("linear_m1", "fwd", "bf16", M=1, N=7680, K=2048, act="none", residual=True),
        # a ragged batch of tokens through a wide layer with an odd width
        _linear("linear_m37", "fwd", "bf16", M=37, N=4097, K=7168, act="gelu", residual=False),
        # training step of a small fp32 layer, odd sizes
        _linear("linear_train_f32", "train", "f32", M=777, N=1001, K=512, act="gelu_tanh", residual=True),
        # training step of a mid-size dense layer
        _linear("linear_train_mid", "train", "bf16", M=4096, N=2816, K=2048, act="silu", residual=False),
        # training step of the projection back to the hidden size, 8K tokens
        _linear("linear_train_large", "train", "bf16", M=8192, N=7680, K=2048, act="none", residual=True),
        # one user's draft of four tokens
        _verify("verify_b1", "f32", B=1, n=4, V=32000, ragged=False),
        # drafts of unequal lengths, bf16 probabilities, odd vocabulary
        _verify("verify_b16", "bf16", B=16, n=5, V=50001, ragged=True),
        # a large batch of drafts over a large vocabulary
        _verify("verify_b128", "f32", B=128, n=8, V=131072, ragged=False),
    ]


def _decode(name, dtype, **sizes):
    return dict(name=name, op="decode", dtype=dtype, **sizes)


def _linear(name, direction, dtype, **sizes):
    return dict(name=name, op="linear", dir=direction, dtype=dtype, **sizes)


def _verify(name, dtype, **sizes):
    return dict(name=name, op="verify", dtype=dtype, **sizes)


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("decode", "linear", "verify"))
    while True:
        case = {"decode": _draw_decode, "linear": _draw_linear, "verify": _draw_verify}[op](rng)
        if _allowed(case):
            case.pop("name")
            return case


def _draw_decode(rng):
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    unit = 64 if dtype == "bf16" else 8
    most = (7680, 2048, 256) if dtype == "bf16" else (1024, 512, 32)
    E = _log(rng, 4, most[2])
    S = rng.choice((0, 1, 1, 2))
    f = unit * _log(rng, max(1, 128 // unit), most[1] // unit)
    return _decode("", dtype, T=_log(rng, 1, 64), d=unit * _log(rng, 256 // unit, most[0] // unit), E=E,
                   k=rng.randint(1, min(E, 8)), f=f, S=S, f_s=f if S else 0, zipf=rng.choice((0.0, 0.8, 1.1)))


def _draw_linear(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    direction = rng.choice(("fwd", "train"))
    most = 8192 if dtype == "bf16" else 1024
    M = _log(rng, 1, 512) if direction == "fwd" else _log(rng, 64, most)
    K = 8 * _log(rng, 32, 960 if dtype == "bf16" else 256)
    N = _log(rng, 256, 7680 if dtype == "bf16" else 2048)
    return _linear("", direction, dtype, M=M, N=N, K=K, act=rng.choice(ACTS), residual=rng.random() < 0.5)


def _draw_verify(rng):
    return _verify("", rng.choice(("f32", "bf16")), B=_log(rng, 1, 128), n=rng.randint(1, 8),
                   V=_log(rng, 1000, 131072), ragged=rng.random() < 0.5)


def _allowed(c):
    """A drawn case costs no more than the largest listed one of its operator."""
    if c["op"] == "decode":
        weights = 3 * c["d"] * c["f"]
        size = 2 if c["dtype"] == "bf16" else 4
        return (c["E"] + c["S"]) * weights * size <= MAX_DECODE_BYTES and c["T"] * c["k"] * weights * 2 / 3 <= MAX_DECODE_COPIES
    if c["op"] == "linear":
        return c["M"] * c["N"] * c["K"] <= (8192 * 7680 * 2048 if c["dtype"] == "bf16" else 1024 * 1024 * 1024)
    return c["B"] * (c["n"] + 1) * c["V"] <= 128 * 9 * 131072


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    """Inputs and weights on the GPU, and with ``own`` the operator's handle (its workspace)."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"decode": _prepare_decode, "linear": _prepare_linear, "verify": _prepare_verify}[case["op"]](case, g)
    state["case"] = case
    if own:
        from dropless_token_routing_gb300 import api
        state["handle"] = _handle(api, case, state)
    return state


def _normal(g, dtype, std, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _zipf_bias(E, s, seed):
    """A routing skew: bias -s ln(rank), the ranks in random order."""
    ranks = np.random.RandomState(seed).permutation(E) + 1
    return -s * np.log(ranks.astype(np.float64))


def _prepare_decode(c, g):
    dt, T, d, E, f, S, f_s = _dtype(c), c["T"], c["d"], c["E"], c["f"], c["S"], c["f_s"]
    s = dict(x=_normal(g, dt, 1.0, T, d), w_r=_normal(g, torch.float32, WEIGHT_STD, d, E),
             w13=_normal(g, dt, WEIGHT_STD, E, 2 * f, d), w2=_normal(g, dt, WEIGHT_STD, E, d, f),
             ws13=_normal(g, dt, WEIGHT_STD, S, 2 * f_s, d) if S else None,
             ws2=_normal(g, dt, WEIGHT_STD, S, d, f_s) if S else None,
             residual=_normal(g, dt, 1.0, T, d), bias=None)
    if c["zipf"]:
        s["bias"] = torch.tensor(_zipf_bias(E, c["zipf"], E), dtype=torch.float32, device="cuda")
    return s


def _prepare_linear(c, g):
    dt, M, N, K = _dtype(c), c["M"], c["N"], c["K"]
    s = dict(x=_normal(g, dt, 1.0, M, K), w=_normal(g, dt, 1.0 / math.sqrt(K), N, K), bias=_normal(g, dt, 0.1, N),
             residual=_normal(g, dt, 1.0, M, N) if c["residual"] else None)
    if c["dir"] == "train":
        s["dy"] = _normal(g, dt, 1.0, M, N)
    return s


def _prepare_verify(c, g):
    """A draft model near the target: the target's scores are the draft's with noise."""
    dt, B, n, V = _dtype(c), c["B"], c["n"], c["V"]
    q = torch.empty(B, n, V, dtype=dt, device="cuda")
    p = torch.empty(B, n + 1, V, dtype=dt, device="cuda")
    tokens = torch.empty(B, n, dtype=torch.int32, device="cuda")
    for i in range(n + 1):
        scores = _normal(g, torch.float32, 2.5, B, V)
        p[:, i] = torch.softmax(scores + _normal(g, torch.float32, 0.4, B, V), -1).to(dt)
        if i < n:
            q[:, i] = torch.softmax(scores, -1).to(dt)
            tokens[:, i] = torch.multinomial(q[:, i].float(), 1, generator=g)[:, 0].to(torch.int32)
    s = dict(draft_tokens=tokens, draft_probs=q, target_probs=p,
             u_accept=torch.rand(B, n, generator=g, device="cuda"), u_sample=torch.rand(B, generator=g, device="cuda"),
             draft_len=None)
    if c["ragged"]:
        s["draft_len"] = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _handle(api, c, s):
    """What a program makes once and keeps: the layer's weights and its workspace."""
    if c["op"] == "decode":
        params = api.LayerParams(w13=s["w13"], w2=s["w2"], w_r=s["w_r"], bias=s["bias"], ws13=s["ws13"], ws2=s["ws2"])
        return api.MoEDecodeLayer(params, c["T"], c["d"], c["E"], c["k"], c["f"], c["S"], c["f_s"], _dtype(c))
    if c["op"] == "linear":
        return api.Linear(s["w"], s["bias"], act=c["act"], max_rows=c["M"])
    return api.DraftVerifier(c["B"], c["n"], c["V"], _dtype(c))


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"decode": _own_decode, "linear": _own_linear, "verify": _own_verify}[c["op"]](c, state)
    return {"decode": _plain_decode, "linear": _plain_linear, "verify": _plain_verify}[c["op"]](c, state)


def _own_decode(c, s):
    return {"y": s["handle"].forward(s["x"], residual=s["residual"])}


def _own_linear(c, s):
    lin = s["handle"]
    if c["dir"] == "fwd":
        return {"y": lin.forward(s["x"], residual=s["residual"])}
    y = lin.forward(s["x"], residual=s["residual"], save=True)
    grads = lin.backward(s["dy"])
    return {"y": y, "dx": grads["dx"], "dw": grads["dw"], "db": grads["db"]}


def _own_verify(c, s):
    tokens, accepted = s["handle"].verify(s["draft_tokens"], s["draft_probs"], s["target_probs"], s["u_accept"],
                                          s["u_sample"], draft_len=s["draft_len"])
    return {"tokens": tokens, "accepted": accepted}


def _swiglu_rows(x, w13, w2):
    """x [..., d], w13 [..., 2f, d], w2 [..., d, f]: one row through one SwiGLU network."""
    a, b = torch.matmul(w13, x.unsqueeze(-1)).squeeze(-1).chunk(2, -1)
    h = a / (1 + torch.exp(-a)) * b
    return torch.matmul(w2, h.unsqueeze(-1)).squeeze(-1)


def _plain_decode(c, s):
    T, k, d = c["T"], c["k"], c["d"]
    x = s["x"].float()
    scores = x @ s["w_r"]
    if s["bias"] is not None:
        scores = scores + s["bias"]
    top, idx = torch.sort(scores, dim=-1, descending=True, stable=True)   # ties go to the lower index
    top, idx = top[:, :k], idx[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(-1, keepdim=True)
    flat = idx.reshape(-1)
    copies = x.unsqueeze(1).expand(T, k, d).reshape(T * k, d)
    rows = _swiglu_rows(copies, s["w13"][flat].float(), s["w2"][flat].float()).reshape(T, k, d)
    y = (w.unsqueeze(-1) * rows).sum(1)
    if c["S"]:
        a, b = torch.einsum("td,sfd->stf", x, s["ws13"].float()).chunk(2, -1)
        y = y + torch.einsum("stf,sdf->td", a / (1 + torch.exp(-a)) * b, s["ws2"].float())
    return {"y": (y + s["residual"].float()).to(_dtype(c))}


def _act(name, z):
    """The activation and its derivative in z's type."""
    one = torch.ones_like(z)
    if name == "relu":
        return torch.maximum(z, torch.zeros_like(z)), (z > 0).to(z.dtype)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return z * sg, sg * (1 + z * (1 - sg))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    return z, one


def _plain_linear(c, s):
    dt = _dtype(c)
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T + s["bias"].float()
    y, slope = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if c["dir"] == "fwd":
        return {"y": y.to(dt)}
    dz = s["dy"].float() * slope
    return {"y": y.to(dt), "dx": (dz @ w).to(dt), "dw": (dz.T @ x).to(dt), "db": dz.sum(0).to(dt)}


def _masses(r):
    """Sampling weights as whole multiples of 2^-40: NaN counts as 0, the rest is clamped to [0, 1]."""
    return (torch.nan_to_num(r, nan=0.0).clamp(0.0, 1.0) * 2.0 ** MASS_BITS).to(torch.int64)


def _plain_verify(c, s):
    B, n, V = c["B"], c["n"], c["V"]
    tokens, p, q, u = s["draft_tokens"], s["target_probs"], s["draft_probs"], s["u_accept"]
    at = tokens.long().unsqueeze(-1)
    pt = p[:, :n].gather(2, at).squeeze(-1).float()
    qt = q.gather(2, at).squeeze(-1).float()
    step = torch.arange(n, device=tokens.device)
    length = s["draft_len"].long() if s["draft_len"] is not None else torch.full_like(tokens[:, 0], n).long()
    ok = (u * qt < pt) & (step < length.unsqueeze(-1))
    accepted = torch.cumprod(ok.to(torch.int64), 1).sum(1)
    b = torch.arange(B, device=tokens.device)
    prow = p[b, accepted].float()
    qrow = q[b, accepted.clamp(max=n - 1)].float()
    refused = (accepted < length).unsqueeze(-1)
    m = _masses(torch.where(refused, prow - qrow, prow))
    m = torch.where(m.sum(1, keepdim=True) > 0, m, _masses(prow))
    cum = m.cumsum(1)
    total = cum[:, -1]
    un = (s["u_sample"] * 2.0 ** UNIFORM_BITS).to(torch.int64)
    low = 2 ** UNIFORM_BITS - 1
    level = (total >> UNIFORM_BITS) * un + (((total & low) * un) >> UNIFORM_BITS)
    drawn = (cum <= level.unsqueeze(-1)).sum(1)
    drawn = torch.where(total > 0, drawn, torch.full_like(drawn, -1)).to(torch.int32)
    cols = torch.arange(n + 1, device=tokens.device)
    padded = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], 1)
    out = torch.where(cols < accepted.unsqueeze(-1), padded, torch.full_like(padded, -1))
    out = torch.where(cols == accepted.unsqueeze(-1), drawn.unsqueeze(-1), out)
    return {"tokens": out, "accepted": accepted.to(torch.int32)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    return {"decode": _work_decode, "linear": _work_linear, "verify": _work_verify}[case["op"]](case)


def _work_decode(c):
    size = 2 if c["dtype"] == "bf16" else 4
    T, d, E, k = c["T"], c["d"], c["E"], c["k"]
    # experts that T tokens select: scores of the same distribution as the layer's
    scores = np.random.RandomState(7).standard_normal((16, T, E)) * WEIGHT_STD * math.sqrt(d)
    if c["zipf"]:
        scores = scores + _zipf_bias(E, c["zipf"], E)
    chosen = np.argsort(-scores, -1)[..., :k].reshape(16, -1)
    active = float(np.mean([len(set(r.tolist())) for r in chosen]))
    weights = 3 * d * (active * c["f"] + c["S"] * c["f_s"])
    return {"bytes": weights * size + 4 * d * E + 3 * T * d * size,
            "flops": 2 * T * d * E + 6 * T * d * (k * c["f"] + c["S"] * c["f_s"])}


def _work_linear(c):
    size = 2 if c["dtype"] == "bf16" else 4
    M, N, K = c["M"], c["N"], c["K"]
    fwd = M * K + N * K + N + (M * N if c["residual"] else 0) + M * N
    if c["dir"] == "fwd":
        return {"bytes": fwd * size, "flops": 2 * M * N * K}
    return {"bytes": (fwd + M * N + M * K + N * K + N) * size, "flops": 6 * M * N * K}


def _work_verify(c):
    size = 2 if c["dtype"] == "bf16" else 4
    B, n, V = c["B"], c["n"], c["V"]
    return {"bytes": B * (2 * V * size + n * (2 * size + 12) + 12), "flops": 3 * B * V}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"decode": _exact_decode, "linear": _exact_linear, "verify": _exact_verify}[case["op"]](case, s)


def _exact_decode(c, s):
    k, f = c["k"], c["f"]
    x = s["x"].double()
    scores = (x @ s["w_r"].double()).cpu().numpy()
    if s["bias"] is not None:
        scores = scores + s["bias"].double().cpu().numpy()
    order = np.argsort(-scores, axis=1, kind="stable")[:, :k]
    gates = np.zeros_like(scores)
    for t, chosen in enumerate(order):
        e = np.exp(scores[t, chosen] - scores[t, chosen[0]])
        gates[t, chosen] = e / e.sum()
    y = s["residual"].double()

    def network(rows, w13, w2, width):
        z = rows @ w13.double().T
        a, b = z[:, :width], z[:, width:]
        return (a * torch.sigmoid(a) * b) @ w2.double().T

    for e in np.unique(order):
        t = np.nonzero(gates[:, e])[0]
        at = torch.from_numpy(t).to(x.device)
        gate = torch.from_numpy(gates[t, e]).to(x.device)
        y[at] += gate[:, None] * network(x[at], s["w13"][int(e)], s["w2"][int(e)], f)
    for i in range(c["S"]):
        y += network(x, s["ws13"][i], s["ws2"][i], c["f_s"])
    return {"y": y}


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.addmm(s["bias"].double(), x, w.t()).requires_grad_(True)
    y = {"none": lambda v: v * 1.0, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[c["act"]](z)
    out = y.detach() if s["residual"] is None else y.detach() + s["residual"].double()
    if c["dir"] == "fwd":
        return {"y": out}
    (dz,) = torch.autograd.grad(y, z, s["dy"].double())
    return {"y": out, "dx": dz @ w, "dw": dz.t() @ x, "db": dz.sum(0)}


def _exact_verify(c, s):
    host = {key: v.float().cpu().numpy() if v is not None and v.is_floating_point() else v
            for key, v in s.items() if key not in ("case", "draft_probs", "target_probs")}
    drafted = host["draft_tokens"].cpu().numpy()
    lengths = host["draft_len"].cpu().numpy() if host["draft_len"] is not None else np.full(c["B"], c["n"])
    tokens = np.full((c["B"], c["n"] + 1), -1, np.int32)
    accepted = np.zeros(c["B"], np.int32)
    for b in range(c["B"]):
        a = 0
        while a < lengths[b]:
            v = int(drafted[b, a])
            pv, qv = (np.float32(s[name][b, a, v].item()) for name in ("target_probs", "draft_probs"))
            if not np.float32(host["u_accept"][b, a]) * qv < pv:
                break
            tokens[b, a] = v
            a += 1
        p = s["target_probs"][b, a].float().cpu().numpy()
        r = p - s["draft_probs"][b, a].float().cpu().numpy() if a < lengths[b] else p
        for row in (r, p):
            mass = (np.clip(np.nan_to_num(row, nan=0.0), 0, 1).astype(np.float64) * 2.0 ** MASS_BITS).astype(np.int64)
            total = int(mass.sum())
            if total:
                break
        if total:
            level = (int(float(host["u_sample"][b]) * 2 ** UNIFORM_BITS) * total) >> UNIFORM_BITS
            tokens[b, a] = int(np.searchsorted(np.cumsum(mass), level, side="right"))
        accepted[b] = a
    return {"tokens": tokens, "accepted": accepted}
