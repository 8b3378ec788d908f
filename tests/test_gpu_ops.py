"""The few-token operators against plain 64-bit implementations: the whole layer for a few
tokens, the linear layer with its gradients, and the verification of drafted tokens.

Bounds (relative, 2-norm). bf16: a result is rounded once (each element off by at most 2^-9 of
itself, 2^-9 / sqrt 3 = 1.1e-3 in the mean) and one intermediate (h times its gate, z or dz) is
rounded before a product, which adds as much again; 5e-3 holds both with room for one more
rounding. fp32: sums of K products are off by at most sqrt(K) 2^-24 of their terms' norm in the
mean, 5e-6 at K = 8192; 1e-5. Whole numbers are equal.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = {torch.bfloat16: 5e-3, torch.float32: 1e-5}


def _api():
    from dropless_token_routing_gb300 import api
    return api


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _close(got, ref, dtype, what=""):
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    norm = float(ref.norm())
    err = float((got - ref).norm())
    assert err <= BOUND[dtype] * norm + 1e-30, (what, err / max(norm, 1e-30))
    # no single element is far off either: 40 times the bound of the larger of it and the rms
    rms = norm / math.sqrt(max(1, ref.numel()))
    assert float(((got - ref).abs() / ref.abs().clamp(min=rms + 1e-30)).max() if ref.numel() else 0.0) <= 40 * BOUND[dtype], what


# ------------------------------------------------------------------ the layer for a few tokens
def _layer(T, d, E, k, f, S, f_s, dtype, seed=0, bias=False):
    g = _gen(seed)
    w = dict(w_r=_rand(g, d, E, std=0.05), w13=_rand(g, E, 2 * f, d, std=d ** -0.5, dtype=dtype),
             w2=_rand(g, E, d, f, std=f ** -0.5, dtype=dtype),
             ws13=_rand(g, S, 2 * f_s, d, std=d ** -0.5, dtype=dtype) if S else None,
             ws2=_rand(g, S, d, f_s, std=max(1, f_s) ** -0.5, dtype=dtype) if S else None,
             bias=_rand(g, E) if bias else None)
    return w, _rand(g, T, d, dtype=dtype), _rand(g, T, d, dtype=dtype)


def _swiglu64(x, w13, w2):
    a, b = (w13.double() @ x).chunk(2)
    return w2.double() @ (a / (1 + torch.exp(-a)) * b)


def _decode64(w, x, residual, k, scores=None):
    """Token by token, from the definition."""
    x = x.double()
    if scores is None:
        scores = x @ w["w_r"].double()
    if w["bias"] is not None:
        scores = scores + w["bias"].double()
    y = torch.zeros_like(x) if residual is None else residual.double().clone()
    idx = torch.zeros(x.shape[0], k, dtype=torch.int32)
    gate = torch.zeros(x.shape[0], k, dtype=torch.float64)
    for t in range(x.shape[0]):
        order = sorted(range(scores.shape[1]), key=lambda e: (-float(scores[t, e]), e))[:k]
        e = torch.exp(scores[t, order] - scores[t, order[0]])
        idx[t], gate[t] = torch.tensor(order, dtype=torch.int32), e / e.sum()
        for j, q in enumerate(order):
            y[t] += gate[t, j] * _swiglu64(x[t], w["w13"][q], w["w2"][q])
        if w["ws13"] is not None:
            for s in range(w["ws13"].shape[0]):
                y[t] += _swiglu64(x[t], w["ws13"][s], w["ws2"][s])
    return y, idx, gate


def _cuda(t):
    return None if t is None else t.cuda()


def _decode_layer(w, max_tokens, d, E, k, f, S, f_s, dtype):
    A = _api()
    p = A.LayerParams(**{n: _cuda(w[n]) for n in ("w13", "w2", "w_r", "bias", "ws13", "ws2")})
    return A.MoEDecodeLayer(p, max_tokens, d, E, k, f, S, f_s, dtype)


DECODE = [  # T, d, E, k, f, S, f_s
    (1, 64, 1, 1, 64, 0, 0), (1, 512, 8, 2, 256, 0, 0), (2, 128, 4, 4, 64, 1, 128), (3, 192, 7, 3, 320, 2, 64),
    (17, 256, 16, 2, 128, 1, 64), (33, 448, 33, 5, 192, 0, 0), (64, 320, 40, 8, 64, 3, 192), (64, 64, 2, 1, 128, 0, 0),
    (5, 2048, 64, 6, 1408, 2, 1408), (16, 128, 300, 32, 64, 1, 64), (31, 64, 1024, 2, 64, 0, 0), (8, 1024, 3, 1, 2048, 1, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,E,k,f,S,f_s", DECODE)
def test_decode_layer(T, d, E, k, f, S, f_s, dtype):
    w, x, res = _layer(T, d, E, k, f, S, f_s, dtype, seed=T * 7 + E, bias=E % 2 == 0)
    layer = _decode_layer(w, T, d, E, k, f, S, f_s, dtype)
    y = layer.forward(x.cuda(), residual=res.cuda())
    ref, idx, gate = _decode64(w, x, res, k)
    assert torch.equal(layer.topk_idx.cpu(), idx)
    assert float((layer.topk_w.cpu().double() - gate).norm()) <= 1e-5 * float(gate.norm())
    _close(y, ref, dtype, "y")
    assert _api().get_device_error(layer.ws) == 0


def test_decode_fp32_narrow_unit():
    """fp32 widths are multiples of 8, not of 64."""
    T, d, E, k, f = 3, 72, 5, 2, 40
    w, x, _ = _layer(T, d, E, k, f, 1, 24, torch.float32, seed=5)
    layer = _decode_layer(w, T, d, E, k, f, 1, 24, torch.float32)
    _close(layer.forward(x.cuda()), _decode64(w, x, None, k)[0], torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_repeated_calls_with_fewer_tokens(dtype):
    """One layer serves calls of 0 to max_tokens tokens; every call's result is its own, twice
    the same bits, and nothing of an earlier call stays."""
    d, E, k, f, S, f_s = 256, 12, 3, 192, 1, 64
    w, x, res = _layer(40, d, E, k, f, S, f_s, dtype, seed=2)
    layer = _decode_layer(w, 40, d, E, k, f, S, f_s, dtype)
    ref, idx, _ = _decode64(w, x, res, k)
    xc, rc = x.cuda(), res.cuda()
    for T in (40, 1, 7, 0, 24, 40, 2):
        y1 = layer.forward(xc[:T], residual=rc[:T]).clone()
        y2 = layer.forward(xc[:T], residual=rc[:T])
        assert torch.equal(y1, y2) and y1.shape == (T, d)
        assert torch.equal(layer.topk_idx.cpu(), idx[:T])
        if T:
            _close(y1, ref[:T], dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_given_scores_ties_and_in_place(dtype):
    T, d, E, k, f = 9, 128, 10, 4, 64
    w, x, _ = _layer(T, d, E, k, f, 0, 0, dtype, seed=4)
    g = _gen(9)
    scores = torch.randint(-2, 3, (T, E), generator=g).float()   # ties everywhere
    scores[0] = 0.0
    scores[1, ::2] = -0.0
    scores[2] = torch.finfo(torch.float32).min
    scores[2, 7] = 1.0
    layer = _decode_layer(w, T, d, E, k, f, 0, 0, dtype)
    ref, idx, _ = _decode64(w, x, x, k, scores=scores.double())
    buf = x.cuda()
    y = layer.forward(buf, residual=buf, logits_in=scores.cuda(), out=buf)
    assert y is buf and torch.equal(layer.topk_idx.cpu(), idx)
    _close(buf, ref, dtype)


def test_decode_all_tokens_on_one_expert_and_none_on_others():
    T, d, E, k, f = 64, 128, 16, 1, 128
    w, x, _ = _layer(T, d, E, k, f, 0, 0, torch.bfloat16, seed=8)
    scores = torch.zeros(T, E)
    scores[:, 11] = 5.0
    layer = _decode_layer(w, T, d, E, k, f, 0, 0, torch.bfloat16)
    y = layer.forward(x.cuda(), logits_in=scores.cuda())
    _close(y, _decode64(w, x, None, k, scores=scores.double())[0], torch.bfloat16)


def test_decode_other_experts_are_not_read():
    """Weights of experts that no token selects may hold anything."""
    T, d, E, k, f = 4, 128, 8, 2, 64
    w, x, _ = _layer(T, d, E, k, f, 0, 0, torch.bfloat16, seed=1)
    scores = torch.full((T, E), -1.0)
    scores[:, 2], scores[:, 5] = 1.0, 0.5
    ref = _decode64(w, x, None, k, scores=scores.double())[0]
    for e in (0, 1, 3, 4, 6, 7):
        w["w13"][e] = float("nan")
        w["w2"][e] = float("inf")
    layer = _decode_layer(w, T, d, E, k, f, 0, 0, torch.bfloat16)
    _close(layer.forward(x.cuda(), logits_in=scores.cuda()), ref, torch.bfloat16)


def test_decode_token_with_nan_stays_alone():
    """A token whose row is not finite spoils no other token."""
    T, d, E, k, f, S, f_s = 6, 128, 8, 2, 64, 1, 64
    w, x, _ = _layer(T, d, E, k, f, S, f_s, torch.bfloat16, seed=3)
    g = _gen(1)
    scores = torch.randn(T, E, generator=g)
    ref = _decode64(w, x, None, k, scores=scores.double())[0]
    bad = x.clone()
    bad[2] = float("nan")
    bad[4, 5] = float("inf")
    layer = _decode_layer(w, T, d, E, k, f, S, f_s, torch.bfloat16)
    y = layer.forward(bad.cuda(), logits_in=scores.cuda())
    keep = [0, 1, 3, 5]
    _close(y[keep], ref[keep], torch.bfloat16)


def test_decode_on_another_stream_and_in_a_graph():
    T, d, E, k, f, S, f_s = 5, 256, 8, 2, 128, 1, 128
    w, x, res = _layer(T, d, E, k, f, S, f_s, torch.bfloat16, seed=6)
    layer = _decode_layer(w, T, d, E, k, f, S, f_s, torch.bfloat16)
    xc, rc = x.cuda(), res.cuda()
    want = layer.forward(xc, residual=rc).clone()
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer.forward(xc, residual=rc, out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(xc, residual=rc, out=out)
    for seed in (0, 1):
        fresh = _rand(_gen(seed), T, d, dtype=torch.bfloat16).cuda()
        want = layer.forward(fresh, residual=rc).clone()
        xc.copy_(fresh)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_decode_matches_the_training_layer():
    """The few-token call and moe_layer_fwd compute the same layer."""
    A = _api()
    T, d, E, k, f, S, f_s = 48, 256, 16, 4, 128, 1, 128
    w, x, _ = _layer(T, d, E, k, f, S, f_s, torch.bfloat16, seed=12)
    layer = _decode_layer(w, T, d, E, k, f, S, f_s, torch.bfloat16)
    y = layer.forward(x.cuda())
    full = A.MoELayer(layer.params, T, d, E, k, f, S, f_s, torch.bfloat16)
    _close(y, full.forward(x.cuda()).cpu(), torch.bfloat16)


# ------------------------------------------------------------------ linear
def _act64(name, z):
    F = torch.nn.functional
    return {"none": lambda v: v * 1.0, "relu": torch.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](z)


def _linear64(x, w, b, r, act, dy=None):
    x, w = x.double(), w.double()
    z = x @ w.T + (b.double() if b is not None else 0.0)
    z.requires_grad_(True)
    a = _act64(act, z)
    y = a.detach() + (r.double() if r is not None else 0.0)
    if dy is None:
        return y, None
    (dz,) = torch.autograd.grad(a, z, dy.double())
    return y, dict(dx=dz @ w, dw=dz.T @ x, db=dz.sum(0))


LINEAR = [  # M, N, K
    (1, 1, 1), (1, 128, 64), (1, 7680, 2048), (2, 129, 72), (3, 5, 7), (16, 256, 512), (17, 300, 136), (37, 1025, 1024),
    (64, 64, 8), (65, 130, 200), (100, 512, 1000), (128, 128, 128), (200, 777, 333), (257, 513, 264), (300, 96, 4096),
    (512, 1024, 512), (1000, 264, 520), (777, 1001, 512),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_forward_and_backward(M, N, K, dtype):
    A = _api()
    act = ("none", "relu", "silu", "gelu", "gelu_tanh")[(M + N + K) % 5]
    g = _gen(M + N * 3 + K * 5)
    x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K ** -0.5, dtype=dtype)
    b = _rand(g, N, std=0.3, dtype=dtype) if N % 2 else None
    r = _rand(g, M, N, dtype=dtype) if M % 2 else None
    dy = _rand(g, M, N, dtype=dtype)
    lin = A.Linear(w.cuda(), _cuda(b), act=act, max_rows=M)
    y, ref = _linear64(x, w, b, r, act, dy)
    _close(lin.forward(x.cuda(), residual=_cuda(r)), y, dtype, "y")
    _close(lin.forward(x.cuda(), residual=_cuda(r), save=True), y, dtype, "y saved")
    grads = lin.backward(dy.cuda())
    for name in ("dx", "dw", "db"):
        if name == "db" and b is None:
            assert grads["db"] is None
            continue
        _close(grads[name], ref[name], dtype, name)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_activations(act, dtype):
    """Every activation, with large and exactly zero pre-activations among them."""
    A = _api()
    M, N, K = 96, 160, 64
    g = _gen(3)
    x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=0.5, dtype=dtype)
    x[:4] = 0.0
    x[4:8] *= 8.0
    dy = _rand(g, M, N, dtype=dtype)
    lin = A.Linear(w.cuda(), None, act=act, max_rows=M)
    y, ref = _linear64(x, w, None, None, act, dy)
    _close(lin.forward(x.cuda(), save=True), y, dtype)
    grads = lin.backward(dy.cuda())
    for name in ("dx", "dw"):
        _close(grads[name], ref[name], dtype, name)


def test_linear_gradient_against_differences():
    """fp32 gradients against central differences of the 64-bit function along random directions:
    with a step h the difference is off by about h^2 of the third derivative (1e-6 at 1e-3)."""
    A = _api()
    M, N, K = 5, 7, 16
    g = _gen(21)
    x, w, b = _rand(g, M, K), _rand(g, N, K, std=0.3), _rand(g, N)
    dy = _rand(g, M, N)
    for act in ("silu", "gelu", "gelu_tanh"):
        lin = A.Linear(w.cuda(), b.cuda(), act=act, max_rows=M)
        lin.forward(x.cuda(), save=True)
        grads = lin.backward(dy.cuda())
        for name, at in (("dx", 0), ("dw", 1), ("db", 2)):
            v = _rand(g, *(x, w, b)[at].shape).double()
            h = 1e-3

            def loss(sign):
                p = [t.double() for t in (x, w, b)]
                p[at] = p[at] + sign * h * v
                return float((dy.double() * _act64(act, p[0] @ p[1].T + p[2])).sum())

            slope = (loss(1) - loss(-1)) / (2 * h)
            got = float((grads[name].cpu().double() * v).sum())
            assert abs(got - slope) <= 1e-4 * (float(grads[name].norm()) * float(v.norm())), (act, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,pad", [(3, 8), (3, 3), (130, 8), (130, 1), (300, 24)])
def test_linear_strided_rows_and_in_place_residual(M, pad, dtype):
    A = _api()
    N, K = 264, 136
    g = _gen(M + pad)

    def strided(rows, cols):
        t = torch.full((rows, cols + pad), 7.0, dtype=dtype)
        t[:, :cols] = _rand(g, rows, cols, dtype=dtype)
        return t.cuda()

    xs, ws, rs, dys = strided(M, K), strided(N, K), strided(M, N), strided(M, N)
    x, w, r, dy = xs[:, :K], ws[:, :K], rs[:, :N], dys[:, :N]
    w.mul_(K ** -0.5)
    lin = A.Linear(w, None, act="gelu", max_rows=M + 2)
    y, ref = _linear64(x.cpu(), w.cpu(), None, r.cpu(), "gelu", dy.cpu())
    got = lin.forward(x, residual=r, save=True, out=r)      # y over the residual
    assert got is r
    _close(r, y, dtype)
    assert bool((rs[:, N:] == 7.0).all())                   # nothing past the rows' ends
    grads = lin.backward(dy)
    for name in ("dx", "dw"):
        _close(grads[name], ref[name], dtype, name)


def test_linear_shapes_change_between_calls():
    A = _api()
    g = _gen(4)
    N, K = 200, 128
    w = _rand(g, N, K, std=0.1, dtype=torch.bfloat16)
    lin = A.Linear(w.cuda(), None, act="silu", max_rows=700)
    for M in (700, 1, 0, 64, 65, 3, 700):
        x = _rand(g, M, K, dtype=torch.bfloat16)
        dy = _rand(g, M, N, dtype=torch.bfloat16)
        y, ref = _linear64(x, w, None, None, "silu", dy)
        got = lin.forward(x.cuda(), save=True)
        again = lin.forward(x.cuda()).clone()
        assert got.shape == (M, N) and torch.equal(got, again)
        lin.forward(x.cuda(), save=True)
        grads = lin.backward(dy.cuda())
        if M:
            _close(got, y, torch.bfloat16)
            _close(grads["dx"], ref["dx"], torch.bfloat16)
            _close(grads["dw"], ref["dw"], torch.bfloat16)
        else:
            assert grads["dx"].shape == (0, K) and float(grads["dw"].float().abs().max()) == 0.0


def test_linear_repeats_bit_for_bit_and_on_another_stream():
    A = _api()
    g = _gen(5)
    for M, N, K in ((1, 512, 2048), (40, 1000, 512), (600, 520, 256)):
        w, x = _rand(g, N, K, std=0.1, dtype=torch.bfloat16).cuda(), _rand(g, M, K, dtype=torch.bfloat16).cuda()
        dy = _rand(g, M, N, dtype=torch.bfloat16).cuda()
        lin = A.Linear(w, None, act="gelu", max_rows=M)
        side = torch.cuda.Stream()
        runs = []
        for st in (None, side, None):
            torch.cuda.synchronize()
            y = lin.forward(x, save=True, stream=st)
            gr = lin.backward(dy, stream=st)
            torch.cuda.synchronize()
            runs.append((y.clone(), gr["dx"].clone(), gr["dw"].clone()))
        for run in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(run, runs[0]))


# ------------------------------------------------------------------ verification of drafts
def _verify64(tokens, length, q, p, u, us):
    """Sequence by sequence, in whole numbers."""
    B, n = tokens.shape
    V = p.shape[2]
    out = np.full((B, n + 1), -1, np.int32)
    acc = np.zeros(B, np.int32)

    def masses(row):
        return [int(v) for v in np.clip(np.nan_to_num(row, nan=0.0, posinf=1.0, neginf=0.0), 0, 1).astype(np.float64) * 2.0 ** 40]

    for b in range(B):
        L = n if length is None else min(max(int(length[b]), 0), n)
        a = 0
        while a < L:
            t = int(tokens[b, a])
            if not (0 <= t < V and np.float32(u[b, a]) * q[b, a, t] < p[b, a, t]):
                break
            out[b, a] = t
            a += 1
        acc[b] = a
        with np.errstate(invalid="ignore"):
            m = masses(p[b, a] - q[b, a] if a < L else p[b, a])
        if sum(m) == 0:
            m = masses(p[b, a])
        total = sum(m)
        if total:
            level = (min(max(int(np.float64(us[b]) * 2 ** 24), 0), 2 ** 24 - 1) * total) >> 24
            cum = 0
            for j, v in enumerate(m):
                cum += v
                if cum > level:
                    out[b, a] = j
                    break
    return out, acc


def _drafts(B, n, V, dtype, seed, noise=0.5):
    g = _gen(seed)
    scores = torch.randn(B, n + 1, V, generator=g) * 2
    p = torch.softmax(scores + noise * torch.randn(B, n + 1, V, generator=g), -1).to(dtype)
    q = torch.softmax(scores[:, :n], -1).to(dtype)
    tokens = torch.multinomial(q.float().reshape(B * n, V) + 1e-9, 1, generator=g).reshape(B, n).to(torch.int32) if n else torch.zeros(B, 0, dtype=torch.int32)
    return tokens, q, p, torch.rand(B, n, generator=g), torch.rand(B, generator=g)


def _check_verify(tokens, q, p, u, us, length=None):
    B, n = tokens.shape
    ver = _api().DraftVerifier(B, n, p.shape[2], p.dtype)
    got, acc = ver.verify(tokens.cuda(), q.cuda(), p.cuda(), u.cuda(), us.cuda(),
                          draft_len=_cuda(length))
    ref, racc = _verify64(tokens.numpy(), None if length is None else length.numpy(), q.float().numpy(),
                          p.float().numpy(), u.numpy(), us.numpy())
    assert np.array_equal(acc.cpu().numpy(), racc)
    assert np.array_equal(got.cpu().numpy(), ref)
    return racc


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (1, 4, 32000), (2, 3, 31), (7, 5, 1001), (40, 8, 4099), (3, 40, 200),
                                   (300, 2, 129), (1, 0, 777), (2, 1, 131072)])
def test_verify(B, n, V, dtype):
    _check_verify(*_drafts(B, n, V, dtype, seed=B + n + V))
    length = torch.randint(-1, n + 2, (B,), generator=_gen(B)).to(torch.int32)   # clamped to [0, n]
    _check_verify(*_drafts(B, n, V, dtype, seed=B + n + V + 1), length=length)


def test_verify_every_refusal_position():
    B, n, V = 9, 8, 64
    tokens, q, p, u, us = _drafts(B, n, V, torch.float32, seed=5)
    for b in range(B):      # sequence b refuses at b (or nowhere)
        for i in range(n):
            p[b, i, tokens[b, i]] = 0.0 if i == b else 1.0
    assert _check_verify(tokens, q, p, u, us).tolist() == list(range(9))


def test_verify_rows_without_weight_and_values_out_of_range():
    B, n, V = 10, 2, 515
    tokens, q, p, u, us = _drafts(B, n, V, torch.float32, seed=6)
    u[:] = 0.999
    p[0] = q[0, :1]                     # p == q at the first refusal: the draw falls back to p
    q[0, :, int(tokens[0, 0])] = 1.0
    p[0, 0] = q[0, 0]
    p[1] = 0.0                          # no weight anywhere
    p[2, :, 3] = float("nan")
    p[3, :, 4] = float("inf")
    q[4, :, 5] = float("nan")
    p[5] = torch.finfo(torch.float32).min
    tokens[6, 0], tokens[7, 1] = -1, V   # no such token: refused
    us[8], us[9] = 0.0, float(np.nextafter(np.float32(1), np.float32(0)))
    _check_verify(tokens, q, p, u, us)


def test_verify_draws_every_token_of_a_flat_row():
    """Sampling from p alone (nothing drafted): u = (j + 1/2) / V draws token j."""
    V = 256
    p = torch.full((V, 1, V), 1.0 / V)
    us = (torch.arange(V).float() + 0.5) / V
    ver = _api().DraftVerifier(V, 0, V)
    empty = torch.zeros(V, 0, dtype=torch.int32).cuda()
    got, acc = ver.verify(empty, torch.zeros(V, 0, V).cuda(), p.cuda(), torch.zeros(V, 0).cuda(), us.cuda())
    assert got[:, 0].tolist() == list(range(V)) and int(acc.sum()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_padded_rows(dtype):
    B, n, V = 5, 3, 333
    tokens, q, p, u, us = _drafts(B, n, V, dtype, seed=7)
    want = _verify64(tokens.numpy(), None, q.float().numpy(), p.float().numpy(), u.numpy(), us.numpy())
    wide_q = torch.full((B, n, V + 3), 9.0, dtype=dtype).cuda()
    wide_p = torch.full((B, n + 1, V + 8), 9.0, dtype=dtype).cuda()
    wide_q[..., :V], wide_p[..., :V] = q.cuda(), p.cuda()
    got, acc = _api().DraftVerifier(B, n, V, dtype).verify(tokens.cuda(), wide_q[..., :V], wide_p[..., :V], u.cuda(), us.cuda())
    assert np.array_equal(got.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


# ------------------------------------------------------------------ together
def test_draft_block_example():
    """The four calls of examples/draft_verify.py in a row, against the same steps in 64 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_verify.py")
    spec = importlib.util.spec_from_file_location("draft_verify", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.DraftBlock(users=6, drafted=4)
    attended, x, tokens, probs, u, us = ex.inputs(block)
    got, acc = block.step(attended, x, tokens, probs, u, us)
    # the block's probabilities again, and the verification of them in whole numbers
    h = block.project.forward(attended, residual=x).clone()
    _close(h, _linear64(attended.cpu(), block.project.w.cpu(), None, x.cpu(), "none")[0], torch.bfloat16)
    y = block.layer.forward(h, residual=h).clone()
    p = block.layer.params
    w = dict(w_r=p.w_r.cpu(), w13=p.w13.cpu(), w2=p.w2.cpu(), ws13=p.ws13.cpu(), ws2=p.ws2.cpu(), bias=None)
    _close(y, _decode64(w, h.cpu(), h.cpu(), 2)[0], torch.bfloat16)
    target = torch.softmax(block.head.forward(y).float(), -1).view(6, 5, -1)
    ref, racc = _verify64(tokens.cpu().numpy(), None, probs.cpu().numpy(), target.cpu().numpy(), u.cpu().numpy(),
                          us.cpu().numpy())
    assert np.array_equal(got.cpu().numpy(), ref) and np.array_equal(acc.cpu().numpy(), racc)


# ------------------------------------------------------------------ large and odd memory
def test_linear_output_past_32_bit_offsets():
    """y holds more than 2^31 elements; the last rows and some between are compared."""
    A = _api()
    M, N, K = 70001, 32768, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16) * 0.1
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    y = A.Linear(w, None, max_rows=M).forward(x)
    rows = torch.tensor([0, 1, 255, 256, 32767, 65535, 65536, 65599, 69999, 70000], device="cuda")
    _close(y[rows], x[rows].cpu().double() @ w.cpu().double().T, torch.bfloat16)


def test_verify_probabilities_past_32_bit_offsets():
    """Row n of the target starts past element 2^31."""
    n, V, ld = 1024, 1000, 1 << 21
    p = torch.zeros(1, n + 1, ld, dtype=torch.bfloat16, device="cuda")[..., :V]
    q = torch.zeros(1, n, V, dtype=torch.bfloat16, device="cuda")
    tokens = torch.randint(0, V, (1, n), generator=_gen(2)).to(torch.int32)
    at = tokens.long().cuda().unsqueeze(-1)
    p[:, :n].scatter_(2, at, 1.0)            # every drafted token is kept
    q.scatter_(2, at, 1.0)
    p[0, n, 777] = 1.0                       # and the one after them is certain
    u, us = torch.full((1, n), 0.5), torch.tensor([0.25])
    got, acc = _api().DraftVerifier(1, n, V, torch.bfloat16).verify(tokens.cuda(), q, p, u.cuda(), us.cuda())
    assert int(acc) == n and got[0, :n].tolist() == tokens[0].tolist() and int(got[0, n]) == 777


@pytest.mark.parametrize("M", [5, 40, 100, 300])
@pytest.mark.parametrize("N", [264, 301])
def test_linear_rows_with_nan_and_inf_stay_alone(M, N):
    """A row of x that is not finite spoils no other row of y, and no other row of dx."""
    A = _api()
    K = 136
    g = _gen(M + N)
    w, x = _rand(g, N, K, std=0.1, dtype=torch.bfloat16), _rand(g, M, K, dtype=torch.bfloat16)
    r, dy = _rand(g, M, N, dtype=torch.bfloat16), _rand(g, M, N, dtype=torch.bfloat16)
    y, ref = _linear64(x, w, None, r, "silu", dy)
    bad, bad_dy = x.clone(), dy.clone()
    bad[1] = float("nan")
    bad[M - 1, 7] = float("inf")
    bad_dy[1] = float("nan")
    lin = A.Linear(w.cuda(), None, act="silu", max_rows=M)
    keep = [i for i in range(M) if i not in (1, M - 1)]
    _close(lin.forward(bad.cuda(), residual=r.cuda(), save=True)[keep], y[keep], torch.bfloat16)
    _close(lin.backward(bad_dy.cuda(), need=("dx",))["dx"][keep], ref["dx"][keep], torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_long_contractions_divided(dtype):
    """Few outputs and a long K: the sums of many partial ones."""
    A = _api()
    for M, N, K in ((300, 64, 8192), (260, 130, 5000), (20, 40, 9000)):
        g = _gen(K)
        x, w = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K ** -0.5, dtype=dtype)
        dy = _rand(g, M, N, dtype=dtype)
        lin = A.Linear(w.cuda(), None, max_rows=M)
        y, ref = _linear64(x, w, None, None, "none", dy)
        _close(lin.forward(x.cuda(), save=True), y, dtype)
        grads = lin.backward(dy.cuda())
        _close(grads["dx"], ref["dx"], dtype)
        _close(grads["dw"], ref["dw"], dtype)


def test_workspaces_report_no_error_after_use():
    A = _api()
    g = _gen(0)
    lin = A.Linear(_rand(g, 500, 256, std=0.1, dtype=torch.bfloat16).cuda(), None, act="gelu", max_rows=400)
    x = _rand(g, 400, 256, dtype=torch.bfloat16).cuda()
    lin.forward(x, save=True)
    lin.backward(lin.forward(x, save=True).clone())
    assert A.get_device_error(lin.ws) == 0


def test_wrappers_refuse_what_does_not_fit():
    A = _api()
    w = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    lin = A.Linear(w, None, max_rows=4)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :32], torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            lin.forward(bad)
    with pytest.raises(ValueError):
        lin.backward(torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"))   # nothing saved
    with pytest.raises(ValueError):
        lin.forward(x, residual=x)
    with pytest.raises(KeyError):
        A.Linear(w, None, act="tanh")
    wl, xl, _ = _layer(4, 128, 8, 2, 64, 0, 0, torch.bfloat16)
    layer = _decode_layer(wl, 4, 128, 8, 2, 64, 0, 0, torch.bfloat16)
    for bad in (xl.float().cuda(), torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda"), xl[:, :64].cuda()):
        with pytest.raises(ValueError):
            layer.forward(bad)
    with pytest.raises(A.N.MoeError):
        _decode_layer(wl, 65, 128, 8, 2, 64, 0, 0, torch.bfloat16)
    ver = A.DraftVerifier(2, 3, 16)
    good = dict(draft_tokens=torch.zeros(2, 3, dtype=torch.int32).cuda(), draft_probs=torch.zeros(2, 3, 16).cuda(),
                target_probs=torch.zeros(2, 4, 16).cuda(), u_accept=torch.zeros(2, 3).cuda(), u_sample=torch.zeros(2).cuda())
    ver.verify(**good)
    for name, bad in (("draft_tokens", torch.zeros(2, 3).cuda()), ("target_probs", torch.zeros(2, 3, 16).cuda()),
                      ("draft_probs", torch.zeros(2, 3, 16).bfloat16().cuda()), ("u_sample", torch.zeros(3).cuda()),
                      ("draft_probs", torch.zeros(2, 16, 3).cuda().transpose(1, 2))):
        with pytest.raises(ValueError):
            ver.verify(**{**good, name: bad})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_made_for_many_rows_used_with_few(dtype):
    A = _api()
    N, K = 1500, 333
    g = _gen(9)
    w = _rand(g, N, K, std=K ** -0.5, dtype=dtype)
    lin = A.Linear(w.cuda(), None, act="relu", max_rows=6000)
    for M in (100, 1, 6000, 700):
        x, dy = _rand(g, M, K, dtype=dtype), _rand(g, M, N, dtype=dtype)
        y, ref = _linear64(x, w, None, None, "relu", dy)
        _close(lin.forward(x.cuda(), save=True), y, dtype)
        grads = lin.backward(dy.cuda())
        _close(grads["dw"], ref["dw"], dtype)
        _close(grads["dx"], ref["dx"], dtype)


# ------------------------------------------------------------------ weights that are replaced
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layers_use_replaced_weights(dtype):
    """A weight that is replaced between two calls (the tensor, or its storage) is the one used."""
    A = _api()
    T, d, E, k, f, S, f_s = 6, 128, 8, 2, 64, 1, 64
    w, x, _ = _layer(T, d, E, k, f, S, f_s, dtype, seed=31, bias=True)
    other, _, _ = _layer(T, d, E, k, f, S, f_s, dtype, seed=32, bias=True)
    layer = _decode_layer(w, T, d, E, k, f, S, f_s, dtype)
    xc = x.cuda()
    _close(layer.forward(xc), _decode64(w, x, None, k)[0], dtype)
    for i, name in enumerate(("w2", "w13", "ws13", "ws2", "w_r", "bias")):
        w[name] = other[name]
        if i % 2:
            getattr(layer.params, name).data = other[name].cuda()
        else:
            setattr(layer.params, name, other[name].cuda())
        y = layer.forward(xc)
        ref, idx, _ = _decode64(w, x, None, k)
        assert torch.equal(layer.topk_idx.cpu(), idx), name
        _close(y, ref, dtype, name)
    M, n = 40, 72
    g = _gen(33)
    lin = A.Linear(_rand(g, n, d, std=0.1, dtype=dtype).cuda(), _rand(g, n, dtype=dtype).cuda(), act="silu", max_rows=M)
    xl, dy = _rand(g, M, d, dtype=dtype), _rand(g, M, n, dtype=dtype)
    lin.forward(xl.cuda(), save=True)
    for pad in (0, 3, 8):
        w2, b2 = _rand(g, n, d, std=0.1, dtype=dtype), _rand(g, n, dtype=dtype)
        wide = torch.full((n, d + pad), 5.0, dtype=dtype)
        wide[:, :d] = w2
        if pad == 3:
            lin.w.data, lin.bias.data = wide.cuda()[:, :d], b2.cuda()
        else:
            lin.w, lin.bias = wide.cuda()[:, :d], b2.cuda()
        y, ref = _linear64(xl, w2, b2, None, "silu", dy)
        _close(lin.forward(xl.cuda(), save=True), y, dtype, pad)
        grads = lin.backward(dy.cuda())
        for name in ("dx", "dw", "db"):
            _close(grads[name], ref[name], dtype, (name, pad))
    assert A.get_device_error(lin.ws) == 0 and A.get_device_error(layer.ws) == 0


@pytest.mark.parametrize("M", [3, 200])
def test_linear_applied_to_its_own_result(M):
    """A square layer: its own y (dx) is refused as x (dy); through another buffer it is right."""
    A = _api()
    n = 128
    g = _gen(41)
    w, x = _rand(g, n, n, std=n ** -0.5), _rand(g, M, n)
    lin = A.Linear(w.cuda(), None, max_rows=M)
    y = lin.forward(x.cuda())
    with pytest.raises(ValueError):
        lin.forward(y)
    twice = lin.forward(y, out=torch.empty(M, n, device="cuda"), save=True)
    _close(twice, x.double() @ w.double().T @ w.double().T, torch.float32)
    dx = lin.backward(x.cuda())["dx"]
    with pytest.raises(ValueError):
        lin.backward(dx)
    _close(lin.backward(dx.clone())["dx"], x.double() @ w.double() @ w.double(), torch.float32)
    # in and out side by side in the rows of one buffer
    wide = torch.zeros(M, 3 * n, device="cuda")
    wide[:, :n] = x.cuda()
    lin.forward(wide[:, :n], out=wide[:, n:2 * n])
    lin.forward(wide[:, n:2 * n], residual=wide[:, :n], out=wide[:, :n])
    h = x.double() @ w.double().T
    _close(wide[:, n:2 * n], h, torch.float32)
    _close(wide[:, :n], h @ w.double().T + x.double(), torch.float32)
    assert float(wide[:, 2 * n:].abs().max()) == 0.0


# ------------------------------------------------------------------ a wait that runs out
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,E,k,f", [(5, 1024, 16, 6, 512), (40, 192, 9, 2, 64)])
def test_decode_wait_that_runs_out(T, d, E, k, f, dtype):
    """The hidden rows of a CTA that does not exist are waited for: after the limit of one second the
    launch winds down at once (no stage of the weight ring is waited for any longer), the status
    says so, and the next call on the workspace is right."""
    import ctypes
    import time
    A = _api()
    w, x, _ = _layer(T, d, E, k, f, 0, 0, dtype, seed=51)
    layer = _decode_layer(w, T, d, E, k, f, 0, 0, dtype)
    ref = _decode64(w, x, None, k)[0]
    xc, y = x.cuda(), torch.zeros(T, d, dtype=dtype, device="cuda")
    _close(layer.forward(xc), ref, dtype)
    c, dims = layer.params.c(), A.make_dims(T, d, E, k, f, dtype=dtype)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    st = A.N.lib().moe_debug_decode_timeout_probe(ctypes.byref(c), xc.data_ptr(), ctypes.byref(dims), y.data_ptr(),
                                                  layer.ws.ptr, layer.ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert A.get_device_error(layer.ws) == A.N.STATUS_CODE["MOE_ERR_DEVICE_TIMEOUT"]
    took = time.perf_counter() - t0
    # the wait itself, and once more for a CTA that waits for one that gave up
    assert 0.9 < took < 3.0, took
    _close(layer.forward(xc), ref, dtype)
    assert A.get_device_error(layer.ws) == 0


# ------------------------------------------------------------------ activations far out
def _act_slope64(name, z):
    """Value and derivative in 64 bits, by formulas that keep their relative accuracy in the tails."""
    z = z.double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s, r = torch.sigmoid(2 * u), torch.sigmoid(-2 * u)
    return z * s, s + z * s * r * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _through_layer(act, z, dtype=torch.float32):
    """act(z) and act'(z) of every z by a layer of one input and one output: y = act(z * 1), dx = dy act'(z)."""
    A = _api()
    M = z.numel()
    lin = A.Linear(torch.ones(1, 1, dtype=dtype, device="cuda"), None, act=act, max_rows=M)
    x = z.to(dtype).reshape(M, 1).cuda()
    y = lin.forward(x, save=True).clone()
    dx = lin.backward(torch.ones(M, 1, dtype=dtype, device="cuda"), need=("dx",))["dx"]
    return y.cpu().double().reshape(-1), dx.cpu().double().reshape(-1)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_fp32_gelu_keeps_its_accuracy_in_the_tail(act):
    """Element by element. For z in [-6, -3] the function is e^(-t) times a factor of order 1 with t
    up to 25; t is made by at most five fp32 operations, each off by 2^-24 of it, and the rest by ten
    more: 25 * 5 * 6e-8 + 1e-6 = 8.5e-6; 2e-5 is twice that. The derivative is a sum of two
    such terms, of which the larger is at most 1.15 times the result there: 4e-5."""
    z = torch.linspace(-6, -3, 3001).float()
    y, slope = _through_layer(act, z)
    ry, rs = _act_slope64(act, z)
    assert float(((y - ry) / ry).abs().max()) <= 2e-5
    assert float(((slope - rs) / rs).abs().max()) <= 4e-5
    # and around 0 and above, where nothing is small: 2^-24 of ten operations on values up to 6
    z = torch.linspace(-3, 6, 3001).float()
    y, slope = _through_layer(act, z)
    ry, rs = _act_slope64(act, z)
    assert float((y - ry).abs().max()) <= 6e-6
    assert float((slope - rs).abs().max()) <= 6e-6


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_huge_finite_values(act, dtype):
    """Finite z, however large, have the function's limits: z and 0, slopes 1 and 0."""
    z = torch.tensor([1e4, 1e10, 1e13, 1e18, 1e20, 1e25, 1e30, 3e38])
    y, slope = _through_layer(act, torch.cat([z, -z]), dtype)
    zd = z.to(dtype).double()
    assert torch.equal(y[:8], zd) and float(y[8:].abs().max()) == 0.0
    assert torch.equal(slope[:8], torch.ones(8).double()) and float(slope[8:].abs().max()) == 0.0


def test_linear_repeats_with_and_without_save_at_changing_rows():
    """The result of every call, kept before the next one writes the layer's buffer: equal bits with
    and without the pre-activation stored, and again after calls of other sizes."""
    A = _api()
    g = _gen(61)
    N, K = 200, 128
    w = _rand(g, N, K, std=0.1, dtype=torch.bfloat16)
    lin = A.Linear(w.cuda(), None, act="silu", max_rows=700)
    first = {}
    for M in (700, 1, 64, 65, 3, 700, 65, 1, 64):
        x = _rand(_gen(M), M, K, dtype=torch.bfloat16)
        saved = lin.forward(x.cuda(), save=True).clone()
        assert torch.equal(lin.forward(x.cuda()), saved)
        lin.forward(-x.cuda())          # something else in the buffer
        assert torch.equal(lin.forward(x.cuda()), saved)
        _close(saved, _linear64(x, w, None, None, "silu")[0], torch.bfloat16, M)
        assert torch.equal(saved, first.setdefault(M, saved))


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 67), (3, 72), (130, 65)])
def test_linear_rows_far_apart(M, K, dtype, act):
    """The last positions of sequences: rows of x a sequence apart, dx in rows of its own."""
    A = _api()
    N, far = 136, 5003
    g = _gen(M + K)
    x, w, b = _rand(g, M, K, dtype=dtype), _rand(g, N, K, std=K ** -0.5, dtype=dtype), _rand(g, N, dtype=dtype)
    dy = _rand(g, M, N, dtype=dtype)
    wide = torch.full((M, far), 3.0, dtype=dtype)
    wide[:, 16:16 + K] = x
    rows = wide.cuda()[:, 16:16 + K]
    lin = A.Linear(w.cuda(), b.cuda(), act=act, max_rows=M + 1)
    y, ref = _linear64(x, w, b, None, act, dy)
    _close(lin.forward(rows, save=True), y, dtype)
    grads = lin.backward(dy.cuda())
    for name in ("dx", "dw", "db"):
        _close(grads[name], ref[name], dtype, name)


def test_rows_a_long_sequence_apart():
    """Rows 2^28 elements and more apart (x) and 2^24 and more (probabilities of the last position)."""
    A = _api()
    M, N, K, far = 2, 40, 72, (1 << 28) + 64
    g = _gen(71)
    w = _rand(g, N, K, std=0.1, dtype=torch.bfloat16)
    x, dy = _rand(g, M, K, dtype=torch.bfloat16), _rand(g, M, N, dtype=torch.bfloat16)
    wide = torch.zeros(M, far, dtype=torch.bfloat16, device="cuda")
    rows = wide[:, far - 80:far - 8]
    rows.copy_(x)
    lin = A.Linear(w.cuda(), None, max_rows=M)
    y, ref = _linear64(x, w, None, None, "none", dy)
    _close(lin.forward(rows, save=True), y, torch.bfloat16)
    grads = lin.backward(dy.cuda())
    _close(grads["dx"], ref["dx"], torch.bfloat16)
    _close(grads["dw"], ref["dw"], torch.bfloat16)
    B, S, V = 2, 40, 500000
    p = torch.zeros(B, S, V, device="cuda")
    p[0, -1, 123456] = 0.5
    p[1, -1, 499999] = 0.25
    got, acc = A.DraftVerifier(B, 0, V).verify(torch.zeros(B, 0, dtype=torch.int32).cuda(), torch.zeros(B, 0, V).cuda(),
                                               p[:, -1:], torch.zeros(B, 0).cuda(), torch.tensor([0.1, 0.9]).cuda())
    assert got[:, 0].tolist() == [123456, 499999] and acc.tolist() == [0, 0]


def test_linear_buffers_belong_to_the_call_s_stream():
    """The layer's buffers are made in a call: memory that the current stream still reads (freed, but
    with work pending) must not become the output of a call on another stream."""
    A = _api()
    M, N, K = 256, 4096, 64
    g = _gen(81)
    w, x = _rand(g, N, K, std=0.1, dtype=torch.bfloat16).cuda(), _rand(g, M, K, dtype=torch.bfloat16).cuda()
    dy = _rand(g, M, N, dtype=torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    lin = A.Linear(w, torch.zeros(N, dtype=torch.bfloat16, device="cuda"), act="silu", max_rows=M)
    torch.cuda.synchronize()
    shapes = ((M, N), (M, N), (M, K), (N, K), (1, N))      # y, z, dx, dw, db
    freed = [torch.full(s, 1.0, dtype=torch.bfloat16, device="cuda") for s in shapes]
    copies = [torch.empty_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)      # tens of milliseconds on the current stream
    for c, t in zip(copies, freed):
        c.copy_(t)
    del freed, t
    lin.forward(x, save=True, stream=side)
    grads = lin.backward(dy, stream=side)
    torch.cuda.synchronize()
    for c in copies:
        assert bool((c == 1.0).all())
    _close(grads["dw"], _linear64(x.cpu(), w.cpu(), None, None, "silu", dy.cpu())[1]["dw"], torch.bfloat16)
