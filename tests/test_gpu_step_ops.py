"""The operators around the layer in training against plain 64-bit implementations: the layer norm
with its gradients, the log probabilities of given tokens with theirs, and the clipping of
gradients.

Bounds, for every element: half a step of the result's type relative to the value (one rounding),
plus fp32's half step, 2^-24, for every operation that can add its error to a value's terms: a sum goes
through at most 64 additions in a row (32 elements of a thread, then a tree, or rows in turn), so 64 and
a few more for what stands around it, times the size of the terms. Whole numbers are equal.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _api():
    from dropless_token_routing_gb300 import api
    return api


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _near(got, ref, dtype, terms, steps=96, what="", flushed=0.0):
    """|got - ref| within half a step of `dtype` and `steps` fp32 half steps of the terms' size, and
    2^-126 `flushed`."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, what
    half = torch.finfo(dtype).eps / 2
    tol = half * ref.abs() + steps * H * terms * (1 + half) + 1e-37 + 2.0 ** -126 * flushed
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / tol).nan_to_num(nan=1e30).max()))


# ------------------------------------------------------------------ layer norm
def _norm_ref(x, r, w, b, eps):
    s = x.double() + (r.double() if r is not None else 0)
    mean = s.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + eps)
    y = (s - mean) * rstd * w.double()
    return s, mean, rstd, y + b.double() if b is not None else y


def _norm_grads(s, mean, rstd, w, dy, ds):
    xh, dy = (s.double() - mean) * rstd, dy.double()
    u = dy * w.double()
    dx = rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return xh, u, dx + ds.double() if ds is not None else dx, (dy * xh).sum(0), dy.sum(0)


def _check_norm(M, N, dtype, w_dtype, residual, bias, seed=0, eps=1e-5, shift=0.0, ld=None):
    A, g = _api(), _gen(seed)
    wide = lambda t: t if ld is None or t is None else _strided(t, ld)  # noqa: E731
    x, r = _rand(g, M, N, dtype=F32).add(shift).to(dtype), _rand(g, M, N, std=2, dtype=dtype) if residual else None
    dy, ds = _rand(g, M, N, dtype=dtype), _rand(g, M, N, dtype=dtype) if residual else None
    w, b = (1 + 0.3 * _rand(g, N)).to(w_dtype), _rand(g, N, dtype=w_dtype) if bias else None
    cuda = lambda t: None if t is None else wide(t.cuda())  # noqa: E731
    ln = A.LayerNorm(w.cuda(), None if b is None else b.cuda(), eps=eps, max_rows=M, dtype=dtype)
    got = ln.forward(cuda(x), residual=cuda(r), save=True)
    y, s_got = got if residual else (got, x)
    s, mean, rstd, ref = _norm_ref(x, r, w, b, eps)
    terms = lambda v: v.abs().amax(1, keepdim=True)  # noqa: E731
    spread = terms(s) * rstd + 1          # an error of the mean, in units of y before the weight
    y_terms = spread * w.double().abs() + (b.double().abs() if b is not None else 0)
    _near(y, ref, dtype, y_terms, what="y")
    if residual:
        _near(s_got, s, dtype, s.abs(), steps=2, what="sum")
    grads = ln.backward(cuda(dy), d_sum=cuda(ds))
    # what the backward reads: x and the residual in bf16, the sum as it was rounded in fp32
    kept = s if dtype == BF else s_got.detach().cpu()
    xh, u, dx, dw, db = _norm_grads(kept, mean, rstd, w, dy, ds)
    dx_terms = rstd * terms(u) * (1 + terms(xh)) * (1 + spread) + (ds.double().abs() if ds is not None else 0)
    _near(grads["dx"], dx, dtype, dx_terms, what="dx")
    rows = 96 + M // 512
    _near(grads["dw"], dw, w_dtype, (dy.double().abs() * (xh.abs() + spread)).sum(0), steps=rows, what="dw")
    if bias:
        _near(grads["db"], db, w_dtype, dy.double().abs().sum(0), steps=rows, what="db")
    else:
        assert grads["db"] is None
    return ln


def _strided(t, ld):
    buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("dtype,w_dtype", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (3, 2), (1, 7), (5, 8), (33, 9), (200, 64), (7, 65), (64, 127), (777, 1001), (1, 1001),
                                 (300, 1024), (41, 1032), (513, 2048), (19, 2056), (100, 4096), (9, 4097), (350, 7680), (3, 8191),
                                 (77, 8192), (5, 8200), (400, 12288), (6, 16384), (330, 9000), (5, 16392), (4, 32761), (3, 32768), (1500, 512), (2000, 200)])
def test_norm_sizes(M, N, dtype, w_dtype):
    _check_norm(M, N, dtype, w_dtype, residual=(M + N) % 2 == 0, bias=M % 3 != 0, seed=M + N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,ld", [(20, 100, 104), (20, 104, 109), (20, 100, 100), (9, 1004, 1004), (7, 1001, 1016), (31, 2048, 4096), (6, 7680, 7683)])
def test_norm_strides(M, N, ld, dtype, residual):
    _check_norm(M, N, dtype, dtype, residual, True, seed=ld, ld=ld)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_rows_far_from_zero(dtype):
    """The variance is that of the centred values: a mean of 300 deviations does not cost it."""
    _check_norm(40, 1000, dtype, dtype, False, True, seed=3, shift=300.0)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,ld", [(1217, 4096, None), (611, 5120, None), (2435, 1544, 1552), (640, 5001, None), (4867, 999, None),
                                    (609, 8192, None), (9729, 200, 203)])
def test_norm_of_many_rows_two_at_a_time(M, N, ld, residual):
    """Rows enough for every group of the device, an odd one at the end."""
    _check_norm(M, N, BF, BF, residual, True, seed=M, ld=ld)


def test_norm_many_rows():
    _check_norm(9001, 520, BF, F32, True, True, seed=4)
    _check_norm(20011, 72, F32, F32, False, True, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_constant_rows_and_no_eps(dtype):
    """A constant row has variance 0: y is the bias, and finite with an eps; a row of zeros too."""
    A = _api()
    x = torch.full((3, 256), 2.0, dtype=dtype)
    x[1] = 0
    b = _rand(_gen(1), 256, dtype=dtype)
    ln = A.LayerNorm(torch.ones(256, dtype=dtype, device="cuda"), b.cuda(), eps=1e-6, max_rows=3)
    assert torch.equal(ln.forward(x.cuda()).cpu(), b.expand(3, 256))
    _check_norm(6, 100, dtype, dtype, False, False, eps=0.0)


def test_norm_rows_that_are_not_finite_stay_their_own():
    A, g = _api(), _gen(7)
    x = _rand(g, 9, 640)
    x[2, 5], x[4, 0], x[6, 639] = float("nan"), float("inf"), -float("inf")
    ln = A.LayerNorm(torch.ones(640, device="cuda"), max_rows=9)
    y = ln.forward(x.cuda(), save=True).cpu()
    dx = ln.backward(_rand(g, 9, 640).cuda(), need=("dx",))["dx"].cpu()
    for out in (y, dx):
        assert torch.equal(torch.isfinite(out).all(1), torch.tensor([i not in (2, 4, 6) for i in range(9)]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [512, 333, 8200])
def test_norm_in_place(dtype, N):
    """Results in the buffers of their operands have the same bits as elsewhere."""
    A, g, M = _api(), _gen(N), 70
    x, r, dy, ds = (_rand(g, M, N, dtype=dtype).cuda() for _ in range(4))
    w, b = _rand(g, N, dtype=dtype).cuda(), _rand(g, N, dtype=dtype).cuda()
    ln, other = A.LayerNorm(w, b, max_rows=M), A.LayerNorm(w, b, max_rows=M)
    r0 = r.clone()
    y, s = ln.forward(x, residual=r0, sum_out=r0, save=True)     # (the sum is kept, as below)
    grads = ln.backward(dy, d_sum=ds)
    x1, r1 = x.clone(), r.clone()
    y1, s1 = other.forward(x1, residual=r1, out=x1, sum_out=r1, save=True)
    assert y1 is x1 and s1 is r1 and torch.equal(y1, y) and torch.equal(s1, s)
    for place in ("dy", "d_sum", "s"):
        s1.copy_(s)
        ops = dict(dy=dy.clone(), d_sum=ds.clone(), s=s1)
        got = other.backward(ops["dy"], d_sum=ops["d_sum"], out=ops[place])
        for k in ("dx", "dw", "db"):
            assert torch.equal(got[k], grads[k]), (place, k)
    x2 = x.clone()
    assert torch.equal(other.forward(x2, out=x2), ln.forward(x))


def test_norm_needs():
    A, g = _api(), _gen(2)
    x, dy, w, b = _rand(g, 50, 96).cuda(), _rand(g, 50, 96).cuda(), _rand(g, 96).cuda(), _rand(g, 96).cuda()
    ln = A.LayerNorm(w, b, max_rows=64)
    ln.forward(x, save=True)
    full = {k: v.clone() for k, v in ln.backward(dy).items()}
    for need in (("dx",), ("dw",), ("db",), ("dw", "db"), ("dx", "db"), ()):
        got = ln.backward(dy, need=need)
        for k in ("dx", "dw", "db"):
            assert torch.equal(got[k], full[k]) if k in need else got[k] is None, (need, k)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_fewer_rows_and_none(dtype):
    A, g = _api(), _gen(3)
    N = 264
    x, dy = _rand(g, 40, N, dtype=dtype).cuda(), _rand(g, 40, N, dtype=dtype).cuda()
    ln = A.LayerNorm(torch.ones(N, dtype=dtype, device="cuda"), torch.zeros(N, dtype=dtype, device="cuda"), max_rows=40)
    whole = ln.forward(x).clone()
    for M in (40, 3, 0, 17):
        y = ln.forward(x[:M], save=True)
        assert torch.equal(y, whole[:M])
        grads = ln.backward(dy[:M])
        assert grads["dx"].shape == (M, N)
        if M == 0:
            assert not grads["dw"].any() and not grads["db"].any()
    with pytest.raises(ValueError):
        ln.forward(torch.zeros(41, N, dtype=dtype, device="cuda"))


def test_norm_rows_beyond_31_bits():
    """Rows 2^29 elements apart: offsets pass 32 bits."""
    A, M, N, ld = _api(), 6, 1000, 1 << 29
    buf = torch.empty((M - 1) * ld + N, dtype=BF, device="cuda")
    x = buf.as_strided((M, N), (ld, 1))
    x.copy_(_rand(_gen(1), M, N, dtype=BF))
    w = torch.ones(N, dtype=BF, device="cuda")
    ln = A.LayerNorm(w, max_rows=M)
    want = ln.forward(x.contiguous(), save=True).clone()
    dy = _rand(_gen(2), M, N, dtype=BF).cuda()
    grads = {k: v.clone() for k, v in ln.backward(dy).items() if v is not None}
    assert torch.equal(ln.forward(x, save=True), want)
    got = ln.backward(dy, out=x)
    assert torch.equal(got["dx"], grads["dx"]) and torch.equal(got["dw"], grads["dw"])


@pytest.mark.parametrize("M,N,ld", [(1300, 1001, 1001), (2500, 777, 779), (700, 6145, 6145), (250, 8191, 8193), (40, 6401, 6401),
                                    (900, 3001, 3001), (700, 8192, 8192), (5000, 100, 101)])
def test_norm_gradients_of_fp32_rows_and_their_residual(M, N, ld):
    """What the layer does not do, as it keeps the sum: all four operands of the backward in fp32."""
    from dropless_token_routing_gb300 import _native as native
    A, g = _api(), _gen(M + N)
    x, r, dy, ds = (_rand(g, M, N) for _ in range(4))
    w = 1 + _rand(g, N, std=0.3)
    xd, rd, dyd, dsd, dx = (_strided(t.cuda(), ld) for t in (x, r, dy, ds, torch.zeros(M, N)))
    ln = A.LayerNorm(w.cuda(), max_rows=M)
    ln.forward(xd, residual=rd, save=True)
    dims = native.NormDims(M, N, native.MOE_F32, native.MOE_F32, 1e-5, ld, ld, ld, ld, ld)
    ws = A.OpWorkspace(native.lib().moe_norm_workspace_bytes(native.ctypes.byref(dims)), "moe_norm_workspace_bytes", "cuda")
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    native.check(native.lib().moe_norm_bwd(xd.data_ptr(), rd.data_ptr(), dyd.data_ptr(), dsd.data_ptr(), ln.weight.data_ptr(),
                                           ln._bufs["stats"].data_ptr(), native.ctypes.byref(dims), dx.data_ptr(), dw.data_ptr(),
                                           db.data_ptr(), ws.ptr, ws.nbytes, torch.cuda.current_stream().cuda_stream), "moe_norm_bwd")
    s, mean, rstd, _ = _norm_ref(x, r, w, None, 1e-5)
    xh, u, want, want_dw, want_db = _norm_grads(s, mean, rstd, w, dy, ds)
    spread = s.abs().amax(1, keepdim=True) * rstd + 1
    big = lambda v: v.abs().amax(1, keepdim=True)  # noqa: E731
    # (as _check_norm: and the sum's own rounding, half a step of it)
    _near(dx, want, F32, rstd * big(u) * (1 + big(xh)) * (1 + spread) + ds.double().abs(), what="dx")
    rows = 96 + M // 512
    _near(dw, want_dw, F32, (dy.double().abs() * (xh.abs() + spread)).sum(0), steps=rows, what="dw")
    _near(db, want_db, F32, dy.double().abs().sum(0), steps=rows, what="db")
    assert ld == N or torch.isnan(dx._base[:, N:]).all()


def test_norm_gradient_by_differences():
    """The gradients along a direction are the differences of the 64-bit form along it."""
    A, g, M, N, eps = _api(), _gen(11), 13, 72, 1e-3
    x, r, w, b = _rand(g, M, N), _rand(g, M, N), 1 + _rand(g, N, std=0.3), _rand(g, N)
    dy, ds = _rand(g, M, N), _rand(g, M, N)
    ln = A.LayerNorm(w.cuda(), b.cuda(), eps=eps, max_rows=M)
    ln.forward(x.cuda(), residual=r.cuda(), save=True)
    grads = ln.backward(dy.cuda(), d_sum=ds.cuda())

    def loss(x, w, b):
        s, _, _, y = _norm_ref(x, r, w, b, eps)
        return float((y * dy.double()).sum() + (s * ds.double()).sum())

    step = 1e-5
    for name, at in (("dx", 0), ("dw", 1), ("db", 2)):
        args = [x.double(), w.double(), b.double()]
        v = torch.randn(args[at].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + step * v, args[at] - step * v
        want = (loss(*up) - loss(*down)) / (2 * step)
        got = float((grads[name].cpu().double() * v).sum())
        assert abs(got - want) <= 1e-4 * (1 + abs(want)), name


# ------------------------------------------------------------------ log probabilities
def _lp_ref(x):
    """ln p and p of rows in 64 bits; a row of -inf has ln p = -inf and p = 0."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    e = torch.where(m > -math.inf, torch.exp(x - m), torch.zeros_like(x))
    lp = torch.where(x > -math.inf, x - m - torch.log(e.sum(1, keepdim=True)), torch.full_like(x, -math.inf))
    return lp, torch.where(lp > -math.inf, torch.exp(lp), torch.zeros_like(lp))


def _top_ref(x, n):
    rows = []
    for row in x.float().tolist():
        order = sorted((j for j, v in enumerate(row) if v > -math.inf), key=lambda j: (-row[j], j))[:n]
        rows.append(order + [-1] * (n - len(order)))
    return torch.tensor(rows, dtype=torch.int32).view(x.shape[0], n)


def _check_lp(x, tokens, top, seed=0, scores=None, bwd=True):
    """x: values on the CPU; scores: where they lie on the GPU."""
    A, (M, V), dtype = _api(), x.shape, x.dtype
    scores = x.cuda() if scores is None else scores
    lp = A.TokenLogprobs(M, V, top=top, dtype=dtype)
    out = lp.forward(scores, tokens.cuda(), entropy=True, save=True)
    ref, p = _lp_ref(x)
    given = (tokens >= 0) & (tokens < V)
    at = tokens.clamp(0, V - 1).long()[:, None]
    want = torch.where(given, ref.gather(1, at)[:, 0], torch.zeros(M, dtype=torch.float64))
    size = lambda v: torch.where(v > -math.inf, v.abs(), torch.zeros_like(v))  # noqa: E731
    _equal_inf(out["logprob"], want)
    _near(out["logprob"].cpu().clamp(min=-3e38), want.clamp(min=-3e38), F32, 1 + size(want), what="logprob")
    ent = torch.where(p > 0, -p * ref, torch.zeros_like(p)).sum(1)
    log_v = 1 + math.log(V)
    # e^(x - m) is off by 2^-22 and by the rounding of its argument: (4 + 3 (ln V + ln p)) of p ln p
    _near(out["entropy"], ent, F32, torch.full_like(ent, log_v), steps=128, what="entropy")
    if top:
        idx = _top_ref(x, top)
        assert torch.equal(out["top_idx"].cpu(), idx)
        tw = ref.gather(1, idx.clamp(min=0).long()).masked_fill(idx < 0, -math.inf)
        _equal_inf(out["top_logprob"], tw)
        _near(out["top_logprob"].cpu().clamp(min=-3e38), tw.clamp(min=-3e38), F32, 1 + size(tw), what="top")
    if not bwd:
        return lp
    g = _gen(seed + 1)
    gl, gh = _rand(g, M), _rand(g, M)
    gl[M // 2:M // 2 + 1] = 0
    gh[M // 2:M // 2 + 1] = 0
    for a, b in ((gl, gh), (gl, None), (None, gh)):
        d = torch.zeros(M, V, dtype=torch.float64)
        terms = torch.zeros(M, V, dtype=torch.float64)
        # a probability below 2^-126 counts as 0, which is off by at most 2^-126 times what p is multiplied
        # by: g, and h (ln p + H) with |ln p| about 88 (h = 0.06 and ln p = -88: 5e-37, above the 1e-37 that all have)
        flushed = torch.zeros(M, V, dtype=torch.float64)
        lps = size(ref)
        if a is not None:
            one = torch.zeros(M, V, dtype=torch.float64).scatter_(1, at, 1.0) * (given & (x > -math.inf).any(1))[:, None]
            ga = (a.double() * given)[:, None]
            d += ga * (one - p)
            terms += ga.abs() * (one + p * (1 + lps))
            flushed += ga.abs()
        if b is not None:
            t = torch.where(p > 0, p * (lps.neg() + ent[:, None]), torch.zeros_like(p))
            d -= b.double()[:, None] * t
            terms += b.double().abs()[:, None] * p * (lps + log_v) * (1 + lps)
            flushed += b.double().abs()[:, None] * (lps + log_v)
        got = lp.backward(None if a is None else a.cuda(), d_entropy=None if b is None else b.cuda())
        _near(got, d, dtype, terms, steps=160, what="d_scores", flushed=flushed)
    return lp


def _equal_inf(got, want):
    assert torch.equal(torch.isinf(got.cpu()), torch.isinf(want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (2, 2, 5), (3, 5, 32), (4, 31, 3), (2, 33, 32), (5, 100, 0), (3, 1000, 20),
                                     (7, 1001, 8), (2, 4097, 32), (300, 777, 4), (3, 32000, 20), (2, 50001, 5), (1, 131072, 20),
                                     (1, 131071, 32), (5, 131072, 0), (33, 9000, 1), (200, 4096, 2), (700, 600, 10)])
def test_logprob_sizes(M, V, top, dtype):
    g = _gen(M * 31 + V)
    x = _rand(g, M, V, std=3, dtype=dtype)
    tokens = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    _check_lp(x, tokens, top, seed=V)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 1000, 20001, 32768])
def test_logprob_masks(V, dtype):
    """Rows: nothing left; one score left; masked by the type's lowest value (all, all but one, half);
    -inf in half; masked first and last; huge scores."""
    g, low = _gen(V), torch.finfo(dtype).min
    x = _rand(g, 10, V, std=3, dtype=dtype)
    x[0] = -math.inf
    x[1, :] = -math.inf
    x[1, V // 2] = 3.0
    x[2, :] = low
    x[3, :] = low
    x[3, 7] = 1.0
    x[4, ::2] = low
    x[5, torch.rand(V, generator=g) < 0.5] = -math.inf
    x[6, :V // 2] = -math.inf
    x[7, V // 2:] = -math.inf
    x[8, 3] = torch.finfo(dtype).max
    x[9] *= 1e30
    tokens = torch.tensor([1, V // 2, 5, 7, 9, 0, V - 1, 0, 3, 4], dtype=torch.int32)
    _check_lp(x, tokens, 12, seed=V)
    _check_lp(x, torch.tensor([-1, 0, V, 2 ** 31 - 1, -2 ** 31, -100, 0, 0, 1, int(x[9].argmax())], dtype=torch.int32), 32, seed=V)


def test_logprob_not_finite():
    """NaN or +inf: the row's own results are NaN, the alternatives the scores that order."""
    A, V = _api(), 5000
    x = _rand(_gen(1), 4, V)
    x[1, 17], x[2, 40] = float("nan"), float("inf")
    lp = A.TokenLogprobs(4, V, top=3)
    out = {k: v.cpu() for k, v in lp.forward(x.cuda(), torch.zeros(4, dtype=torch.int32).cuda(), entropy=True, save=True).items()}
    sick = torch.tensor([False, True, True, False])
    for k in ("logprob", "entropy"):
        assert torch.equal(torch.isnan(out[k]), sick), k
    want = _top_ref(torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x), 3)
    assert torch.equal(out["top_idx"], want) and torch.equal(torch.isnan(out["top_logprob"]).all(1), sick)
    g = torch.tensor([1.0, 1.0, 0.0, 1.0]).cuda()
    d = lp.backward(g).cpu()
    assert torch.isnan(d[1]).any() and not d[2].any() and torch.isfinite(d[[0, 3]]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,top", [(64, 32), (3000, 20), (40000, 32), (131072, 7)])
def test_logprob_alternatives_of_rows_in_order(V, top, dtype):
    """Equal scores, ascending and descending ones, a few values many times, both zeros, one block of high ones."""
    g = _gen(V + top)
    few = torch.randint(0, 4, (V,), generator=g).float()
    zeros = torch.zeros(V)
    zeros[::3] = -0.0
    block = _rand(g, V)
    block[V // 2:V // 2 + 60] += 50
    x = torch.stack([torch.zeros(V), torch.arange(V).float(), -torch.arange(V).float(), few, zeros, block,
                     torch.where(torch.arange(V) % 517 == 5, 3.0, -1.0)]).to(dtype)
    _check_lp(x, torch.full((7,), V - 1, dtype=torch.int32), top, bwd=V <= 3000)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", [(9, 131071), (40, 20001), (700, 4099), (700, 1000)])
def test_logprob_alternatives_among_equal_scores(M, V, dtype):
    """A finite mask that leaves fewer tokens than are asked for, or as many; a value that many scores share at
    the last places, alone or below some others; equal scores in the first or last part of a row only."""
    g = _gen(M + V)
    x = torch.full((M, V), -1e9, dtype=dtype)
    for m in range(M):
        kind, j = m % 9, torch.randperm(V, generator=g)
        if kind < 4:
            x[m, j[:(0, 1, 19, 20)[kind]]] = _rand(g, (0, 1, 19, 20)[kind], dtype=dtype)
        elif kind < 6:
            x[m] = _rand(g, V, dtype=dtype).clamp(max=(1.0, 0.0)[kind - 4])
            x[m, j[:11]] = torch.arange(1, 12).to(dtype)
        else:
            x[m] = -math.inf
            part = (slice(0, V // 3), slice(V - V // 3, V), slice(V // 2, V // 2 + 300))[kind - 6]
            x[m, part] = 2.0
            x[m, j[0]] = 3.0
    _check_lp(x, torch.full((M,), V - 1, dtype=torch.int32), 20, bwd=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,ld", [(1000, 1008), (1001, 1003), (32000, 32001), (640, 5000)])
def test_logprob_strides_and_in_place(V, ld, dtype):
    A, g, M = _api(), _gen(V + ld), 21
    x = _rand(g, M, V, std=2, dtype=dtype)
    tokens = torch.randint(-1, V, (M,), generator=g, dtype=torch.int32)
    lp = _check_lp(x, tokens, 4, scores=_strided(x.cuda(), ld))
    gl, gh = _rand(g, M).cuda(), _rand(g, M).cuda()
    buf = _strided(x.cuda(), ld)
    lp.forward(buf, tokens.cuda(), entropy=True, save=True)
    want = lp.backward(gl, d_entropy=gh).clone()
    got = lp.backward(gl, d_entropy=gh, out=buf)
    assert got is buf and torch.equal(buf, want)
    rest = buf.as_strided((M - 1, ld - V), (ld, 1), V)
    assert torch.isnan(rest).all()      # what lies between the rows is left as it was


def test_logprob_scores_beyond_31_bits():
    A, M, V, ld = _api(), 5, 3000, 1 << 29
    buf = torch.empty((M - 1) * ld + V, dtype=BF, device="cuda")
    x = _rand(_gen(3), M, V, std=2, dtype=BF)
    scores = buf.as_strided((M, V), (ld, 1))
    scores.copy_(x)
    tokens = torch.randint(0, V, (M,), dtype=torch.int32)
    lp = _check_lp(x, tokens, 5, scores=scores)
    gl = _rand(_gen(4), M).cuda()
    lp.forward(scores, tokens.cuda(), save=True)
    want = lp.backward(gl).clone()
    assert torch.equal(lp.backward(gl, out=scores), want)


def test_logprob_of_more_than_31_bits_of_scores():
    A, M, V = _api(), 17000, 131072
    x = torch.randn(M, V, dtype=BF, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    tokens = torch.randint(0, V, (M,), dtype=torch.int32, device="cuda")
    lp = A.TokenLogprobs(M, V, top=2, dtype=BF)
    out = lp.forward(x, tokens, save=True)
    rows = torch.tensor([0, 1, 8191, 16383, 16384, 16385, M - 1])      # both sides of 2^31 elements
    ref, p = _lp_ref(x[rows].cpu())
    at = tokens[rows].cpu().long()[:, None]
    _near(out["logprob"][rows], ref.gather(1, at)[:, 0], F32, 1 + ref.gather(1, at)[:, 0].abs())
    assert torch.equal(out["top_idx"][rows].cpu(), _top_ref(x[rows].cpu(), 2))
    g = torch.ones(M, device="cuda")
    d = lp.backward(g, out=x)[rows].cpu()
    want = torch.zeros_like(p).scatter_(1, at, 1.0) - p
    _near(d, want, BF, torch.zeros_like(p).scatter_(1, at, 1.0) + p * (1 + ref.abs()), steps=160)


def test_logprob_parts_on_their_own():
    """Alternatives without tokens; log probabilities alone; no rows."""
    A, g, V = _api(), _gen(5), 2000
    x = _rand(g, 9, V).cuda()
    tokens = torch.randint(0, V, (9,), generator=g, dtype=torch.int32).cuda()
    lp = A.TokenLogprobs(16, V, top=6)
    full = {k: v.clone() for k, v in lp.forward(x, tokens, entropy=True).items()}
    only = lp.forward(x)
    assert set(only) == {"top_idx", "top_logprob"} and all(torch.equal(only[k], full[k]) for k in only)
    some = lp.forward(x[2:5], tokens[2:5])
    assert torch.equal(some["logprob"], full["logprob"][2:5]) and "entropy" not in some
    assert lp.forward(x[:0], tokens[:0], save=True)["logprob"].shape == (0,)
    assert lp.backward(torch.zeros(0, device="cuda")).shape == (0, V)
    lp.forward(x, tokens, save=True)
    with pytest.raises(ValueError):
        lp.backward(d_entropy=torch.zeros(9, device="cuda"))


def test_logprob_gradient_by_differences():
    A, g, M, V = _api(), _gen(12), 6, 90
    x = _rand(g, M, V, std=2)
    x[:, 10:20] = -math.inf
    tokens = torch.randint(20, V, (M,), generator=g, dtype=torch.int32)
    tokens[2] = -1
    gl, gh = _rand(g, M), _rand(g, M)
    lp = A.TokenLogprobs(M, V)
    lp.forward(x.cuda(), tokens.cuda(), entropy=True, save=True)
    d = lp.backward(gl.cuda(), d_entropy=gh.cuda()).cpu().double()

    def loss(x):
        l, p = _lp_ref(x)
        ent = -torch.where(p > 0, p * l, torch.zeros_like(p)).sum(1)
        t = torch.where(tokens >= 0, l.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0], torch.zeros(M, dtype=torch.float64))
        return float((t * gl.double() + ent * gh.double()).sum())

    for _ in range(3):
        v = torch.randn(M, V, generator=g, dtype=torch.float64)
        want = (loss(x.double() + 1e-6 * v) - loss(x.double() - 1e-6 * v)) / 2e-6
        assert abs(float((d * v).sum()) - want) <= 1e-4 * (1 + abs(want))


# ------------------------------------------------------------------ clipping
def _check_clip(tensors, max_norm, out=None):
    A = _api()
    ref = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in tensors))
    scale = min(1.0, max_norm / (ref + 1e-6))
    dev = [t.cuda() for t in tensors]
    clipper = A.GradClipper(dev, out=out)
    assert abs(float(clipper.norm()) - ref) <= 40 * H * ref
    assert abs(float(clipper.clip(max_norm)) - ref) <= 40 * H * ref
    assert abs(float(clipper.scale) - scale) <= 44 * H * scale
    for t, o, d in zip(tensors, clipper.out, dev):
        _near(o, t.double() * scale, t.dtype, (t.double() * scale).abs(), steps=48)
        if out is not None:
            assert torch.equal(d.cpu(), t)
    return clipper


SIZES = [[1], [0], [], [7, 0, 9], [16384], [16385, 3, 16383], [1 << 20, 5], [100003, 77777, 1, 2, 3, 8], [3_000_001]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("types", [(BF,), (F32,), (F32, BF)])
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_clip_sizes(sizes, types, max_norm):
    g = _gen(len(sizes) + sum(sizes))
    tensors = [_rand(g, n, std=10.0 ** (i % 3), dtype=types[i % len(types)]) for i, n in enumerate(sizes)]
    _check_clip(tensors, max_norm)
    _check_clip(tensors, max_norm, out=[torch.empty_like(t, device="cuda") for t in tensors])


@pytest.mark.parametrize("count", [16, 17, 512, 513, 1300])
def test_clip_many_tensors(count):
    g = _gen(count)
    sizes = torch.randint(0, 3000, (count,), generator=g).tolist()
    tensors = [_rand(g, n, dtype=BF if i % 2 else F32) for i, n in enumerate(sizes)]
    _check_clip(tensors, 3.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_clip_views_at_any_element(dtype):
    """Slices of one flat buffer, at every offset from a 16-byte boundary; what lies between them stays."""
    A, g = _api(), _gen(6)
    flat, into = _rand(g, 400_000, dtype=dtype).cuda(), torch.full((400_000,), 7.0, dtype=dtype, device="cuda")
    at, places = 0, []
    for i in range(24):
        n = (1, 3, 17, 16384, 20001, 16391)[i % 6]
        places.append((at, at + n))
        at += n + 1 + i % 5
    grads, outs = [flat[a:b] for a, b in places], [into[a + 1:b + 1] for a, b in places]
    before = flat.clone()
    clipper = A.GradClipper(grads, out=outs)
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    clipper.clip(2.0)
    scale = 2.0 / (norm + 1e-6)
    mine = torch.zeros(400_000, dtype=torch.bool)
    for (a, b), o in zip(places, outs):
        _near(o, before[a:b].cpu().double() * scale, dtype, (before[a:b].cpu().double() * scale).abs(), steps=48)
        mine[a + 1:b + 1] = True
    assert torch.equal(flat, before) and bool((into.cpu()[~mine] == 7.0).all())
    A.GradClipper(grads).clip(2.0)       # in place
    mine = torch.zeros(400_000, dtype=torch.bool)
    for (a, b), o in zip(places, outs):
        assert torch.equal(flat[a:b], o)
        mine[a:b] = True
    assert torch.equal(flat.cpu()[~mine], before.cpu()[~mine])


def test_clip_beyond_the_range_of_squares():
    """Squares that fp32 does not hold: large, tiny, and both in one thread's share."""
    for values in ([3e25, -4e25], [3e-25, 4e-25], [1e-38, 0.0], [3e38] * 5, [2e19] * 2000, [1e-30] * 40000, [1e-42, 1e-44]):
        t = torch.tensor(values, dtype=F32)
        A = _api()
        ref = math.sqrt(math.fsum(float(v) ** 2 for v in t.double()))
        got = float(A.GradClipper([t.cuda()]).norm())
        want = float(torch.tensor(ref, dtype=torch.float64).to(F32))
        assert got == want or abs(got - ref) <= 40 * H * ref + 2.0 ** -149, values[:2]
    mixed = torch.zeros(200_000)
    mixed[5], mixed[100_000], mixed[6] = 1e-30, 1e22, 1.0
    assert abs(float(_api().GradClipper([mixed.cuda()]).norm()) - 1e22) <= 4 * H * 1e22


def test_clip_tensor_beyond_31_bits():
    """More than 2^31 elements, the last ones counted and scaled like the first."""
    n = (1 << 31) + 20001
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[:3], t[n - 20000:] = 3.0, -2.0
    ref = math.sqrt(3 * 9 + 20000 * 4)
    c = _api().GradClipper([t])
    assert abs(float(c.clip(1.0)) - ref) <= 40 * H * ref
    scale = 1.0 / (ref + 1e-6)
    _near(t[-4:], torch.full((4,), -2.0 * scale, dtype=torch.float64), BF, torch.full((4,), 2.0 * scale, dtype=torch.float64), steps=48)
    _near(t[:4], torch.tensor([3.0, 3.0, 3.0, 0.0]).double() * scale, BF, torch.full((4,), 3.0 * scale, dtype=torch.float64), steps=48)
    assert not t[3:n - 20000:99991].any()


def test_clip_not_finite():
    """The formula's scale: 0 for an infinite norm (infinities times it are NaN), NaN for NaN."""
    A = _api()
    for bad, kind in ((float("inf"), torch.isinf), (float("nan"), torch.isnan)):
        t = torch.ones(1000, device="cuda")
        t[77] = bad
        u = torch.ones(5, dtype=BF, device="cuda")
        c = A.GradClipper([t, None, u])
        assert bool(kind(c.clip(1.0)))
        if bad == float("inf"):
            assert float(c.scale) == 0 and not u.any() and bool(torch.isnan(t[77])) and not t[78:].any()
        else:
            assert bool(torch.isnan(t).all()) and bool(torch.isnan(u.float()).all())


def test_clip_limits():
    A = _api()
    t = torch.full((1000,), 2.0, device="cuda")
    c = A.GradClipper([t])
    c.clip(float("inf"))
    assert float(c.scale) == 1 and bool((t == 2).all())
    c.clip(0.0)
    assert float(c.scale) == 0 and not t.any()
    t.data = torch.full((1000,), 3.0, device="cuda")     # the tensor has moved
    assert abs(float(c.norm()) - 3 * math.sqrt(1000)) < 1e-4
    empty = A.GradClipper([])
    assert float(empty.clip(1.0)) == 0 and float(empty.scale) == 1


def test_clip_same_bits_every_time():
    A, g = _api(), _gen(9)
    ts = [_rand(g, 700_001, dtype=BF).cuda(), _rand(g, 300_007).cuda()]
    c = A.GradClipper(ts)
    first = c.norm().clone()
    for _ in range(5):
        assert torch.equal(c.norm(), first)


# ------------------------------------------------------------------ streams and graphs
def test_step_operators_in_a_graph():
    """Captured once, replayed with new values in the same buffers: the eager results' bits."""
    A, g, M, N, V = _api(), _gen(20), 65, 512, 3001
    x, r, dy = (_rand(g, M, N, dtype=BF).cuda() for _ in range(3))
    w, b = _rand(g, N, dtype=BF).cuda(), _rand(g, N, dtype=BF).cuda()
    scores, tokens, gl = _rand(g, M, V).cuda(), torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda(), _rand(g, M).cuda()

    def make():
        return A.LayerNorm(w, b, max_rows=M), A.TokenLogprobs(M, V, top=5)

    def step(ln, lp, clipper=None):
        y, s = ln.forward(x, residual=r, save=True)
        grads = ln.backward(dy, d_sum=dy)
        out = lp.forward(scores, tokens, entropy=True, save=True)
        d = lp.backward(gl, d_entropy=gl)
        outs = [y, s, grads["dx"], grads["dw"], grads["db"], *out.values(), d]
        clipper = clipper or A.GradClipper([grads["dw"], grads["db"], d])
        return outs + [clipper.clip(0.5), clipper.scale], clipper

    captured, eager = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        clipper = step(*captured)[1]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, _ = step(*captured, clipper)
    for seed in (1, 2):
        for t in (x, r, dy, scores, gl):
            t.copy_(_rand(_gen(seed), *t.shape, dtype=t.dtype))
        graph.replay()
        got = [t.clone() for t in outs]
        want, _ = step(*eager)
        for a, e in zip(got, want):
            assert torch.equal(a, e)


def test_two_calls_at_once():
    """Two sets of handles on two streams, their kernels interleaved: the results of each alone."""
    A, M, N, V = _api(), 400, 1000, 6001
    sets = []
    for i in range(2):
        g = _gen(30 + i)
        w = _rand(g, N).cuda()
        sets.append(dict(x=_rand(g, M, N).cuda(), dy=_rand(g, M, N).cuda(), scores=_rand(g, M, V).cuda(), gl=_rand(g, M).cuda(),
                         tokens=torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda(), ln=A.LayerNorm(w, max_rows=M),
                         lp=A.TokenLogprobs(M, V, top=4), stream=torch.cuda.Stream()))
    torch.cuda.synchronize()

    def step(s):
        y = s["ln"].forward(s["x"], save=True, stream=s["stream"])
        grads = s["ln"].backward(s["dy"], stream=s["stream"])
        out = s["lp"].forward(s["scores"], s["tokens"], save=True, stream=s["stream"])
        d = s["lp"].backward(s["gl"], stream=s["stream"])
        if "clip" not in s:
            s["clip"] = A.GradClipper([grads["dx"], grads["dw"], d], stream=s["stream"])
        return [y, grads["dx"], grads["dw"], *out.values(), d, s["clip"].norm(stream=s["stream"])]

    alone = []
    for s in sets:
        results = step(s)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in results])
    torch.cuda.synchronize()
    for _ in range(10):
        both = [step(s) for s in sets]
    torch.cuda.synchronize()
    for got, want in zip(both, alone):
        for a, e in zip(got, want):
            assert torch.equal(a, e)


def test_step_operators_on_another_stream():
    A, g, M, N, V = _api(), _gen(21), 300, 1024, 5000
    x, dy, scores = _rand(g, M, N).cuda(), _rand(g, M, N).cuda(), _rand(g, M, V).cuda()
    tokens, gl = torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda(), _rand(g, M).cuda()
    w = _rand(g, N).cuda()
    torch.cuda.synchronize()
    results = []
    for stream in (None, torch.cuda.Stream()):
        ln, lp = A.LayerNorm(w, max_rows=M, stream=stream), A.TokenLogprobs(M, V, top=3, stream=stream)
        y = ln.forward(x, save=True, stream=stream)
        dx = ln.backward(dy, stream=stream)["dx"]
        out = lp.forward(scores, tokens, save=True, stream=stream)
        d = lp.backward(gl, stream=stream)
        c = A.GradClipper([dx, d], stream=stream)
        norm = c.clip(1.0, stream=stream)
        torch.cuda.synchronize()
        results.append([y, dx, *out.values(), d, norm])
    for a, e in zip(*results):
        assert torch.equal(a, e)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", [(1, 40000), (3, 777), (300, 1000)])
def test_logprob_entropy_changed_before_the_backward(M, V, dtype):
    """The gradient is that of the entropy that was taken, whatever has become of the results since."""
    A, g = _api(), _gen(M + V)
    x, tokens = _rand(g, M, V, std=2, dtype=dtype).cuda(), torch.randint(-1, V, (M,), generator=g, dtype=torch.int32).cuda()
    gl, gh = _rand(g, M).cuda(), _rand(g, M).cuda()
    lp = A.TokenLogprobs(M + 5, V, top=2, dtype=dtype)
    lp.forward(x, tokens, entropy=True, save=True)
    want = lp.backward(gl, d_entropy=gh).clone()
    out = lp.forward(x, tokens, entropy=True, save=True)
    out["entropy"].neg_().add_(7.0)
    out["logprob"].zero_()
    assert torch.equal(lp.backward(gl, d_entropy=gh), want)


def test_logprob_entropy_where_the_caller_keeps_it():
    """The library's calls with two statistics for a row and the entropy beside them: the wrapper's bits."""
    from dropless_token_routing_gb300 import _native as native
    A, g, M, V = _api(), _gen(8), 37, 1200
    x, tokens = _rand(g, M, V, std=2).cuda(), torch.randint(-1, V, (M,), generator=g, dtype=torch.int32).cuda()
    gl, gh = _rand(g, M).cuda(), _rand(g, M).cuda()
    lp = A.TokenLogprobs(M, V)
    out = lp.forward(x, tokens, entropy=True, save=True)
    want = lp.backward(gl, d_entropy=gh)
    dims = native.LogprobDims(M, V, 0, native.MOE_F32, 0, 0, 0)
    ref, st = native.ctypes.byref(dims), torch.cuda.current_stream().cuda_stream
    logprob, entropy, stats, d = (torch.full(s, float("nan"), device="cuda") for s in ((M,), (M,), (2 * M + 8,), (M, V)))
    native.check(native.lib().moe_token_logprob(x.data_ptr(), tokens.data_ptr(), ref, logprob.data_ptr(), entropy.data_ptr(),
                                                stats.data_ptr(), None, None, st), "moe_token_logprob")
    native.check(native.lib().moe_token_logprob_bwd(x.data_ptr(), tokens.data_ptr(), stats.data_ptr(), entropy.data_ptr(),
                                                    gl.data_ptr(), gh.data_ptr(), ref, d.data_ptr(), st), "moe_token_logprob_bwd")
    assert torch.equal(logprob, out["logprob"]) and torch.equal(entropy, out["entropy"]) and torch.equal(d, want)
    assert torch.isnan(stats[2 * M:]).all() and not torch.isnan(stats[:2 * M]).any()


# ------------------------------------------------------------------ results in rows of their own distances
def _nan_rows(M, N, ld, dtype):
    return torch.full((M, ld), float("nan"), dtype=dtype, device="cuda")[:, :N]


def _gaps_are_left(t):
    M, N = t.shape
    rest = t._base[:, N:]
    return bool(torch.isnan(rest).all())


ODD = dict(x=3, r=8, y=5, s=1, dy=2, ds=7, dx=9)
WHOLE = dict(x=0, r=16, y=8, s=24, dy=40, ds=32, dx=48)     # on top of a multiple of 8


@pytest.mark.parametrize("dtype,w_dtype", TYPES)
@pytest.mark.parametrize("pads", [ODD, WHOLE], ids=["odd", "whole"])
@pytest.mark.parametrize("M,N", [(1, 77), (20, 100), (37, 1001), (200, 264), (2000, 333), (640, 5001), (31, 2048), (9, 8191), (700, 8192),
                                 (5, 8200), (250, 9000), (3, 12288), (4, 16392)])
def test_norm_results_in_rows_of_other_distances(M, N, pads, dtype, w_dtype):
    """Every operand and result has its own distance between rows, and so its own place within 16 bytes; what lies
    between the results' rows is left as it was. Bounds as in _check_norm; a row of M / 152 to a group of warps adds one
    rounding each to a column's sum."""
    A, g = _api(), _gen(M + N)
    dist = {k: (N + 7 & ~7 if pads is WHOLE else N) + p for k, p in pads.items()}
    x, r, dy, ds = (_rand(g, M, N, std=std, dtype=dtype) for std in (1, 2, 1, 1))
    w, b = (1 + 0.3 * _rand(g, N)).to(w_dtype), _rand(g, N, dtype=w_dtype)
    ops = {k: _strided(t.cuda(), dist[k]) for k, t in dict(x=x, r=r, dy=dy, ds=ds).items()}
    ln = A.LayerNorm(w.cuda(), b.cuda(), max_rows=M, dtype=dtype)
    big = lambda v: v.abs().amax(1, keepdim=True)  # noqa: E731
    rows = 96 + M // 152
    for residual in (True, False):
        y, sm, dx = (_nan_rows(M, N, dist[k], dtype) for k in ("y", "s", "dx"))
        if residual:
            got = ln.forward(ops["x"], residual=ops["r"], save=True, out=y, sum_out=sm)
            assert got[0] is y and got[1] is sm
        else:
            assert ln.forward(ops["x"], save=True, out=y) is y
        s, mean, rstd, ref = _norm_ref(x, r if residual else None, w, b, 1e-5)
        spread = big(s) * rstd + 1
        _near(y, ref, dtype, spread * w.double().abs() + b.double().abs(), what="y")
        if residual:
            _near(sm, s, dtype, s.abs(), steps=2, what="sum")
        grads = ln.backward(ops["dy"], d_sum=ops["ds"] if residual else None, out=dx)
        assert grads["dx"] is dx
        kept = sm.cpu() if residual and dtype == F32 else s
        xh, u, want, dw, db = _norm_grads(kept, mean, rstd, w, dy, ds if residual else None)
        _near(dx, want, dtype, rstd * big(u) * (1 + big(xh)) * (1 + spread) + (ds.double().abs() if residual else 0), what="dx")
        _near(grads["dw"], dw, w_dtype, (dy.double().abs() * (xh.abs() + spread)).sum(0), steps=rows, what="dw")
        _near(grads["db"], db, w_dtype, dy.double().abs().sum(0), steps=rows, what="db")
        assert all(map(_gaps_are_left, (y, sm, dx)))
        # the same in the operands' places (rows of the same distances there: the same kernels, the same bits)
        at = {k: _strided(t.cuda(), dist[k]) for k, t in dict(x=x, r=r, dy=dy, ds=ds).items()}
        y2, sm2 = _nan_rows(M, N, dist["x"], dtype), _nan_rows(M, N, dist["r"], dtype)
        if residual:
            ln.forward(ops["x"], residual=ops["r"], out=y2, sum_out=sm2)
            ln.forward(at["x"], residual=at["r"], out=at["x"], sum_out=at["r"])
            assert torch.equal(at["r"], sm2) and _gaps_are_left(at["r"])
        else:
            ln.forward(ops["x"], out=y2)
            ln.forward(at["x"], out=at["x"])
        assert torch.equal(at["x"], y2) and _gaps_are_left(at["x"])
        ln.forward(ops["x"], save=True)
        dx2 = _nan_rows(M, N, dist["dy"], dtype)
        d2 = ops["ds"] if residual else None
        want = {k: v.clone() for k, v in ln.backward(ops["dy"], d_sum=d2, out=dx2).items()}
        got = ln.backward(at["dy"], d_sum=d2, out=at["dy"])
        assert all(torch.equal(got[k], want[k]) for k in want) and _gaps_are_left(at["dy"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V,ld,ld_d", [(1, 1001, 1001, 1013), (5, 1000, 1008, 1003), (21, 1001, 1003, 1001), (9, 4099, 5000, 4101),
                                         (3, 50001, 50048, 50001), (300, 777, 777, 784), (4, 131072, 131072, 131075)])
def test_logprob_gradient_in_rows_of_another_distance(M, V, ld, ld_d, dtype):
    """Each gradient is a function of its score and the row's statistics: the same bits wherever it goes."""
    A, g = _api(), _gen(M + V)
    x, tokens = _rand(g, M, V, std=2, dtype=dtype).cuda(), torch.randint(-1, V, (M,), generator=g, dtype=torch.int32).cuda()
    gl, gh = _rand(g, M).cuda(), _rand(g, M).cuda()
    gl[M // 2], gh[M // 2] = 0, 0       # a row that is not read
    lp = A.TokenLogprobs(M, V, dtype=dtype)
    lp.forward(_strided(x, ld), tokens, entropy=True, save=True)
    want = lp.backward(gl, d_entropy=gh).clone()
    out = _nan_rows(M, V, ld_d, dtype)
    assert lp.backward(gl, d_entropy=gh, out=out) is out
    assert torch.equal(out, want) and (ld_d == V or _gaps_are_left(out)) and not want[M // 2].any()


@pytest.mark.parametrize("sign", [False, True])
def test_norm_weight_gradients_of_many_rows_to_a_group(sign):
    """60000 rows, 395 to a block: a column's sum takes that many roundings in a row, then one of each block and a
    few; of gradients of one sign too, whose sums only grow."""
    A, M, N = _api(), 60000, 5000
    gen = torch.Generator("cuda").manual_seed(3)
    x, dy = (torch.randn(M, N, dtype=BF, device="cuda", generator=gen) for _ in range(2))
    if sign:
        dy.abs_()
    w = torch.ones(N, device="cuda")
    ln = A.LayerNorm(w, w.clone(), max_rows=M, dtype=BF)
    ln.forward(x, save=True)
    grads = ln.backward(dy, need=("dw", "db"))
    ref = [torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(4)]
    for i in range(0, M, 4000):
        s, d = x[i:i + 4000].double(), dy[i:i + 4000].double()
        mean = s.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + 1e-5)
        xh, spread = (s - mean) * rstd, s.abs().amax(1, keepdim=True) * rstd + 1
        for t, v in zip(ref, (d * xh, d, d.abs() * (xh.abs() + spread), d.abs())):
            t += v.sum(0)
    dw, db, dw_terms, db_terms = (t.cpu() for t in ref)
    _near(grads["dw"], dw, F32, dw_terms, steps=96 + M // 152, what="dw")
    _near(grads["db"], db, F32, db_terms, steps=96 + M // 152, what="db")


def test_step_operators_look_at_their_tensors_again():
    """Another type or order at the address of before: taken as it is, or refused; nothing behind it is touched."""
    A = _api()
    buf = torch.full((1000,), 3.0, device="cuda")
    t = buf[:500]
    clip = A.GradClipper([t])
    clip.norm()
    t.data = buf.view(BF)[:500]             # 1000 of the 4000 bytes
    before = buf.clone()
    ref = math.sqrt(float((t.double() ** 2).sum()))
    assert abs(float(clip.clip(1.0)) - ref) <= 40 * H * ref
    assert torch.equal(buf[250:], before[250:])
    _near(t, before.view(BF)[:500].cpu().double() / (ref + 1e-6), BF, before.view(BF)[:500].cpu().double() / ref, steps=48)
    m, out = torch.ones(64, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    clip = A.GradClipper([m], out=[out])
    clip.clip(1.0)
    m.data = m.data.t()
    with pytest.raises(ValueError):
        clip.clip(1.0)
    w, x = torch.ones(64, device="cuda"), torch.randn(3, 64, device="cuda")
    ln = A.LayerNorm(w, max_rows=3)
    ln.forward(x)
    here = w.data
    for other in (here[:63], here.view(torch.int32), here.view(BF)[:64]):
        w.data = other
        with pytest.raises(ValueError):
            ln.forward(x)
    w.data = here
    ln.forward(x)
