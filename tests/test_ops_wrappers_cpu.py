"""What the wrappers of the few-token operators hand to the library, and what they refuse (CPU
only: the library's calls are recorded, not made; only its size calls run)."""
import os

import pytest
import torch

from dropless_token_routing_gb300 import builder as B

if not os.path.exists(B.LIB):
    B.build()

from dropless_token_routing_gb300 import _native as N  # noqa: E402
from dropless_token_routing_gb300 import api as A  # noqa: E402


class Stream:
    cuda_stream = 0


ST = Stream()
DEV = "cpu:0"   # the layers' device in these tests


class Recorder:
    """Stands in for the library: size calls go to it, all others are recorded and succeed."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return getattr(self.lib, name)

        def call(*args):
            # structures change between calls: their values now
            values = [getattr(a, "_obj", a) for a in args]
            values = [{f: getattr(v, f) for f, _ in v._fields_} if hasattr(v, "_fields_") else v for v in values]
            self.calls.append((name, values))
            return 0

        return call

    def last(self, name):
        got = [values for n, values in self.calls if n == name]
        return got[-1]


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder(N.lib())
    monkeypatch.setattr(N, "lib", lambda: rec)
    return rec


def linear(N_=32, K=64, rows=8, dtype=torch.float32, **kw):
    return A.Linear(torch.zeros(N_, K, dtype=dtype), None, max_rows=rows, device=DEV, stream=ST, **kw)


# ------------------------------------------------------------------ rows that lie on one another
def test_linear_refuses_rows_closer_than_their_width(lib):
    """A broadcast row (stride 0) is no matrix of M rows: the library would take stride 0 for
    the default and read M - 1 rows past its end."""
    M, n, k = 4, 32, 64
    lin = linear()
    x, r, dy = torch.zeros(M, k), torch.zeros(M, n), torch.zeros(M, n)
    row = torch.zeros(n).expand(M, n)
    near = torch.zeros(M * n).as_strided((M, n), (n - 1, 1))   # rows overlap by one element
    lin.forward(x, residual=r, save=True, stream=ST)
    for bad in (row, near):
        with pytest.raises(ValueError):
            lin.forward(x, residual=bad, stream=ST)
        with pytest.raises(ValueError):
            lin.forward(x, out=bad, stream=ST)
    with pytest.raises(ValueError):
        lin.forward(torch.zeros(k).expand(M, k), stream=ST)
    lin.forward(x, save=True, stream=ST)
    with pytest.raises(ValueError):
        lin.backward(torch.zeros(M, n).sum(0).expand(M, n), stream=ST)
    lin.backward(dy, stream=ST)
    with pytest.raises(ValueError):
        A.Linear(torch.zeros(k).expand(n, k), None, max_rows=M, device=DEV, stream=ST)
    # a width of one element: its rows overlap with stride 0 alone
    one = A.Linear(torch.zeros(1, 1), None, max_rows=M, device=DEV, stream=ST)
    with pytest.raises(ValueError):
        one.forward(torch.zeros(1, 1).expand(M, 1), stream=ST)
    one.forward(torch.zeros(M, 1), stream=ST)


def test_linear_accepts_one_row_of_any_stride(lib):
    lin = linear()
    lin.forward(torch.zeros(64).expand(1, 64), residual=torch.zeros(32).expand(1, 32), stream=ST)
    dims = lib.last("moe_linear_fwd")[4]
    assert dims["M"] == 1 and dims["ld_x"] in (0, 64) and dims["ld_res"] in (0, 32)


# ------------------------------------------------------------------ operands of another device
DIMS = dict(d=64, E=4, k=2, f=64, S=1, f_s=64)


def decode_params(dtype=torch.bfloat16, d=64, E=4, f=64, S=1, f_s=64, **kw):
    p = dict(w13=torch.zeros(E, 2 * f, d, dtype=dtype), w2=torch.zeros(E, d, f, dtype=dtype), w_r=torch.zeros(d, E),
             bias=torch.zeros(E), ws13=torch.zeros(S, 2 * f_s, d, dtype=dtype), ws2=torch.zeros(S, d, f_s, dtype=dtype))
    return A.LayerParams(**{**p, **kw})


def decode_layer(params=None, tokens=8, dtype=torch.bfloat16):
    params = decode_params(dtype) if params is None else params
    return A.MoEDecodeLayer(params, tokens, dtype=dtype, device=DEV, stream=ST, **DIMS)


def drafts(B_=2, n=3, V=16):
    return dict(draft_tokens=torch.zeros(B_, n, dtype=torch.int32), draft_probs=torch.zeros(B_, n, V),
                target_probs=torch.zeros(B_, n + 1, V), u_accept=torch.zeros(B_, n), u_sample=torch.zeros(B_),
                draft_len=torch.zeros(B_, dtype=torch.int32))


def elsewhere(t):
    return t.to("meta")


def test_linear_refuses_operands_of_another_device(lib):
    lin = linear()
    x, y = torch.zeros(4, 64), torch.zeros(4, 32)
    lin.forward(x, residual=y, save=True, stream=ST)
    for bad in (dict(x=elsewhere(x)), dict(x=x, residual=elsewhere(y)), dict(x=x, out=elsewhere(y))):
        with pytest.raises(ValueError, match="device"):
            lin.forward(stream=ST, **bad)
    lin.forward(x, save=True, stream=ST)
    with pytest.raises(ValueError, match="device"):
        lin.backward(elsewhere(y), stream=ST)
    for w, b in ((torch.zeros(32, 64, device="meta"), None), (torch.zeros(32, 64), torch.zeros(32, device="meta"))):
        with pytest.raises(ValueError, match="device"):
            A.Linear(w, b, device=DEV, stream=ST)


def test_decode_refuses_operands_of_another_device(lib):
    layer = decode_layer()
    x, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 4)
    layer.forward(x, residual=x, logits_in=s, stream=ST)
    for bad in (dict(x=elsewhere(x)), dict(x=x, residual=elsewhere(x)), dict(x=x, logits_in=elsewhere(s)),
                dict(x=x, out=elsewhere(x))):
        with pytest.raises(ValueError, match="device"):
            layer.forward(stream=ST, **bad)


@pytest.mark.parametrize("name", ["w13", "w2", "w_r", "bias", "ws13", "ws2"])
def test_decode_refuses_weights_that_do_not_fit(lib, name):
    """The kernel would read past a smaller, narrower or strided tensor."""
    good = getattr(decode_params(), name)
    for bad in (elsewhere(good), good[:-1], good.to(torch.float64), torch.zeros(*good.shape, 2, dtype=good.dtype)[..., 0]):
        with pytest.raises(ValueError, match=name):
            decode_layer(decode_params(**{name: bad}))
    decode_layer(decode_params(**{name: good.clone()}))


def test_decode_weights_that_are_not_used_may_be_missing(lib):
    p = decode_params(w_r=None, bias=None, ws13=None, ws2=None)
    layer = A.MoEDecodeLayer(p, 4, 64, 4, 2, 64, device=DEV, stream=ST)
    layer.forward(torch.zeros(2, 64, dtype=torch.bfloat16), logits_in=torch.zeros(2, 4), stream=ST)


def test_verify_refuses_operands_of_another_device(lib):
    ver = A.DraftVerifier(2, 3, 16, device=DEV)
    good = drafts()
    ver.verify(**good, stream=ST)
    for name in good:
        with pytest.raises(ValueError, match="device"):
            ver.verify(**{**good, name: elsewhere(good[name])}, stream=ST)


# ------------------------------------------------------------------ weights that are replaced
PARAM_FIELDS = [f for f, _ in N.LayerParams._fields_]


@pytest.mark.parametrize("how", ["tensor", "storage"])
@pytest.mark.parametrize("name", ["w13", "w2", "w_r", "bias", "ws13", "ws2"])
def test_decode_reads_the_present_weights(lib, name, how):
    """LayerParams may be changed (a training layer shares it): every call takes its present tensors."""
    layer = decode_layer()
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    layer.forward(x, stream=ST)
    old = getattr(layer.params, name)
    new = old.clone()
    if how == "tensor":
        setattr(layer.params, name, new)
    else:
        old.data = new
    layer.forward(x, stream=ST)
    given = lib.last("moe_layer_decode")[0]
    assert given[name] == new.data_ptr()
    for field in PARAM_FIELDS:
        assert given[field] == getattr(layer.params, field).data_ptr()
    setattr(layer.params, name, new[:-1])
    with pytest.raises(ValueError, match=name):
        layer.forward(x, stream=ST)
    setattr(layer.params, name, new)
    layer.forward(x, stream=ST)


def test_decode_reads_a_bias_that_comes_and_goes(lib):
    layer = decode_layer(decode_params(bias=None))
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    layer.forward(x, stream=ST)
    assert lib.last("moe_layer_decode")[0]["bias"] is None
    layer.params.bias = torch.zeros(4)
    layer.forward(x, stream=ST)
    assert lib.last("moe_layer_decode")[0]["bias"] == layer.params.bias.data_ptr()
    layer.params.bias = None
    layer.forward(x, stream=ST)
    assert lib.last("moe_layer_decode")[0]["bias"] is None


@pytest.mark.parametrize("how", ["tensor", "storage"])
def test_linear_reads_the_present_weights(lib, how):
    lin = A.Linear(torch.zeros(32, 64), torch.zeros(32), max_rows=8, device=DEV, stream=ST)
    x, dy = torch.zeros(4, 64), torch.zeros(4, 32)
    lin.forward(x, save=True, stream=ST)
    w, b = torch.zeros(32, 70)[:, :64], torch.zeros(32)
    if how == "tensor":
        lin.w, lin.bias = w, b
    else:
        lin.w.data, lin.bias.data = w, b
    lin.forward(x, save=True, stream=ST)
    given = lib.last("moe_linear_fwd")
    assert given[1] == w.data_ptr() and given[2] == b.data_ptr() and given[4]["ld_w"] == 70
    grads = lin.backward(dy, stream=ST)
    given = lib.last("moe_linear_bwd")
    assert given[1] == w.data_ptr() and given[4]["ld_w"] == 70
    assert grads["dw"].stride() == (70, 1) and grads["db"] is not None
    lin.bias = None
    lin.forward(x, stream=ST)
    assert lib.last("moe_linear_fwd")[2] is None
    for bad in (torch.zeros(31, 64), torch.zeros(32, 64, dtype=torch.bfloat16), torch.zeros(64, 32).t()):
        lin.w = bad
        with pytest.raises(ValueError):
            lin.forward(x, stream=ST)


def test_linear_workspace_follows_the_weights_stride(lib):
    """bf16 rows of W that are not whole vectors are copied into the workspace: it grows when such
    a W replaces another."""
    lin = A.Linear(torch.zeros(32, 64, dtype=torch.bfloat16), None, max_rows=8, device=DEV, stream=ST)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    lin.w = torch.zeros(32, 67, dtype=torch.bfloat16)[:, :64]
    lin.forward(x, save=True, stream=ST)
    given = lib.last("moe_linear_fwd")
    dims = N.LinearDims(8, 32, 64, 0, N.MOE_BF16, 0, 67, 0, 0)
    import ctypes
    assert given[8] >= lib.moe_linear_workspace_bytes(ctypes.byref(dims))
    assert given[7] == lin.ws.ptr and given[8] == lin.ws.nbytes
    inits = [values for n, values in lib.calls if n == "moe_op_workspace_init"]
    assert [v[0] for v in inits].count(lin.ws.ptr) == 1


# ------------------------------------------------------------------ inputs that lie on outputs
def square(rows=8, act="none", **kw):
    return linear(64, 64, rows, act=act, **kw)


def test_linear_refuses_its_own_result_as_input(lib):
    """y (dx) is written while x (dy) is still read."""
    lin = square()
    x = torch.zeros(4, 64)
    y = lin.forward(x, stream=ST)
    calls = len(lib.calls)
    for bad in (y, y[1:], y[:1]):
        with pytest.raises(ValueError, match="overlap"):
            lin.forward(bad, stream=ST)
    assert len(lib.calls) == calls
    z = lin.forward(y, out=torch.zeros(4, 64), stream=ST)      # elsewhere: as before
    lin.forward(z, stream=ST)
    lin.forward(x, save=True, stream=ST)
    grads = lin.backward(torch.zeros(4, 64), stream=ST)
    calls = len(lib.calls)
    with pytest.raises(ValueError, match="overlap"):
        lin.backward(grads["dx"], stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        lin.backward(grads["dw"][:4], stream=ST)
    assert len(lib.calls) == calls
    lin.backward(grads["dx"], need=("dw",), stream=ST)         # dx is not written
    lin.backward(lin.forward(x, save=True, stream=ST), stream=ST)   # y is not written by the backward
    # the saved x: read by dw's product, after dx is written
    kept = grads["dx"]
    lin.forward(kept, save=True, stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        lin.backward(torch.zeros(4, 64), stream=ST)
    lin.backward(torch.zeros(4, 64), need=("dx",), stream=ST)
    lin.forward(grads["dw"][:4], save=True, stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        lin.backward(torch.zeros(4, 64), need=("dw",), stream=ST)
    with_db = A.Linear(torch.zeros(64, 64), torch.zeros(64), max_rows=4, device=DEV, stream=ST)
    with_db.forward(x, save=True, stream=ST)
    db = with_db.backward(torch.zeros(4, 64), stream=ST)["db"]
    with_db.forward(db[None], save=True, stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        with_db.backward(torch.zeros(1, 64), stream=ST)
    # with an activation the gradient of z is made from dy before anything is written
    act = square(act="silu")
    act.forward(x, save=True, stream=ST)
    act.backward(act.backward(torch.zeros(4, 64), stream=ST)["dx"], stream=ST)


def test_linear_refuses_an_out_that_overlaps_an_input(lib):
    lin = square()
    buf = torch.zeros(16, 64)
    with pytest.raises(ValueError, match="overlap"):
        lin.forward(buf[:4], out=buf[3:7], stream=ST)
    lin.forward(buf[:4], out=buf[4:8], stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        lin.forward(buf[:4], residual=buf[4:8], out=buf[5:9], stream=ST)
    lin.forward(buf[:4], residual=buf[4:8], out=buf[4:8], stream=ST)       # in place
    with pytest.raises(ValueError, match="overlap"):
        lin.forward(buf[:4], out=lin.w[8:12], stream=ST)
    b = torch.zeros(2, 64)
    with_bias = A.Linear(torch.zeros(64, 64), b[1], max_rows=4, device=DEV, stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        with_bias.forward(buf[:2], out=b, stream=ST)
    with_bias.forward(buf[:1], out=b[:1], stream=ST)
    # columns of one buffer, side by side: rows lie between one another and share nothing
    wide = torch.zeros(4, 200)
    lin.forward(wide[:, :64], out=wide[:, 64:128], stream=ST)
    lin.forward(wide[:, 100:164], residual=wide[:, :64], out=wide[:, :64], stream=ST)
    with pytest.raises(ValueError, match="overlap"):
        lin.forward(wide[:, :64], out=wide[:, 63:127], stream=ST)


@pytest.mark.parametrize("seed", range(4))
def test_overlap_of_strided_matrices(seed):
    """Against the sets of elements, for equal and for different strides."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.zeros(400)
    at = torch.arange(400)
    seen = set()

    def draw(hi):
        return int(torch.randint(0, hi, (1,), generator=g))

    for _ in range(600):
        shapes = []
        for _ in range(2):
            rows, cols = draw(5), 1 + draw(9)
            ld = cols + draw(12)
            shapes.append((draw(60), rows, cols, ld))
        if draw(2):
            shapes[1] = shapes[1][:3] + (max(shapes[0][3], shapes[1][2]),)
        a, b = (buf.as_strided((r, c), (ld, 1), off) for off, r, c, ld in shapes)
        ia, ib = (at.as_strided((r, c), (ld, 1), off) for off, r, c, ld in shapes)
        want = bool(set(ia.reshape(-1).tolist()) & set(ib.reshape(-1).tolist()))
        assert A._overlap(a, shapes[0][3], b, shapes[1][3]) == want, shapes
        seen.add((want, shapes[0][3] == shapes[1][3]))
    assert len(seen) == 4


def test_decode_refuses_a_residual_that_partly_overlaps_the_output(lib):
    """x is read before any output is written; the residual while others write theirs, so it lies
    where the output does or elsewhere."""
    layer = decode_layer()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    y = layer.forward(x, residual=x, stream=ST)
    assert layer.forward(y, residual=y, stream=ST) is y
    layer.forward(y[:2], residual=y[:2], stream=ST)
    layer.forward(y[1:3], residual=y[:2], stream=ST)
    with pytest.raises(ValueError, match="residual"):
        layer.forward(x[:2], residual=y[1:3], stream=ST)
    buf = torch.zeros(8, 64, dtype=torch.bfloat16)
    layer.forward(buf[:4], residual=buf[4:], out=buf[4:], stream=ST)
    layer.forward(buf[:4], residual=buf[:4], out=buf[4:], stream=ST)
    with pytest.raises(ValueError, match="residual"):
        layer.forward(x, residual=buf[1:5], out=buf[4:], stream=ST)


def test_verify_refuses_its_results_as_inputs(lib):
    """Drafted tokens in the result's buffer: a sequence's results are written while another's (or
    its own, shifted) are read. One sequence's own first n tokens may stay where they are."""
    ver = A.DraftVerifier(4, 3, 16, device=DEV)
    good = drafts(B_=4)
    tokens, accepted = ver.verify(**good, stream=ST)
    flat = tokens.view(-1)
    for at in (0, 2, 4):
        with pytest.raises(ValueError, match="draft_tokens"):
            ver.verify(**{**good, "draft_tokens": flat[at:at + 12].view(4, 3)}, stream=ST)
    one = drafts(B_=1)
    got, n = ver.verify(**one, stream=ST)
    ver.verify(**{**one, "draft_tokens": got[:, :3]}, stream=ST)
    with pytest.raises(ValueError, match="draft_tokens"):
        ver.verify(**{**one, "draft_tokens": got[:, 1:]}, stream=ST)
    ver.verify(**{**good, "draft_len": accepted}, stream=ST)
    with pytest.raises(ValueError, match="draft_len"):
        ver.verify(**{**drafts(B_=2), "draft_len": accepted[1:3]}, stream=ST)


# ------------------------------------------------------------------ rows far apart
def test_linear_rows_far_apart_cost_no_memory(lib):
    """The last positions of long sequences lie a sequence apart: neither the gradient nor anything
    else of the layer's takes that distance."""
    n, k, rows, far = 32, 64, 8, 100000
    lin = linear(n, k, rows)
    x = torch.zeros(3, far)[:, -k:]
    dy = torch.zeros(3, n)
    lin.forward(x, save=True, stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_x"] == far
    for need in (("dx", "dw", "db"), ("dx",), ("dw",)):
        lib.calls.clear()
        grads = lin.backward(dy, need=need, stream=ST)
        calls = [v for name, v in lib.calls if name == "moe_linear_bwd"]
        assert len(calls) == min(2, len(need))
        if "dx" in need:
            assert grads["dx"].shape == (3, k) and grads["dx"].untyped_storage().nbytes() <= 4 * rows * 2 * k
            (with_dx,) = [v for v in calls if v[5] is not None]
            assert with_dx[4]["ld_x"] == grads["dx"].stride(0) and with_dx[6] is None
        if "dw" in need:
            (with_dw,) = [v for v in calls if v[6] is not None]
            assert with_dw[4]["ld_x"] == far and with_dw[0] == x.data_ptr() and with_dw[5] is None
    # a single row has no distance
    one = torch.zeros(1, far)[:, :k]
    lin.forward(one, save=True, stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_x"] == k
    lib.calls.clear()
    lin.backward(torch.zeros(1, n), stream=ST)
    assert len(lib.calls) == 1


def test_one_odd_row_keeps_its_whole_vectors(lib):
    """One bf16 row that has room for whole 16-byte vectors is not copied for their sake."""
    lin = A.Linear(torch.zeros(32, 72, dtype=torch.bfloat16)[:, :67], None, max_rows=8, device=DEV, stream=ST)
    lin.forward(torch.zeros(1, 80, dtype=torch.bfloat16)[:, :67], stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_x"] == 72
    lin.forward(torch.zeros(1, 67, dtype=torch.bfloat16), stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_x"] == 67


# ------------------------------------------------------------------ other tensors at a weight's address
BF = torch.bfloat16


@pytest.mark.parametrize("change", [lambda t: t.view(BF)[:, :32], lambda t: t.view(torch.int32), lambda t: t[:31], lambda t: t.t()])
def test_linear_refuses_a_weight_of_another_type_size_or_order_at_the_same_address(lib, change):
    lin, x, w = linear(N_=32, K=32), torch.zeros(4, 32), torch.zeros(32, 32)
    lin.w.data = w
    lin.forward(x, save=True, stream=ST)
    calls = len(lib.calls)
    lin.w.data = change(w)
    assert lin.w.data_ptr() == w.data_ptr()
    for call in (lambda: lin.forward(x, stream=ST), lambda: lin.backward(x, stream=ST)) * 2:
        with pytest.raises(ValueError):
            call()
    assert len(lib.calls) == calls
    lin.w.data = w
    lin.backward(x, stream=ST)
    lin.forward(x, stream=ST)


def test_linear_takes_another_distance_of_rows_at_the_same_address(lib):
    lin, buf = linear(N_=8, K=16), torch.zeros(8, 64)
    lin.w.data = buf[:, :16]
    lin.forward(torch.zeros(2, 16), stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_w"] == 64
    lin.w.data = buf.view(-1)[:8 * 32].view(8, 32)[:, :16]
    lin.forward(torch.zeros(2, 16), stream=ST)
    assert lib.last("moe_linear_fwd")[4]["ld_w"] == 32


@pytest.mark.parametrize("change", [lambda t: t.view(BF)[:32], lambda t: t.view(torch.int32), lambda t: t[:31], lambda t: t.as_strided((32,), (2,))])
def test_linear_refuses_a_bias_of_another_type_size_or_stride_at_the_same_address(lib, change):
    bias, here = torch.zeros(32), torch.zeros(64)[:32]
    lin = A.Linear(torch.zeros(32, 16), bias, max_rows=4, device=DEV, stream=ST)
    bias.data = here
    lin.forward(torch.zeros(4, 16), stream=ST)
    bias.data = change(here)
    for _ in range(2):
        with pytest.raises(ValueError):
            lin.forward(torch.zeros(4, 16), stream=ST)
    bias.data = here
    lin.forward(torch.zeros(4, 16), stream=ST)


@pytest.mark.parametrize("name", ["w13", "w2", "ws13", "ws2", "w_r", "bias"])
@pytest.mark.parametrize("change", [lambda t: t.view(torch.int32), lambda t: t.view(BF).view(-1)[:t.numel()].view(t.shape),
                                    lambda t: t.view(-1)[:-1], lambda t: t.as_strided(t.shape, t.stride()[:-1] + (2,))])
def test_decode_refuses_weights_of_another_type_size_or_stride_at_the_same_address(lib, name, change):
    d, E, k, f, S = 64, 4, 2, 64, 1
    sizes = dict(w13=(E, 2 * f, d), w2=(E, d, f), w_r=(d, E), bias=(E,), ws13=(S, 2 * f, d), ws2=(S, d, f))
    at = {n: torch.zeros(2 * torch.Size(s).numel()) for n, s in sizes.items()}
    here = {n: at[n][:torch.Size(s).numel()].view(s) for n, s in sizes.items()}
    params = A.LayerParams(**{n: t.view(t.shape) for n, t in here.items()})
    layer = A.MoEDecodeLayer(params, 4, d, E, k, f, S, f, torch.float32, device=DEV, stream=ST)
    x = torch.zeros(2, d)
    layer.forward(x, stream=ST)
    calls, t = len(lib.calls), getattr(params, name)
    t.data = change(here[name])
    assert t.data_ptr() == here[name].data_ptr()
    for _ in range(2):
        with pytest.raises(ValueError):
            layer.forward(x, stream=ST)
    assert len(lib.calls) == calls
    t.data = here[name].reshape(-1)          # any shape of them
    layer.forward(x, stream=ST)
