"""Host-side refusals of the operators around the layer in training, and what their wrappers hand to the
library (CPU only: calls of the C ABI here fail validation or have nothing to do, the wrappers' calls are
recorded, not made)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from dropless_token_routing_gb300 import builder as B

if not os.path.exists(B.LIB):
    B.build()

from dropless_token_routing_gb300 import _native as N  # noqa: E402
from dropless_token_routing_gb300 import api as A  # noqa: E402

L = N.lib()
BAD, GOOD = 0x1008, 0x10000   # fake addresses, never dereferenced
C = N.STATUS_CODE
REF = ctypes.byref
NULL, MIS, DIMS, DTYPE, SMALL = (C["MOE_ERR_" + s] for s in ("NULL_POINTER", "MISALIGNED", "BAD_DIMS", "UNSUPPORTED_DTYPE",
                                                              "WORKSPACE_TOO_SMALL"))


def norm_dims(**kw):
    base = dict(M=4, N=100, dtype=N.MOE_BF16, w_dtype=N.MOE_BF16, eps=1e-5, ld_x=0, ld_res=0, ld_sum=0, ld_y=0, ld_dx=0)
    base.update(kw)
    return N.NormDims(*base.values())


def logprob_dims(**kw):
    base = dict(M=4, V=100, n_top=3, dtype=N.MOE_F32, ld=0, ld_grad=0)
    base.update(kw)
    return N.LogprobDims(*base.values())


def norm_fwd(d, x=GOOD, r=GOOD, w=GOOD, b=GOOD, s=GOOD, y=GOOD, st=GOOD):
    return L.moe_norm_fwd(x, r, w, b, REF(d), s, y, st, None)


def norm_bwd(d, x=GOOD, r=GOOD, dy=GOOD, ds=GOOD, w=GOOD, st=GOOD, dx=GOOD, dw=GOOD, db=GOOD, ws=GOOD, nb=1 << 40):
    return L.moe_norm_bwd(x, r, dy, ds, w, st, REF(d), dx, dw, db, ws, nb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), DIMS), (dict(M=2**31), DIMS), (dict(N=0), DIMS), (dict(N=32769), DIMS), (dict(eps=-1e-9), DIMS),
    (dict(eps=float("nan")), DIMS), (dict(eps=float("inf")), DIMS), (dict(dtype=2), DTYPE), (dict(w_dtype=-1), DTYPE),
    (dict(dtype=N.MOE_F32, w_dtype=N.MOE_BF16), DTYPE), (dict(ld_x=99), DIMS), (dict(ld_res=1), DIMS), (dict(ld_sum=-100), DIMS),
    (dict(ld_y=50), DIMS), (dict(ld_dx=99), DIMS), (dict(ld_x=(1 << 36) + 1), DIMS)])
def test_norm_dims(bad, status):
    d = norm_dims(**bad)
    assert L.moe_norm_workspace_bytes(REF(d)) == 0
    assert norm_fwd(d) == status and norm_bwd(d) == status


def test_norm_pointers():
    d, none = norm_dims(), norm_dims(M=0)
    n = L.moe_norm_workspace_bytes(REF(d))
    for name in ("x", "w", "y"):
        assert norm_fwd(d, **{name: None}) == NULL, name
    for name in ("x", "r", "w", "b", "s", "y", "st"):
        assert norm_fwd(d, **{name: BAD}) == MIS, name
    for name in ("x", "dy", "w", "st", "ws"):
        assert norm_bwd(d, **{name: None}) == NULL, name
    for name in ("x", "r", "dy", "ds", "w", "st", "dx", "dw", "db"):
        assert norm_bwd(d, **{name: BAD}) == MIS, name
    assert norm_bwd(d, ws=GOOD + 16) == MIS and norm_bwd(d, nb=n - 1) == SMALL
    assert L.moe_norm_fwd(GOOD, None, GOOD, None, None, None, GOOD, None, None) == NULL
    assert norm_fwd(none, x=None, r=None, b=None, s=None, y=None, st=None) == 0
    assert norm_bwd(none, x=None, r=None, dy=None, ds=None, w=None, st=None, dx=None, dw=None, db=None) == 0


def test_norm_workspace_serves_fewer_rows_and_any_stride():
    for width in (1, 1001, 7680, 32768):
        sizes = {L.moe_norm_workspace_bytes(REF(norm_dims(M=M, N=width, ld_x=ld))) for M in (0, 1, 500, 10**6) for ld in (0, width + 5)}
        assert len(sizes) == 1 and sizes.pop() >= 24576


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), DIMS), (dict(M=2**31), DIMS), (dict(V=0), DIMS), (dict(V=2**22 + 1), DIMS), (dict(n_top=-1), DIMS),
    (dict(n_top=33), DIMS), (dict(dtype=7), DTYPE), (dict(ld=99), DIMS), (dict(ld_grad=99), DIMS), (dict(ld=(1 << 36) + 1), DIMS),
    (dict(ld_grad=-1), DIMS)])
def test_logprob_dims(bad, status):
    d = logprob_dims(**bad)
    assert L.moe_token_logprob(GOOD, GOOD, REF(d), GOOD, GOOD, GOOD, GOOD, GOOD, None) == status
    assert L.moe_token_logprob_bwd(GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, REF(d), GOOD, None) == status


def test_logprob_pointers():
    def fwd(dims, x=GOOD, t=GOOD, lp=GOOD, e=GOOD, s=GOOD, i=GOOD, v=GOOD):
        return L.moe_token_logprob(x, t, REF(dims), lp, e, s, i, v, None)

    def bwd(dims, x=GOOD, t=GOOD, s=GOOD, e=GOOD, gl=GOOD, ge=GOOD, dx=GOOD):
        return L.moe_token_logprob_bwd(x, t, s, e, gl, ge, REF(dims), dx, None)

    d, none = logprob_dims(), logprob_dims(M=0)
    for name in ("x", "t", "i", "v"):
        assert fwd(d, **{name: None}) == NULL, name
    for name in ("x", "s", "i", "v"):
        assert fwd(d, **{name: BAD}) == MIS, name
    for name in ("t", "lp", "e"):      # one number for a row: aligned to it
        assert fwd(d, **{name: GOOD + 2}) == MIS, name
    for name in ("x", "t", "s", "e", "dx"):
        assert bwd(d, **{name: None}) == NULL, name
    for name in ("x", "s", "dx"):
        assert bwd(d, **{name: BAD}) == MIS, name
    for name in ("t", "e", "gl", "ge"):
        assert bwd(d, **{name: GOOD + 1}) == MIS, name
    assert fwd(none, **dict.fromkeys(("x", "t", "lp", "e", "s", "i", "v"))) == 0
    assert bwd(none, **dict.fromkeys(("x", "t", "s", "e", "gl", "ge", "dx"))) == 0


def test_clip_refusals():
    def call(grads, count=None, max_norm=1.0, ws=GOOD, nb=1 << 40, norm=GOOD, scale=GOOD):
        table = (N.Grad * max(1, len(grads)))(*[N.Grad(*g) for g in grads])
        return L.moe_clip_grads(table, len(grads) if count is None else count, max_norm, norm, scale, ws, nb, None)

    good = (GOOD, GOOD, 10, N.MOE_F32)
    for bad, status in (((None, GOOD, 10, N.MOE_F32), NULL), ((GOOD + 2, GOOD, 10, N.MOE_F32), MIS), ((GOOD, GOOD + 1, 10, N.MOE_BF16), MIS),
                        ((GOOD, GOOD, -1, N.MOE_F32), DIMS), ((GOOD, GOOD, (1 << 44) + 1, N.MOE_F32), DIMS), ((GOOD, GOOD, 10, 5), DTYPE)):
        assert call([good, bad]) == status, bad
    assert call([(GOOD, None, 1 << 43, N.MOE_BF16)] * 3) == DIMS      # all together
    assert call([good], max_norm=-1.0) == DIMS and call([good], max_norm=float("nan")) == DIMS
    assert call([good], ws=None) == NULL and call([good], ws=GOOD + 8) == MIS
    assert call([good], nb=L.moe_clip_workspace_bytes(1) - 1) == SMALL
    assert call([good], norm=GOOD + 2) == MIS and call([good], scale=GOOD + 1) == MIS
    assert L.moe_clip_grads(None, 1, 1.0, GOOD, GOOD, GOOD, 1 << 40, None) == NULL
    assert call([good], count=-1) == DIMS
    assert L.moe_clip_workspace_bytes(-1) == 0
    sizes = [L.moe_clip_workspace_bytes(n) for n in (0, 1, 16, 512, 513, 5000)]
    assert sizes == sorted(sizes) and sizes[0] >= 24576


FAKE_DEVICE = r"""
/* a device of another architecture, as the CUDA runtime would report it */
int cudaGetDevice(int* dev) { *dev = 0; return 0; }
int cudaDeviceGetAttribute(int* value, int attr, int dev) {
  *value = attr == 75 ? 9 : attr == 76 ? 0 : attr == 16 ? 132 : 1;   /* major, minor, SMs */
  return dev;
}
"""


def test_other_devices_are_refused(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "fake.c", tmp_path / "fake.so"
    src.write_text(FAKE_DEVICE)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"""
import sys
sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]
import test_step_ops_cpu as T
t = (T.N.Grad * 1)(T.N.Grad(T.GOOD, T.GOOD, 10, 0))
G, d = T.GOOD, T.logprob_dims()
print([T.norm_fwd(T.norm_dims()), T.norm_bwd(T.norm_dims()), T.L.moe_token_logprob(G, G, T.REF(d), G, G, G, G, G, None),
       T.L.moe_token_logprob_bwd(G, G, G, G, G, G, T.REF(d), G, None), T.L.moe_clip_grads(t, 1, 1.0, G, G, G, 1 << 40, None)])
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True,
                         env={**os.environ, "LD_PRELOAD": str(so), "CUDA_VISIBLE_DEVICES": ""})
    assert out.stdout.strip() == str([C["MOE_ERR_UNSUPPORTED_DEVICE"]] * 5)


# ------------------------------------------------------------------ the wrappers
class Stream:
    cuda_stream = 0


ST = Stream()
DEV = "cpu:0"
BF, F32 = torch.bfloat16, torch.float32


class Recorder:
    """Stands in for the library: size calls go to it, all others are recorded and succeed."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return getattr(self.lib, name)

        def call(*args):
            values = [getattr(a, "_obj", a) for a in args]
            values = [{f: getattr(v, f) for f, _ in v._fields_} if hasattr(v, "_fields_") else
                      [(g.g, g.out, g.n, g.dtype) for g in v] if isinstance(v, ctypes.Array) else v for v in values]
            self.calls.append((name, values))
            return 0

        return call

    def last(self, name):
        return [values for n, values in self.calls if n == name][-1]


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder(N.lib())
    monkeypatch.setattr(N, "lib", lambda: rec)
    return rec


def layer_norm(n=64, rows=8, dtype=F32, w_dtype=None, bias=True):
    w = torch.zeros(n, dtype=w_dtype or dtype)
    return A.LayerNorm(w, w.clone() if bias else None, max_rows=rows, dtype=dtype, device=DEV)


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_norm_refuses_what_does_not_fit(lib):
    ln, x = layer_norm(), z(4, 64)
    ln.forward(x, residual=x, stream=ST)
    for bad in (z(4, 63), z(4, 64, dtype=BF), x.to("meta"), z(64).expand(4, 64), z(4, 128)[:, ::2], z(9, 64)):
        with pytest.raises(ValueError):
            ln.forward(bad, stream=ST)
    for bad in (z(3, 64), z(4, 64, dtype=BF), x.to("meta"), z(64).expand(4, 64)):
        for kw in (dict(residual=bad), dict(out=bad), dict(residual=x, sum_out=bad)):
            with pytest.raises(ValueError):
                ln.forward(x, stream=ST, **kw)
    with pytest.raises(ValueError):
        ln.forward(x, sum_out=z(4, 64), stream=ST)      # there is no sum
    with pytest.raises(ValueError):
        ln.backward(x, stream=ST)                       # nothing was saved
    ln.forward(x, save=True, stream=ST)
    for kw in (dict(dy=z(3, 64)), dict(dy=x, d_sum=z(4, 63)), dict(dy=x.to("meta")), dict(dy=x, out=z(5, 64))):
        with pytest.raises(ValueError):
            ln.backward(stream=ST, **kw)
    with pytest.raises(ValueError):
        A.LayerNorm(z(64), z(63), device=DEV)
    with pytest.raises(ValueError):
        A.LayerNorm(z(64), z(64, dtype=BF), device=DEV)
    for kw in (dict(dtype=F32, weight=z(64, dtype=BF)), dict(weight=z(40000)), dict(weight=z(64), eps=-1.0)):
        with pytest.raises(N.MoeError):
            A.LayerNorm(device=DEV, **kw)


def test_norm_refuses_results_over_operands(lib):
    """In place is allowed where a result lies just where its operand does, not a row further."""
    ln, buf = layer_norm(), z(9, 64)
    x, later, r = buf[:4], buf[1:5], z(4, 64)
    ln.forward(x, out=x, stream=ST)
    ln.forward(x, residual=r, out=x, sum_out=r, stream=ST)
    ln.forward(x, residual=r, out=r, sum_out=x, stream=ST)
    for kw in (dict(x=x, out=later), dict(x=r, residual=x, out=later), dict(x=r, residual=x, sum_out=later),
               dict(x=x, residual=r, sum_out=later), dict(x=x, residual=r, out=later, sum_out=later),
               dict(x=x, residual=r, out=x, sum_out=x), dict(x=x, save=True, out=x), dict(x=x, out=ln.weight.expand(1, 64))):
        if kw.get("out") is not None and kw["out"].shape[0] == 1:
            kw["x"] = x[:1]
        with pytest.raises(ValueError):
            ln.forward(stream=ST, **kw)
    y = ln.forward(x, stream=ST)
    ln.forward(y, stream=ST)                            # its own result, in place
    with pytest.raises(ValueError):
        ln.forward(ln._bufs["y"][1:4], stream=ST)       # a row further
    ln.forward(x, residual=r, save=True, stream=ST)
    s = ln.backward(x, d_sum=r, out=r, stream=ST)["dx"]
    assert s is r
    for kw in (dict(dy=x, out=later), dict(dy=r, d_sum=x, out=later), dict(dy=r, out=ln._bufs["sum"][1:5])):
        with pytest.raises(ValueError):
            ln.backward(stream=ST, **kw)


def test_norm_reads_the_present_weights(lib):
    ln, x = layer_norm(), z(4, 64)
    ln.forward(x, save=True, stream=ST)
    for name, at in (("weight", 2), ("bias", 3)):
        for how in ("tensor", "storage"):
            new = z(64)
            if how == "tensor":
                setattr(ln, name, new)
            else:
                getattr(ln, name).data = new
            ln.forward(x, save=True, stream=ST)
            assert lib.last("moe_norm_fwd")[at] == new.data_ptr()
            ln.backward(x, stream=ST)
            assert lib.last("moe_norm_bwd")[4] == ln.weight.data_ptr()
    ln.weight = z(63)
    for _ in range(2):                                  # (not taken the second time either)
        with pytest.raises(ValueError):
            ln.forward(x, stream=ST)


def test_norm_hands_over_strides_and_what_it_kept(lib):
    n = 64
    x, r, dy, ds, out = (z(8, w)[:4, :n] for w in (70, 72, 80, 66, 96))
    ln = layer_norm()
    ln.forward(x, residual=r, save=True, stream=ST)
    d = lib.last("moe_norm_fwd")[4]
    assert (d["M"], d["N"], d["ld_x"], d["ld_res"], d["ld_sum"], d["ld_y"]) == (4, n, 70, 72, n, n)
    ln.backward(dy, d_sum=ds, out=out, stream=ST)
    v = lib.last("moe_norm_bwd")
    assert v[0] == ln._bufs["sum"].data_ptr() and v[1] is None      # the sum
    d = v[6]
    assert (d["ld_x"], d["ld_res"], d["ld_sum"], d["ld_y"], d["ld_dx"]) == (n, 0, 66, 80, 96)
    # bf16 rows: x and the residual, unless one of them was overwritten
    x, r = z(4, n, dtype=BF), z(4, n, dtype=BF)
    for w_dtype in (BF, F32):
        ln = layer_norm(dtype=BF, w_dtype=w_dtype)
        ln.forward(x, residual=r, save=True, stream=ST)
        ln.backward(x, stream=ST)
        assert lib.last("moe_norm_bwd")[:2] == [x.data_ptr(), r.data_ptr()]
    ln.forward(x, residual=r, sum_out=r, save=True, stream=ST)
    ln.backward(x, stream=ST)
    assert lib.last("moe_norm_bwd")[:2] == [r.data_ptr(), None]
    ln.forward(x, stream=ST)
    with pytest.raises(ValueError):
        ln.backward(x, stream=ST)       # this forward kept nothing


def test_logprob_wrapper(lib):
    lp = A.TokenLogprobs(6, 50, top=1, device=DEV, stream=None)
    x, t = z(4, 50), torch.zeros(4, dtype=torch.int32)
    for bad in (z(4, 49), z(7, 50), z(4, 50, dtype=BF), x.to("meta"), z(50).expand(4, 50), z(4, 100)[:, ::2]):
        with pytest.raises(ValueError):
            lp.forward(bad, stream=ST)
    for bad in (t[:3], t.long(), t.to("meta"), torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            lp.forward(x, bad, stream=ST)
    with pytest.raises(ValueError):
        lp.backward(z(4), stream=ST)
    out = lp.forward(x, t, entropy=True, save=True, stream=ST)
    assert set(out) == {"logprob", "entropy", "top_idx", "top_logprob"}
    lp.backward(z(4), d_entropy=z(4), stream=ST)
    for kw in (dict(d_logprob=z(3)), dict(d_logprob=z(4, dtype=BF)), dict(d_entropy=z(5)), dict(d_logprob=z(4).to("meta")),
               dict(d_logprob=z(4), out=z(4, 49)), dict(d_logprob=z(4), out=z(50).expand(4, 50))):
        with pytest.raises(ValueError):
            lp.backward(stream=ST, **kw)
    assert lp.backward(z(4), out=x, stream=ST) is x
    buf = z(9, 50)
    lp.forward(buf[:4], t, save=True, stream=ST)
    with pytest.raises(ValueError):
        lp.backward(z(4), out=buf[1:5], stream=ST)      # a row further than the scores
    with pytest.raises(ValueError):
        lp.backward(d_entropy=z(4), stream=ST)          # no entropy was taken
    # the last alternatives as the next tokens: they are overwritten before the backward reads them
    own = lp.forward(x, stream=ST)["top_idx"][:, 0]
    lp.forward(x, own, stream=ST)
    with pytest.raises(ValueError):
        lp.forward(x, own, save=True, stream=ST)
    lp.forward(z(4, 64)[:, :50], t, stream=ST)
    assert lib.last("moe_token_logprob")[2]["ld"] == 64
    for kw in (dict(V=0), dict(V=1 << 23), dict(top=33), dict(top=-1)):
        with pytest.raises(N.MoeError):
            A.TokenLogprobs(**{**dict(max_rows=4, V=50, device=DEV), **kw})


def clipper(grads, out=None):
    return A.GradClipper(grads, out=out, device=DEV, stream=ST)


def test_clip_hands_over_the_list(lib):
    a, b, c = z(5), z(3, 4, dtype=BF), z(0)
    k = clipper({"a": a, "none": None, "b": b, "c": c})
    k.clip(2.5, stream=ST)
    v = lib.last("moe_clip_grads")
    assert v[0][:2] == [(a.data_ptr(), a.data_ptr(), 5, 0), (b.data_ptr(), b.data_ptr(), 12, 1)] and v[0][2][2] == 0
    assert v[1] == 3 and abs(v[2] - 2.5) < 1e-6
    k.norm(stream=ST)
    v = lib.last("moe_clip_grads")
    assert all(out is None for _, out, _, _ in v[0]) and v[2] == float("inf")
    a.data = z(7)
    k.clip(1.0, stream=ST)
    assert lib.last("moe_clip_grads")[0][0] == (a.data_ptr(), a.data_ptr(), 7, 0)      # moved, and larger
    clipper([]).norm(stream=ST)


def test_clip_refuses_lists_that_do_not_fit(lib):
    flat = z(100)
    clipper([flat[:50], flat[50:]])
    for grads in ([flat[:50], flat[49:]], [flat, flat], [flat[:10], flat[5:6]]):
        with pytest.raises(ValueError, match="overlaps"):
            clipper(grads)
    o = z(100)
    clipper([flat, flat], out=[o, z(100)])              # read twice, written apart
    for grads, out in (([flat[:50], flat[50:]], [o[:50], o[49:99]]), ([flat[:50]], [flat[1:51]]), ([flat[:50], flat[50:]], [flat[50:], o[:50]])):
        with pytest.raises(ValueError, match="overlaps"):
            clipper(grads, out)
    for grads, out in (([z(4, 8)[:, ::2]], None), ([z(4, dtype=torch.float64)], None), ([z(4).to("meta")], None), ([z(4)], [z(5)]),
                       ([z(4)], [z(4, dtype=BF)]), ([z(4)], []), ([z(4), None], [z(4), z(4)])):
        with pytest.raises(ValueError):
            clipper(grads, out)
    k = clipper([flat[:50], flat[50:]])
    k.grads[1].data = flat[:50]                         # moved onto the other one
    with pytest.raises(ValueError, match="overlaps"):
        k.clip(1.0, stream=ST)


def test_results_are_views_of_kept_buffers(lib):
    """A call with fewer rows returns the first rows of the same buffers."""
    ln, lp = layer_norm(), A.TokenLogprobs(8, 30, top=2, device=DEV)
    a, b = ln.forward(z(8, 64), stream=ST), ln.forward(z(3, 64), stream=ST)
    assert a.data_ptr() == b.data_ptr() and b.shape == (3, 64)
    p, q = lp.forward(z(8, 30), stream=ST), lp.forward(z(2, 30), stream=ST)
    assert p["top_idx"].data_ptr() == q["top_idx"].data_ptr() and q["top_logprob"].shape == (2, 2)


def test_what_a_gradient_overwrote_is_no_longer_kept(lib):
    """A second backward would read the first one's result."""
    x, r, s, dy = (z(4, 64, dtype=BF) for _ in range(4))
    ln = layer_norm(dtype=BF)
    for place, kw in ((x, {}), (x, dict(residual=r)), (r, dict(residual=r)), (s, dict(residual=r, out=x, sum_out=s))):
        ln.forward(x, save=True, stream=ST, **kw)
        ln.backward(dy, stream=ST)
        ln.backward(dy, out=dy, stream=ST)
        ln.backward(dy, out=place, need=("dw", "db"), stream=ST)     # not written
        ln.backward(dy, out=place, stream=ST)
        with pytest.raises(ValueError):
            ln.backward(dy, stream=ST)
    lp, x = A.TokenLogprobs(4, 50, device=DEV), z(4, 50)
    lp.forward(x, torch.zeros(4, dtype=torch.int32), save=True, stream=ST)
    lp.backward(z(4), stream=ST)
    lp.backward(z(4), out=x, stream=ST)
    with pytest.raises(ValueError):
        lp.backward(z(4), stream=ST)


def test_logprob_tokens_among_the_alternatives(lib):
    """A row's alternatives would be written over the next rows' tokens."""
    x = z(4, 50)
    for top in (2, 5):
        lp = A.TokenLogprobs(4, 50, top=top, device=DEV)
        idx = lp.forward(x, stream=ST)["top_idx"].view(-1)
        for i in (0, 1, 4 * top - 4):
            with pytest.raises(ValueError):
                lp.forward(x, idx[i:i + 4], stream=ST)
    lp = A.TokenLogprobs(8, 50, top=1, device=DEV)
    idx = lp.forward(z(8, 50), stream=ST)["top_idx"].view(-1)
    lp.forward(x, idx[:4], stream=ST)
    lp.forward(x, idx[4:], stream=ST)
    with pytest.raises(ValueError):
        lp.forward(x, idx[1:5], stream=ST)


def test_views_of_many_numbers_of_rows(lib):
    """What is kept for each number of rows that came up stays bounded, and a backward works all the same."""
    rows = 3 * A._KEPT_VIEWS
    ln, lp, x = layer_norm(n=1, rows=rows), A.TokenLogprobs(rows, 1, top=1, device=DEV), z(rows, 1)
    for M in range(1, rows + 1):
        y = ln.forward(x[:M], save=True, stream=ST)
        assert y.shape == (M, 1) and ln.backward(x[:M], stream=ST)["dx"].shape == (M, 1)
        assert lp.forward(x[:M], stream=ST)["top_idx"].shape == (M, 1)
    assert max(map(len, (ln._views, ln._shapes, lp._views))) <= A._KEPT_VIEWS
    assert lib.last("moe_norm_bwd")[5] == ln._bufs["stats"].data_ptr()


def test_clip_takes_tensors_of_another_type_or_order_at_the_same_address(lib):
    """Address and number of elements alone do not say what lies there."""
    a, o = z(100), z(100)
    for out in (None, [o]):
        for call in ("clip", "norm"):
            a.data, o.data = z(100), z(100)
            k = clipper([a], out=out)
            run = (lambda: k.clip(1.0, stream=ST)) if call == "clip" else (lambda: k.norm(stream=ST))
            run()
            at, here = a.data_ptr(), a.data
            a.data = here.view(BF)[:100]
            if out is not None:
                o.data = o.data.view(BF)[:100]
            run()
            assert lib.last("moe_clip_grads")[0][0] == (at, None if call == "norm" else k.out[0].data_ptr(), 100, N.MOE_BF16)
            a.data = here.view(torch.int32)      # no type that it takes
            with pytest.raises(ValueError):
                run()
            a.data = here
            if out is not None:
                with pytest.raises(ValueError):  # the result's type is still the other one
                    run()


def test_clip_refuses_tensors_that_were_transposed(lib):
    a, o = z(4, 4), z(4, 4)
    for out, t in ((None, a), ([o], a), ([o], o)):
        k = clipper([a], out=out)
        for run in (lambda: k.clip(1.0, stream=ST), lambda: k.norm(stream=ST)):
            run()
            t.data = t.data.t()
            for _ in range(2):                   # (not the second time either)
                with pytest.raises(ValueError):
                    k.clip(1.0, stream=ST)
            t.data = t.data.t()
            run()


def test_clip_takes_fewer_elements_at_the_same_address(lib):
    a = z(100)
    k = clipper([a])
    k.clip(1.0, stream=ST)
    a.data = a.data[:60]
    k.clip(1.0, stream=ST)
    assert lib.last("moe_clip_grads")[0][0] == (a.data_ptr(), a.data_ptr(), 60, 0)


@pytest.mark.parametrize("change", [lambda t: t.view(BF)[:64], lambda t: t.view(torch.int32), lambda t: t[:63],
                                    lambda t: t.as_strided((64,), (2,))])
def test_norm_refuses_weights_of_another_type_size_or_stride_at_the_same_address(lib, change):
    x, ln = z(4, 64), layer_norm()
    for name in ("weight", "bias"):
        t, here = getattr(ln, name), z(128)[:64]
        t.data = here
        ln.forward(x, save=True, stream=ST)
        calls = len(lib.calls)
        t.data = change(here)
        assert t.data_ptr() == here.data_ptr()
        for call in (lambda: ln.forward(x, stream=ST), lambda: ln.backward(x, stream=ST)) * 2:
            with pytest.raises(ValueError):
                call()
        assert len(lib.calls) == calls
        t.data = here
        ln.backward(x, stream=ST)
        ln.forward(x, stream=ST)


def test_norm_weights_that_require_gradients_and_modes(lib):
    """What else may change about a weight changes nothing."""
    x, w = z(4, 64), torch.nn.Parameter(z(64))
    for bias in (None, torch.nn.Parameter(z(64))):
        ln = A.LayerNorm(w, bias, max_rows=4, device=DEV)
        for needed in (True, False, True):
            w.requires_grad_(needed)
            for mode in (torch.enable_grad, torch.no_grad, torch.inference_mode, torch.enable_grad):
                with mode():
                    ln.forward(x, save=True, stream=ST)
                    assert lib.last("moe_norm_fwd")[2] == w.data_ptr()
                    ln.backward(x, stream=ST)


def test_logprob_backward_does_not_read_the_returned_entropy(lib):
    """It may be changed between the passes (masked, weighted): the backward has its own."""
    lp = A.TokenLogprobs(6, 50, device=DEV)
    out = lp.forward(z(4, 50), torch.zeros(4, dtype=torch.int32), entropy=True, save=True, stream=ST)
    stats = lib.last("moe_token_logprob")[5]
    lp.backward(z(4), d_entropy=z(4), stream=ST)
    _, _, kept, entropy, _, _, dims, _, _ = lib.last("moe_token_logprob_bwd")
    assert kept == stats and entropy is None and dims["keep_entropy"] == lib.last("moe_token_logprob")[2]["keep_entropy"] == 1
    assert not any(r.data_ptr() <= stats < r.data_ptr() + 4 * r.numel() for r in out.values())


def test_logprob_entropy_among_the_statistics():
    G = GOOD
    for bad in (-1, 2):
        d = logprob_dims(keep_entropy=bad)
        assert L.moe_token_logprob(G, G, REF(d), G, G, G, G, G, None) == DIMS
        assert L.moe_token_logprob_bwd(G, G, G, G, G, G, REF(d), G, None) == DIMS
    with_own, kept = logprob_dims(M=0), logprob_dims(M=0, keep_entropy=1)
    for d in (with_own, kept):
        assert L.moe_token_logprob_bwd(G, G, G, None, G, G, REF(d), G, None) == 0
    assert L.moe_token_logprob_bwd(G, G, G, None, G, G, REF(logprob_dims()), G, None) == NULL
    assert L.moe_token_logprob_bwd(G, G, None, None, G, G, REF(logprob_dims(keep_entropy=1)), G, None) == NULL


def test_norm_refuses_operands_in_its_own_weight_gradients(lib):
    """dw is written before dx is formed: an earlier call's dw as an operand would be read half overwritten."""
    for w_dtype, rows in ((F32, 1), (BF, 1), (F32, 2)):
        dtype = BF if rows == 2 else w_dtype
        ln = A.LayerNorm(z(64, dtype=w_dtype), z(64, dtype=w_dtype), max_rows=4, dtype=dtype, device=DEV)
        x, r, dy = (z(rows, 64, dtype=dtype) for _ in range(3))
        ln.forward(x, save=True, stream=ST)
        grads = ln.backward(dy, stream=ST)
        for name in ("dw", "db"):
            own = grads[name].view(dtype)[:rows * 64].view(rows, 64)
            calls = len(lib.calls)
            for kw in (dict(dy=own), dict(dy=dy, d_sum=own), dict(dy=dy, out=own)):
                with pytest.raises(ValueError, match="gradient"):
                    ln.backward(stream=ST, **kw)
            assert len(lib.calls) == calls
            ln.backward(own, need=("dx",), stream=ST)       # neither is written
            ln.forward(own, save=True, stream=ST)
            with pytest.raises(ValueError, match="gradient"):
                ln.backward(dy, stream=ST)
            ln.backward(dy, need=("dx",), stream=ST)
            if dtype == BF:
                ln.forward(x, residual=own, save=True, stream=ST)
                with pytest.raises(ValueError, match="gradient"):
                    ln.backward(dy, stream=ST)
            ln.forward(x, save=True, stream=ST)
            ln.backward(own.clone(), stream=ST)


def test_norm_refuses_weights_in_its_own_results(lib):
    for name in ("weight", "bias"):
        ln, x = layer_norm(), z(4, 64)
        y = ln.forward(x, save=True, stream=ST)
        grads = ln.backward(x, stream=ST)
        good = getattr(ln, name)
        for bad in (grads["dw"], grads["db"], y[1], grads["dx"][3]):
            setattr(ln, name, bad)
            for call in (lambda: ln.forward(x, stream=ST), lambda: ln.backward(x, stream=ST)):
                with pytest.raises(ValueError, match="result"):
                    call()
            setattr(ln, name, bad.clone())
            ln.forward(x, save=True, stream=ST)
        setattr(ln, name, good)
        ln.forward(x, stream=ST)


def test_logprob_refuses_scores_in_its_own_results(lib):
    lp, x = A.TokenLogprobs(8, 20, top=20, device=DEV), z(4, 20)
    top = lp.forward(x, stream=ST)["top_logprob"]
    for bad in (top, top[1:2], top[1:]):
        with pytest.raises(ValueError, match="overlaps"):
            lp.forward(bad, stream=ST)
    lp.forward(top.clone(), stream=ST)
    one = A.TokenLogprobs(8, 1, device=DEV)
    out = one.forward(z(8, 1), torch.zeros(8, dtype=torch.int32), entropy=True, stream=ST)
    for name in ("logprob", "entropy"):
        with pytest.raises(ValueError, match="overlaps"):
            one.forward(out[name][:, None], stream=ST)


def test_logprob_refuses_an_earlier_gradient_as_the_results_gradient(lib):
    """The scores' gradient is written over it while other rows read it."""
    lp, t = A.TokenLogprobs(4, 50, device=DEV), torch.zeros(4, dtype=torch.int32)
    lp.forward(z(4, 50), t, entropy=True, save=True, stream=ST)
    d = lp.backward(z(4), stream=ST)
    for kw in (dict(d_logprob=d[0, :4]), dict(d_logprob=z(4), d_entropy=d[3, 46:]), dict(d_logprob=d[1, 3:7], out=d)):
        with pytest.raises(ValueError, match="overlaps"):
            lp.backward(stream=ST, **kw)
    lp.backward(d[0, :4].clone(), d_entropy=d[1, :4], out=z(4, 50), stream=ST)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode, lambda: torch.autocast("cpu", dtype=BF)])
def test_kept_tensors_in_other_modes(lib, mode):
    """Calls inside and outside of a mode, in turn: the same tensors, the same pointers."""
    a, w, x = z(10), z(64), z(4, 64)
    k, ln = clipper([a]), A.LayerNorm(w, w.clone(), max_rows=4, device=DEV)
    for _ in range(2):
        with mode():
            k.clip(1.0, stream=ST)
            ln.forward(x, save=True, stream=ST)
            ln.backward(x, stream=ST)
        k.norm(stream=ST)
        ln.forward(x, save=True, stream=ST)
        ln.backward(x, stream=ST)
    a.requires_grad_()
    k.clip(1.0, stream=ST)
    assert {v[0][0][0] for n, v in lib.calls if n == "moe_clip_grads"} == {a.data_ptr()}
    assert {v[2] for n, v in lib.calls if n == "moe_norm_fwd"} == {w.data_ptr()}


def test_kept_tensors_where_torch_has_no_check_of_many(lib, monkeypatch):
    """Each is asked then: a change is found as well, and none is where there is none."""
    monkeypatch.delattr(torch._C._dynamo.guards, "TensorGuards")
    monkeypatch.setattr(A, "_addresses_are", None)
    a, w, x = z(10), z(64), z(4, 64)
    k, ln = clipper([a]), A.LayerNorm(w, max_rows=4, device=DEV)
    bound = k._places
    for _ in range(2):
        k.clip(1.0, stream=ST)
        ln.forward(x, stream=ST)
    assert k._places is bound
    here = a.data
    a.data = here.view(BF)[:10]
    k.clip(1.0, stream=ST)
    assert lib.last("moe_clip_grads")[0][0] == (a.data_ptr(), a.data_ptr(), 10, N.MOE_BF16)
    a.data = z(20)[::2]
    w.data = w.data[:63]
    for call in (lambda: k.norm(stream=ST), lambda: ln.forward(x, stream=ST)):
        with pytest.raises(ValueError):
            call()
