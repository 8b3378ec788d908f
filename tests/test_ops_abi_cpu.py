"""Host-side refusals and workspace sizes of the few-token operators (CPU only: every call here
fails validation or has nothing to do, so no CUDA API is touched)."""
import ctypes
import os

import pytest

from dropless_token_routing_gb300 import builder as B

if not os.path.exists(B.LIB):
    B.build()

from dropless_token_routing_gb300 import _native as N  # noqa: E402

L = N.lib()
BAD, GOOD = 0x1008, 0x10000   # fake addresses, never dereferenced
C = N.STATUS_CODE
REF = ctypes.byref


def layer_dims(**kw):
    base = dict(T=4, d=512, E=8, k=2, f=256, S=0, f_s=0, dtype=N.MOE_BF16, capacity=0, rearrange=0)
    base.update(kw)
    return N.MoeDims(*base.values())


def linear_dims(**kw):
    base = dict(M=4, N=96, K=64, act=0, dtype=N.MOE_BF16, ld_x=0, ld_w=0, ld_y=0, ld_res=0)
    base.update(kw)
    return N.LinearDims(*base.values())


def verify_dims(**kw):
    base = dict(B=2, n=3, V=100, dtype=N.MOE_F32, ld_draft=0, ld_target=0)
    base.update(kw)
    return N.VerifyDims(*base.values())


def test_workspace_init_is_checked():
    assert L.moe_op_workspace_init(None, 4096, None) == C["MOE_ERR_NULL_POINTER"]
    assert L.moe_op_workspace_init(GOOD + 16, 4096, None) == C["MOE_ERR_MISALIGNED"]
    assert L.moe_op_workspace_init(GOOD, 4095, None) == C["MOE_ERR_WORKSPACE_TOO_SMALL"]


@pytest.mark.parametrize("bad", [dict(T=65), dict(T=-1), dict(k=9), dict(d=96), dict(E=1025), dict(capacity=4),
                                 dict(rearrange=1), dict(dtype=5), dict(S=9, f_s=64), dict(S=1, f_s=0)])
def test_decode_dims(bad):
    d = layer_dims(**bad)
    assert L.moe_decode_workspace_bytes(REF(d)) == 0
    p = N.LayerParams(GOOD, None, GOOD, GOOD, GOOD, GOOD)
    assert L.moe_layer_decode(REF(p), GOOD, None, None, REF(d), None, None, GOOD, GOOD, 1 << 40, None) < 0


def test_decode_workspace_grows_with_every_size():
    base = dict(T=8, d=512, E=16, k=2, f=256, S=1, f_s=128)
    n0 = L.moe_decode_workspace_bytes(REF(layer_dims(**base)))
    assert n0 >= 4096
    for name, v in (("T", 64), ("E", 1024), ("k", 8), ("f", 4096), ("S", 8), ("f_s", 4096)):
        assert L.moe_decode_workspace_bytes(REF(layer_dims(**{**base, name: v}))) >= n0
    assert L.moe_decode_workspace_bytes(REF(layer_dims(T=0))) >= 4096


def test_decode_pointers():
    d = layer_dims(S=1, f_s=64)
    n = L.moe_decode_workspace_bytes(REF(d))
    full = dict(w_r=GOOD, bias=None, w13=GOOD, w2=GOOD, ws13=GOOD, ws2=GOOD)

    def call(x=GOOD, logits=None, res=None, idx=None, w=None, y=GOOD, ws=GOOD, nb=n, dims=d, **kw):
        p = N.LayerParams(*{**full, **kw}.values())
        return L.moe_layer_decode(REF(p), x, logits, res, REF(dims), idx, w, y, ws, nb, None)

    null, mis = C["MOE_ERR_NULL_POINTER"], C["MOE_ERR_MISALIGNED"]
    for name in ("x", "y", "w_r", "w13", "w2", "ws13", "ws2", "ws"):
        assert call(**{name: None}) == null, name
    for name in ("x", "logits", "res", "idx", "w", "y", "w_r", "bias", "w13", "w2", "ws13", "ws2"):
        assert call(**{name: BAD}) == mis, name
    assert call(ws=GOOD + 16) == mis
    assert call(nb=n - 1) == C["MOE_ERR_WORKSPACE_TOO_SMALL"]
    assert L.moe_layer_decode(None, GOOD, None, None, REF(d), None, None, GOOD, GOOD, n, None) == null
    assert call(x=None, y=None, dims=layer_dims(T=0, S=1, f_s=64)) == 0   # nothing to do


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), "MOE_ERR_BAD_DIMS"), (dict(N=0), "MOE_ERR_BAD_DIMS"), (dict(K=0), "MOE_ERR_BAD_DIMS"),
    (dict(act=5), "MOE_ERR_BAD_DIMS"), (dict(act=-1), "MOE_ERR_BAD_DIMS"), (dict(ld_x=63), "MOE_ERR_BAD_DIMS"),
    (dict(ld_w=10), "MOE_ERR_BAD_DIMS"), (dict(ld_y=95), "MOE_ERR_BAD_DIMS"), (dict(ld_res=1), "MOE_ERR_BAD_DIMS"),
    (dict(M=2**31), "MOE_ERR_BAD_DIMS"), (dict(dtype=2), "MOE_ERR_UNSUPPORTED_DTYPE")])
def test_linear_dims(bad, status):
    d = linear_dims(**bad)
    assert L.moe_linear_workspace_bytes(REF(d)) == 0
    assert L.moe_linear_fwd(GOOD, GOOD, None, None, REF(d), None, GOOD, GOOD, 1 << 40, None) == C[status]
    assert L.moe_linear_bwd(GOOD, GOOD, GOOD, GOOD, REF(d), GOOD, GOOD, GOOD, GOOD, 1 << 40, None) == C[status]


def test_linear_pointers():
    d = linear_dims(act=N.ACTS["gelu"])
    n = L.moe_linear_workspace_bytes(REF(d))
    null, mis = C["MOE_ERR_NULL_POINTER"], C["MOE_ERR_MISALIGNED"]

    def fwd(x=GOOD, w=GOOD, b=None, r=None, z=None, y=GOOD, ws=GOOD, nb=n, dims=d):
        return L.moe_linear_fwd(x, w, b, r, REF(dims), z, y, ws, nb, None)

    def bwd(x=GOOD, w=GOOD, z=GOOD, dy=GOOD, dx=GOOD, dw=GOOD, db=GOOD, ws=GOOD, nb=n, dims=d):
        return L.moe_linear_bwd(x, w, z, dy, REF(dims), dx, dw, db, ws, nb, None)

    for name in ("x", "w", "y", "ws"):
        assert fwd(**{name: None}) == null, name
    for name in ("x", "w", "b", "r", "z", "y"):
        assert fwd(**{name: BAD}) == mis, name
    for name in ("x", "w", "z", "dy", "ws"):
        assert bwd(**{name: None}) == null, name
    for name in ("x", "w", "z", "dy", "dx", "dw", "db"):
        assert bwd(**{name: BAD}) == mis, name
    assert fwd(nb=n - 1) == C["MOE_ERR_WORKSPACE_TOO_SMALL"] and bwd(nb=n - 1) == C["MOE_ERR_WORKSPACE_TOO_SMALL"]
    assert fwd(x=None, y=None, dims=linear_dims(M=0)) == 0
    assert bwd(x=None, z=None, dy=None, dx=None, dw=None, db=None, dims=linear_dims(M=0)) == 0


@pytest.mark.parametrize("bad", [dict(B=-1), dict(n=-1), dict(n=1025), dict(V=0), dict(V=2**22 + 1), dict(ld_draft=99),
                                 dict(ld_target=50)])
def test_verify_dims(bad):
    d = verify_dims(**bad)
    assert L.moe_verify_draft(GOOD, None, GOOD, GOOD, GOOD, GOOD, REF(d), GOOD, GOOD, None) == C["MOE_ERR_BAD_DIMS"]


def test_verify_pointers():
    null, mis = C["MOE_ERR_NULL_POINTER"], C["MOE_ERR_MISALIGNED"]
    order = ("tokens", "length", "q", "p", "u", "us")

    def call(dims, out=GOOD, acc=GOOD, **kw):
        a = {**dict.fromkeys(order, GOOD), "length": None, **kw}
        return L.moe_verify_draft(*[a[k] for k in order], REF(dims), out, acc, None)

    d = verify_dims()
    for name in ("tokens", "q", "p", "u", "us", "out", "acc"):
        assert call(d, **{name: None}) == null, name
    for name in order + ("out", "acc"):
        assert call(d, **{name: BAD}) == mis, name
    assert call(verify_dims(dtype=9)) == C["MOE_ERR_UNSUPPORTED_DTYPE"]
    assert call(verify_dims(n=0), tokens=None, q=None, u=None, p=None) == null
    assert call(verify_dims(B=0), **dict.fromkeys(("tokens", "q", "p", "u", "us", "out", "acc"))) == 0


@pytest.mark.parametrize("dtype", [N.MOE_F32, N.MOE_BF16])
@pytest.mark.parametrize("width", [(64, 64), (1001, 777), (4096, 2048), (200, 100000)])
def test_linear_workspace_serves_fewer_rows(dtype, width):
    """A workspace for M rows is large enough for fewer, with any stride of x and y."""
    last = 0
    for M in (0, 1, 64, 65, 128, 129, 700, 1024, 5000, 9000, 100000):
        dims = N.LinearDims(M, *width, 0, dtype, 0, 0, 0, 0)
        need = L.moe_linear_workspace_bytes(ctypes.byref(dims))
        odd = N.LinearDims(M, *width, 4, dtype, width[1] + 3, 0, width[0] + 1, 0)
        assert need == L.moe_linear_workspace_bytes(ctypes.byref(odd))
        assert need >= last > 0 or M == 0
        last = need


FAKE_DEVICE = r"""
/* a device of another architecture, as the CUDA runtime would report it */
int cudaGetDevice(int* dev) { *dev = 0; return 0; }
int cudaDeviceGetAttribute(int* value, int attr, int dev) {
  *value = attr == 75 ? 9 : attr == 76 ? 0 : attr == 16 ? 132 : 1;   /* major, minor, SMs */
  return dev;
}
"""


@pytest.mark.parametrize("call", ["decode_bf16", "decode_f32", "linear_bf16", "linear_f32", "linear_bwd", "verify"])
def test_other_devices_are_refused(tmp_path, call):
    """The library holds sm_103 code alone: on another device a call is refused, not left to fail
    at its launch. The runtime's answers about the device are faked in a child process."""
    import shutil
    import subprocess
    import sys
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "fake.c", tmp_path / "fake.so"
    src.write_text(FAKE_DEVICE)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    code = f"""
import ctypes, sys
sys.path.insert(0, {os.path.dirname(os.path.dirname(os.path.abspath(__file__)))!r})
from dropless_token_routing_gb300 import _native as N
L, G, R = N.lib(), 0x10000, ctypes.byref
def decode(dtype):
    d = N.MoeDims(4, 512, 8, 2, 256, 0, 0, dtype, 0, 0)
    p = N.LayerParams(G, None, G, G, None, None)
    return L.moe_layer_decode(R(p), G, None, None, R(d), None, None, G, G, 1 << 40, None)
def linear(dtype, bwd=False):
    d = N.LinearDims(4, 96, 64, 0, dtype, 0, 0, 0, 0)
    if bwd:
        return L.moe_linear_bwd(G, G, None, G, R(d), G, G, G, G, 1 << 40, None)
    return L.moe_linear_fwd(G, G, None, None, R(d), None, G, G, 1 << 40, None)
print({{"decode_bf16": lambda: decode(N.MOE_BF16), "decode_f32": lambda: decode(N.MOE_F32),
       "linear_bf16": lambda: linear(N.MOE_BF16), "linear_f32": lambda: linear(N.MOE_F32),
       "linear_bwd": lambda: linear(N.MOE_BF16, True),
       "verify": lambda: L.moe_verify_draft(G, None, G, G, G, G, R(N.VerifyDims(2, 3, 100, N.MOE_F32, 0, 0)), G, G, None),
      }}[{call!r}]())
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True,
                         env={**os.environ, "LD_PRELOAD": str(so), "CUDA_VISIBLE_DEVICES": ""})
    assert int(out.stdout) == C["MOE_ERR_UNSUPPORTED_DEVICE"], out.stdout


def test_long_strides_are_allowed():
    """The last positions of long sequences lie far apart: 2^36 elements and no more."""
    far = 1 << 36
    for name in ("ld_x", "ld_w", "ld_y", "ld_res"):
        for ld, fits in ((1 << 30, True), (far, True), (far + 1, False), (1 << 62, False)):
            assert (L.moe_linear_workspace_bytes(REF(linear_dims(**{name: ld}))) > 0) == fits, (name, ld)
    null, bad = C["MOE_ERR_NULL_POINTER"], C["MOE_ERR_BAD_DIMS"]
    for name in ("ld_draft", "ld_target"):
        for ld, want in ((1 << 30, null), (far, null), (far + 1, bad), (1 << 62, bad)):
            d = verify_dims(**{name: ld})
            assert L.moe_verify_draft(None, None, GOOD, GOOD, GOOD, GOOD, REF(d), GOOD, GOOD, None) == want, (name, ld)


def test_decode_timeout_probe_is_checked():
    p, d = N.LayerParams(GOOD, None, GOOD, GOOD, None, None), layer_dims()
    n = L.moe_decode_workspace_bytes(REF(d))
    call = L.moe_debug_decode_timeout_probe
    assert call(None, GOOD, REF(d), GOOD, GOOD, n, None) == C["MOE_ERR_NULL_POINTER"]
    assert call(REF(p), BAD, REF(d), GOOD, GOOD, n, None) == C["MOE_ERR_MISALIGNED"]
    assert call(REF(p), GOOD, REF(d), GOOD, GOOD, n - 1, None) == C["MOE_ERR_WORKSPACE_TOO_SMALL"]
    assert call(REF(p), GOOD, REF(layer_dims(T=65)), GOOD, GOOD, n, None) == C["MOE_ERR_BAD_DIMS"]
