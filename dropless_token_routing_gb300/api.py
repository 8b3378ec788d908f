"""Torch-facing wrappers of the C ABI: device memory and streams come from PyTorch,
every computation runs in libmoe's kernels.  Names follow include/moe.h."""
from __future__ import annotations

import contextlib
import ctypes
import weakref
from dataclasses import dataclass
from typing import Optional

import torch

from . import _native as N

__all__ = ["make_dims", "Workspace", "router_logits", "route_topk", "permute", "permute_rows",
           "grouped_swiglu_fwd", "unpermute_combine", "grouped_bwd_dx", "grouped_bwd_dw",
           "route_topk_bwd", "LayerParams", "MoELayer", "get_device_error", "debug_timeout_probe",
           "OpWorkspace", "MoEDecodeLayer", "Linear", "DraftVerifier"]


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _s(stream=None):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _dt(dtype) -> int:
    if dtype in (torch.float32, "f32"):
        return N.MOE_F32
    if dtype in (torch.bfloat16, "bf16"):
        return N.MOE_BF16
    raise ValueError(f"unsupported dtype {dtype}")


def make_dims(T, d, E, k, f, S=0, f_s=0, dtype=torch.bfloat16, capacity=0, rearrange=0) -> N.MoeDims:
    """capacity = 0: dropless; C > 0: drop-and-pad with C rows per expert.
    rearrange (flags) = 0: rearranged copies; 1: rearrangement fused into the GEMM loads;
    2: the second expert GEMM writes its rows in token-major order for the combine; 3: both."""
    return N.MoeDims(int(T), int(d), int(E), int(k), int(f), int(S), int(f_s) if S else 0, _dt(dtype),
                     int(capacity), int(rearrange))


def perm_rows(dims: N.MoeDims) -> int:
    """Rows of the permuted buffers: T*k dropless, E*C with a capacity C."""
    return dims.E * dims.capacity if dims.capacity > 0 else dims.T * dims.k


class Workspace:
    """Device workspace of moe_workspace_bytes(dims) bytes, initialised once."""

    def __init__(self, dims: N.MoeDims, device="cuda", stream=None):
        self.dims = dims
        self.nbytes = int(N.lib().moe_workspace_bytes(ctypes.byref(dims)))
        if self.nbytes == 0:
            raise N.MoeError(N.STATUS_CODE["MOE_ERR_BAD_DIMS"], "moe_workspace_bytes")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.buf.data_ptr()) % 256
        self.ptr = self.buf.data_ptr() + off
        N.check(N.lib().moe_workspace_init(self.ptr, self.nbytes, ctypes.byref(dims), _s(stream)),
                "moe_workspace_init")


def get_device_error(ws: Workspace, stream=None) -> int:
    out = ctypes.c_int(0)
    N.check(N.lib().moe_get_device_error(ws.ptr, _s(stream), ctypes.byref(out)), "moe_get_device_error")
    return out.value


def debug_timeout_probe(ws: Workspace, limit_ns: int, stream=None) -> None:
    N.check(N.lib().moe_debug_timeout_probe(ws.ptr, ws.nbytes, int(limit_ns), _s(stream)),
            "moe_debug_timeout_probe")


def router_logits(x, w_r, dims, logits, ws: Workspace, stream=None):
    N.check(N.lib().moe_router_logits(_p(x), _p(w_r), ctypes.byref(dims), _p(logits), ws.ptr,
                                      ws.nbytes, _s(stream)), "moe_router_logits")


def route_topk(logits, bias, k, topk_idx, topk_w, counts, ws: Workspace, stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_topk(_p(logits), _p(bias), T, E, k, _p(topk_idx), _p(topk_w),
                                   _p(counts), ws.ptr, ws.nbytes, _s(stream)), "moe_route_topk")


def permute(x, topk_idx, topk_w, dims, x_perm, dest, row_src, offsets, w_perm, ws: Workspace,
            stream=None):
    N.check(N.lib().moe_permute(_p(x), _p(topk_idx), _p(topk_w), ctypes.byref(dims), _p(x_perm),
                                _p(dest), _p(row_src), _p(offsets), _p(w_perm), ws.ptr, ws.nbytes,
                                _s(stream)), "moe_permute")


def permute_rows(x, dest, dims, x_perm, stream=None):
    N.check(N.lib().moe_permute_rows(_p(x), _p(dest), ctypes.byref(dims), _p(x_perm), _s(stream)),
            "moe_permute_rows")


def grouped_swiglu_fwd(x_perm, x, w13, w2, ws13, ws2, offsets, dims, z, h, z_sh, h_sh, y_perm, y_sh,
                       ws: Workspace, stream=None):
    N.check(N.lib().moe_grouped_swiglu_fwd(
        _p(x_perm), _p(x), _p(w13), _p(w2), _p(ws13), _p(ws2), _p(offsets), ctypes.byref(dims),
        _p(z), _p(h), _p(z_sh), _p(h_sh), _p(y_perm), _p(y_sh), ws.ptr, ws.nbytes, _s(stream)),
        "moe_grouped_swiglu_fwd")


def unpermute_combine(y_perm, dest, topk_w, y_sh, dims, y, stream=None):
    N.check(N.lib().moe_unpermute_combine(_p(y_perm), _p(dest), _p(topk_w), _p(y_sh),
                                          ctypes.byref(dims), _p(y), _s(stream)),
            "moe_unpermute_combine")


def grouped_bwd_dx(dy_perm, dy, z, z_sh, w13, w2, ws13, ws2, w_perm, offsets, dest, dims, dz, dz_sh,
                   hw, hw_sh, dx_perm, dx_sh, dgate, ws: Workspace, stream=None):
    N.check(N.lib().moe_grouped_bwd_dx(
        _p(dy_perm), _p(dy), _p(z), _p(z_sh), _p(w13), _p(w2), _p(ws13), _p(ws2), _p(w_perm),
        _p(offsets), _p(dest), ctypes.byref(dims), _p(dz), _p(dz_sh), _p(hw), _p(hw_sh),
        _p(dx_perm), _p(dx_sh), _p(dgate), ws.ptr, ws.nbytes, _s(stream)), "moe_grouped_bwd_dx")


def grouped_bwd_dw(x_perm, x, hw, hw_sh, dz, dz_sh, dy_perm, dy, offsets, dims, dw13, dw2, dws13,
                   dws2, ws: Workspace, stream=None):
    N.check(N.lib().moe_grouped_bwd_dw(
        _p(x_perm), _p(x), _p(hw), _p(hw_sh), _p(dz), _p(dz_sh), _p(dy_perm), _p(dy), _p(offsets),
        ctypes.byref(dims), _p(dw13), _p(dw2), _p(dws13), _p(dws2), ws.ptr, ws.nbytes, _s(stream)),
        "moe_grouped_bwd_dw")


def route_topk_bwd(topk_idx, topk_w, dgate, E, dlogits, stream=None):
    T, k = topk_idx.shape
    N.check(N.lib().moe_route_topk_bwd(_p(topk_idx), _p(topk_w), _p(dgate), T, E, k, _p(dlogits),
                                       _s(stream)), "moe_route_topk_bwd")


def route_balance(logits, bias, counts, k, alpha, prob_mean, aux_loss, ws: Workspace, stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_balance(_p(logits), _p(bias), _p(counts), T, E, k, float(alpha),
                                      _p(prob_mean), _p(aux_loss), ws.ptr, ws.nbytes, _s(stream)),
            "moe_route_balance")


def route_topk_balance(logits, bias, k, alpha, topk_idx, topk_w, counts, prob_mean, aux_loss, ws: Workspace,
                       stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_topk_balance(_p(logits), _p(bias), T, E, k, float(alpha), _p(topk_idx),
                                           _p(topk_w), _p(counts), _p(prob_mean), _p(aux_loss), ws.ptr,
                                           ws.nbytes, _s(stream)), "moe_route_topk_balance")


def route_balance_bwd(logits, bias, counts, k, alpha, grad, dlogits, stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_balance_bwd(_p(logits), _p(bias), _p(counts), T, E, k, float(alpha),
                                          float(grad), _p(dlogits), _s(stream)),
            "moe_route_balance_bwd")


def route_balance_seq(logits, bias, topk_idx, k, group_len, alpha, prob_mean, counts, aux_loss,
                      ws: Workspace, stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_balance_seq(_p(logits), _p(bias), _p(topk_idx), T, E, k, int(group_len),
                                          float(alpha), _p(prob_mean), _p(counts), _p(aux_loss), ws.ptr,
                                          ws.nbytes, _s(stream)), "moe_route_balance_seq")


def route_balance_seq_bwd(logits, bias, counts, k, group_len, n_groups, alpha, grad, dlogits, stream=None):
    T, E = logits.shape
    N.check(N.lib().moe_route_balance_seq_bwd(_p(logits), _p(bias), _p(counts), T, E, k, int(group_len),
                                              int(n_groups), float(alpha), float(grad), _p(dlogits),
                                              _s(stream)), "moe_route_balance_seq_bwd")


@dataclass
class LayerParams:
    w13: torch.Tensor
    w2: torch.Tensor
    w_r: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    ws13: Optional[torch.Tensor] = None
    ws2: Optional[torch.Tensor] = None

    def c(self) -> N.LayerParams:
        return N.LayerParams(_p(self.w_r), _p(self.bias), _p(self.w13), _p(self.w2), _p(self.ws13),
                             _p(self.ws2))


class MoELayer:
    """One dropless MoE layer: caller-owned saved activations, gradients and workspace.

    ``forward(x, logits_in=None)`` runs moe_layer_fwd; ``backward(dy)`` runs
    moe_layer_bwd on the values the last forward saved. ``recompute=True`` keeps neither
    the rearranged input nor h between the two (selective recompute). ``capacity=C > 0``
    runs the drop-and-pad variant with C rows per expert instead of the dropless layer;
    ``rearrange=1`` fuses the rearrangement into the GEMMs' operand loads, ``rearrange=2`` the
    un-rearrangement into the second GEMM's stores (token-major rows), 3 both.
    """

    def __init__(self, params: LayerParams, T, d, E, k, f, S=0, f_s=0, dtype=torch.bfloat16,
                 device="cuda", logits_input=False, recompute=False, capacity=0, rearrange=0):
        self.params = params
        self.dims = make_dims(T, d, E, k, f, S, f_s, dtype, capacity, rearrange)
        self.T, self.d, self.E, self.k, self.f, self.S, self.f_s = T, d, E, k, f, S, f_s
        self.dtype = dtype
        Tk = T * k
        R = perm_rows(self.dims)
        dev = device
        emp = lambda *shape, dt=dtype: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        self.ws = Workspace(self.dims, device=dev)
        self.saved = dict(
            logits=None if logits_input else emp(T, E, dt=torch.float32),
            topk_idx=emp(T, k, dt=torch.int32), topk_w=emp(T, k, dt=torch.float32),
            counts=emp(E, dt=torch.int32), offsets=emp(E + 1, dt=torch.int32),
            dest=emp(Tk, dt=torch.int32), row_src=emp(R, dt=torch.int32),
            w_perm=emp(R, dt=torch.float32), x_perm=None if recompute else emp(R, d),
            z=emp(R, 2 * f), h=None if recompute else emp(R, f),
            z_sh=emp(S * T, 2 * f_s) if S else None,
            h_sh=emp(S * T, f_s) if (S and not recompute) else None)
        self.y = emp(T, d)
        self.grads = None
        self._x = None

    def _saved_c(self):
        s = self.saved
        return N.LayerSaved(*[_p(s[n]) for n in ("logits", "topk_idx", "topk_w", "counts", "offsets",
                                                  "dest", "row_src", "w_perm", "x_perm", "z", "h",
                                                  "z_sh", "h_sh")])

    def alloc_grads(self, with_dlogits=None):
        T, d, E, f, S, f_s = self.T, self.d, self.E, self.f, self.S, self.f_s
        dev, dt = self.y.device, self.dtype
        want_dl = (self.params.w_r is None) if with_dlogits is None else with_dlogits
        self.grads = dict(
            dx=torch.empty(T, d, dtype=dt, device=dev),
            dw13=torch.empty(E, 2 * f, d, dtype=dt, device=dev),
            dw2=torch.empty(E, d, f, dtype=dt, device=dev),
            dws13=torch.empty(S, 2 * f_s, d, dtype=dt, device=dev) if S else None,
            dws2=torch.empty(S, d, f_s, dtype=dt, device=dev) if S else None,
            dw_r=torch.empty(d, E, dtype=torch.float32, device=dev) if self.params.w_r is not None else None,
            dlogits=torch.empty(T, E, dtype=torch.float32, device=dev) if want_dl else None)
        return self.grads

    def forward(self, x, logits_in=None, stream=None):
        self._x = x
        pc, sc = self.params.c(), self._saved_c()
        N.check(N.lib().moe_layer_fwd(ctypes.byref(pc), _p(x), _p(logits_in), ctypes.byref(self.dims),
                                      ctypes.byref(sc), _p(self.y), self.ws.ptr, self.ws.nbytes,
                                      _s(stream)), "moe_layer_fwd")
        return self.y

    def backward(self, dy, x=None, stream=None):
        if self.grads is None:
            self.alloc_grads()
        x = self._x if x is None else x
        g = self.grads
        gc = N.LayerGrads(*[_p(g[n]) for n in ("dx", "dw13", "dw2", "dws13", "dws2", "dw_r", "dlogits")])
        pc, sc = self.params.c(), self._saved_c()
        N.check(N.lib().moe_layer_bwd(ctypes.byref(pc), ctypes.byref(sc), _p(x), _p(dy),
                                      ctypes.byref(self.dims), ctypes.byref(gc), self.ws.ptr,
                                      self.ws.nbytes, _s(stream)), "moe_layer_bwd")
        return g


# ------------------------------------------------------------------ few-token operators
def _on(stream, device):
    """Memory made inside is the given stream's: what the allocator has of the current stream's may
    still be read there."""
    return torch.cuda.stream(stream) if stream is not None and device.type == "cuda" else contextlib.nullcontext()


class OpWorkspace:
    """Device workspace of a few-token operator: its header is zeroed once, here."""

    def __init__(self, nbytes: int, call: str, device="cuda", stream=None):
        if nbytes == 0:
            raise N.MoeError(N.STATUS_CODE["MOE_ERR_BAD_DIMS"], call)
        self.nbytes = int(nbytes)
        with _on(stream, torch.device(device)):
            self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        self.ptr = self.buf.data_ptr() + (-self.buf.data_ptr()) % 256
        N.check(N.lib().moe_op_workspace_init(self.ptr, self.nbytes, _s(stream)), "moe_op_workspace_init")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device_index):
    """The stream's handle; the current one's without making a Stream object where torch can."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(device_index) if _raw_stream is not None else torch.cuda.current_stream(device_index).cuda_stream


def _refuse(name, dtype, shape, t):
    raise ValueError(f"{name}: expected contiguous {list(shape)} of {dtype}, got {list(t.shape)} of {t.dtype}, "
                     f"strides {t.stride()}")


def _elsewhere(name, device, t):
    raise ValueError(f"{name}: expected on device {device}, got {t.device}")


def _matrix(t, name, dtype, rows, cols, device):
    """Checks a [rows, cols] operand with contiguous rows that do not overlap (an expanded one is
    no matrix: the library takes stride 0 for the default); returns the stride between them."""
    if t.dtype != dtype or t.shape != (rows, cols):
        raise ValueError(f"{name}: expected [{rows}, {cols}] of {dtype}, got {list(t.shape)} of {t.dtype}")
    if t.device != device:
        _elsewhere(name, device, t)
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if ld < cols:
        if rows > 1:
            raise ValueError(f"{name}: rows of {cols} elements are {ld} apart (expanded? make it contiguous)")
        return cols
    return ld if rows > 1 else min(ld, cols + 7 & ~7)   # one row: whole vectors, if there is room for them


def _overlap(a, ld_a, b, ld_b):
    """Whether two matrices of contiguous rows, ld_a and ld_b elements apart, share an element."""
    (Ma, ca), (Mb, cb), size = a.shape, b.shape, a.element_size()
    if a.numel() == 0 or b.numel() == 0:
        return False
    d = b.data_ptr() - a.data_ptr()
    ca, cb, la, lb = ca * size, cb * size, ld_a * size, ld_b * size
    if (Ma - 1) * la + ca <= d or d + (Mb - 1) * lb + cb <= 0:
        return False
    if la == lb or Ma == 1 or Mb == 1:
        # rows i of a and j of b meet where (i - j) l lies above d - ca and below d + cb
        step = la if Mb == 1 else lb
        return max((d - ca) // step + 1, 1 - Mb) <= min(-(-(d + cb) // step) - 1, Ma - 1)
    # the last row of b that starts before a row of a ends is the one that reaches furthest
    start = torch.arange(Ma) * la
    j = ((start + ca - d - 1) // lb).clamp(max=Mb - 1)
    return bool(((j >= 0) & (j * lb + d + cb > start)).any())


def _dense(t, name, dtype, shape, device):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, dtype, shape, t)
    if t.device != device:
        _elsewhere(name, device, t)


def _device(device):
    """The device as its tensors name it, and its index."""
    d = torch.empty(0, device=device).device
    return d, d.index if d.index is not None else 0


def _none():
    return None


def _ref(t):
    """Calls to the tensor, while it exists, or None."""
    return _none if t is None else weakref.ref(t)


def _same(t, ref, ptr):
    """t is the tensor that `ref` stands for, and lies where it did (a freed one's ref gives None too)."""
    return t is ref() and (t.data_ptr() if t is not None else None) == ptr


class MoEDecodeLayer:
    """The whole MoE layer for a few tokens: moe_layer_decode on a kept workspace.

    ``forward(x, residual=None)`` takes 0 to ``max_tokens`` (at most 64) tokens and returns
    y [T, d], the layer's own buffer (overwritten by the next call) unless ``out`` is given
    (x and residual are allowed, a residual that only partly overlaps it is not). ``topk_idx`` and
    ``topk_w`` hold the last call's selection. Every call takes the weights that ``params`` holds
    then (a captured graph those of the capture). One instance serves one stream at a time, which
    waits for the one it was made on.
    """

    def __init__(self, params: LayerParams, max_tokens, d, E, k, f, S=0, f_s=0, dtype=torch.bfloat16,
                 device="cuda", stream=None):
        self.params, self.dtype, self.max_tokens, self.d, self.E, self.k = params, dtype, max_tokens, d, E, k
        self.dims = make_dims(max_tokens, d, E, k, f, S, f_s, dtype)
        self.device, self._index = _device(device)
        self._weights = (("w13", dtype, E * 2 * f * d), ("w2", dtype, E * d * f), ("w_r", torch.float32, d * E),
                         ("bias", torch.float32, E)) + (
            (("ws13", dtype, S * 2 * f_s * d), ("ws2", dtype, S * d * f_s)) if S else ())
        self._row = d * torch.empty(0, dtype=dtype).element_size()   # bytes
        self._c = N.LayerParams()
        self._bind()
        self.ws = OpWorkspace(N.lib().moe_decode_workspace_bytes(ctypes.byref(self.dims)), "moe_decode_workspace_bytes",
                              device, stream)
        self._idx = torch.empty(max_tokens, k, dtype=torch.int32, device=device)
        self._w = torch.empty(max_tokens, k, dtype=torch.float32, device=device)
        self._y = torch.empty(max_tokens, d, dtype=dtype, device=device)
        self._views = {}            # y's first T rows
        self._call = N.lib().moe_layer_decode
        self._refs = (ctypes.byref(self._c), ctypes.byref(self.dims), self._idx.data_ptr(), self._w.data_ptr())
        self._T = 0

    def _present(self):
        p = self.params
        for name, ref, ptr in self._bound:
            t = getattr(p, name)
            if t is not ref() or (t.data_ptr() if t is not None else None) != ptr:
                return False
        return True

    def _bind(self):
        """Takes the weights that params holds; those that are there have the layer's type, size and
        device (any shape of them)."""
        p, c = self.params, self._c
        self._bound = (("w13", lambda: self, 0),)      # none of them, should a check fail
        for name, dtype, n in self._weights:
            t = getattr(self.params, name)
            if t is not None and (t.dtype != dtype or t.numel() != n or not t.is_contiguous()):
                raise ValueError(f"{name}: expected {n} contiguous elements of {dtype}, got {list(t.shape)} of {t.dtype}, "
                                 f"strides {t.stride()}")
            if t is not None and t.device != self.device:
                _elsewhere(name, self.device, t)
        for name, _ in c._fields_:
            setattr(c, name, _p(getattr(p, name)))
        self._bound = tuple((name, _ref(getattr(p, name)), getattr(c, name)) for name, _, _ in self._weights)

    @property
    def topk_idx(self):
        return self._idx[:self._T]

    @property
    def topk_w(self):
        return self._w[:self._T]

    def forward(self, x, residual=None, logits_in=None, out=None, stream=None):
        T, dev = x.shape[0], self.device
        shape = (T, self.d)
        if T > self.max_tokens:
            raise ValueError(f"x: {T} tokens, the layer was made for {self.max_tokens}")
        _dense(x, "x", self.dtype, shape, dev)
        if residual is not None:
            _dense(residual, "residual", self.dtype, shape, dev)
        if logits_in is not None:
            _dense(logits_in, "logits_in", torch.float32, (T, self.E), dev)
        if out is None:
            v = self._views.get(T)
            if v is None:
                v = self._views[T] = self._y[:T], self._y.data_ptr()
            out, yp = v
        else:
            _dense(out, "out", self.dtype, shape, dev)
            yp = out.data_ptr()
        if not self._present():
            self._bind()
        rp = None if residual is None else residual.data_ptr()
        if rp is not None and rp != yp and abs(rp - yp) < T * self._row:
            raise ValueError("residual: overlaps the output and does not lie where it does")
        self._T = self.dims.T = T
        c, dims, idx, w = self._refs
        st = self._call(c, x.data_ptr(), None if logits_in is None else logits_in.data_ptr(),
                        rp, dims, idx, w, yp, self.ws.ptr, self.ws.nbytes, _stream(stream, self._index))
        if st:
            N.check(st, "moe_layer_decode")
        return out


class Linear:
    """y = act(x W^T + b) + residual and its gradients: moe_linear_fwd / moe_linear_bwd on a kept
    workspace for up to ``max_rows`` rows. ``w`` [N, K] may have strided rows; every call takes the
    ``w`` and ``bias`` that the layer holds then.

    ``forward(x, residual=None, save=False)`` returns y [M, N], the layer's own buffer
    (written by the next call, which may therefore not read it: a result that goes through the
    layer again needs another ``out``) unless ``out`` is given; with ``save=True`` it keeps x and the
    pre-activation for ``backward(dy)``, which returns dict(dx, dw, db) (own buffers too; ``need``
    names those to compute). The residual's gradient is dy itself. ``out`` may be the residual. One
    instance serves one stream at a time, which waits for the one it was made on.
    """

    def __init__(self, w, bias=None, act="none", max_rows=1, device=None, stream=None):
        self.w, self.bias, self.dtype, self.max_rows = w, bias, w.dtype, max_rows
        self.N, self.K = w.shape
        self.act, self._size = N.ACTS[act], w.element_size()
        dev, self._index = _device(device if device is not None else w.device)
        self.device = dev
        self.dims = N.LinearDims(int(max_rows), self.N, self.K, self.act, _dt(w.dtype), 0, 0, 0, 0)
        self._workspaces, self.ws = [], None   # one that a wider W has outgrown may still be in use
        self._bind(stream)
        self._x = None
        self._bufs, self._views = {}, {}
        self._dims_ref = ctypes.byref(self.dims)
        self._fwd, self._bwd = N.lib().moe_linear_fwd, N.lib().moe_linear_bwd

    def _bind(self, stream):
        """Takes the present w and bias; bf16 rows of w that are not whole vectors need a larger workspace."""
        w, bias, D = self.w, self.bias, self.dims
        self._w_ref = lambda: None      # nothing, should a check fail
        ld_w = _matrix(w, "w", self.dtype, self.N, self.K, self.device)
        if bias is not None:
            _dense(bias, "bias", self.dtype, (self.N,), self.device)
        most = N.LinearDims(int(self.max_rows), self.N, self.K, self.act, D.dtype, 0, ld_w, 0, 0)
        need = N.lib().moe_linear_workspace_bytes(ctypes.byref(most))
        if self.ws is None or self.ws.nbytes < need:
            self.ws = OpWorkspace(need, "moe_linear_workspace_bytes", self.device, stream)
            self._workspaces.append(self.ws)
        D.ld_w = ld_w
        self._w_ptr, self._b_ptr = w.data_ptr(), _p(bias)
        self._w_ref, self._b_ref = _ref(w), _ref(bias)

    def _own(self, name, rows, cols, stream):
        """The layer's buffer ``name``, made at its first use, of the call's stream."""
        t = self._bufs.get(name)
        if t is None:
            with _on(stream, self.device):
                t = self._bufs[name] = torch.empty(rows, cols, dtype=self.dtype, device=self.device)
        return t

    def _view(self, name, rows, cols, M, width, stream):
        """[M, width] of the buffer ``name`` [rows, cols], and its address."""
        key = (name, M, width)
        v = self._views.get(key)
        if v is None:
            t = self._own(name, rows, cols, stream)[:M, :width]
            v = self._views[key] = t, t.data_ptr()
        return v

    def forward(self, x, residual=None, save=False, out=None, stream=None):
        M, D, dev, dtype, n, size = x.shape[0], self.dims, self.device, self.dtype, self.N, self._size
        if M > self.max_rows:
            raise ValueError(f"{M} rows, the layer was made for {self.max_rows}")
        ld_x, xp = _matrix(x, "x", dtype, M, self.K, dev), x.data_ptr()
        if out is None:
            y, yp = self._view("y", self.max_rows, n, M, n, stream)
            ld_y = n
        else:
            y, yp, ld_y = out, out.data_ptr(), _matrix(out, "out", dtype, M, n, dev)
        if not (_same(self.w, self._w_ref, self._w_ptr) and _same(self.bias, self._b_ref, self._b_ptr)):
            self._bind(stream)
        # what is read may not lie where y is written, but for a residual in the same place
        end = yp + M * ld_y * size
        if xp < end and yp < xp + M * ld_x * size and _overlap(x, ld_x, y, ld_y):
            raise ValueError("x: overlaps the output (a result of this layer? give it another out)")
        if residual is None:
            rp, ld_r = None, 0
        else:
            rp, ld_r = residual.data_ptr(), _matrix(residual, "residual", dtype, M, n, dev)
            if rp < end and yp < rp + M * ld_r * size and not (
                    rp == yp and (ld_r == ld_y or M == 1)) and _overlap(residual, ld_r, y, ld_y):
                raise ValueError("residual: overlaps the output and does not lie where it does")
        if out is not None and (_overlap(self.w, D.ld_w, y, ld_y) or
                                (self.bias is not None and _overlap(self.bias[None], n, y, ld_y))):
            raise ValueError("out: overlaps the layer's weights")
        z = self._own("z", self.max_rows, n + 7 & ~7, stream).data_ptr() if save and self.act != 0 else None
        self._x = x if save else None
        D.M, D.ld_x, D.ld_y, D.ld_res = M, ld_x, ld_y, ld_r
        st = self._fwd(xp, self._w_ptr, self._b_ptr, rp, self._dims_ref, z, yp, self.ws.ptr, self.ws.nbytes,
                       _stream(stream, self._index))
        if st:
            N.check(st, "moe_linear_fwd")
        return y

    def backward(self, dy, need=("dx", "dw", "db"), stream=None):
        x, D, n, size = self._x, self.dims, self.N, self._size
        if x is None:
            raise ValueError("backward: the last forward did not save (save=True)")
        M = x.shape[0]
        if not (_same(self.w, self._w_ref, self._w_ptr) and _same(self.bias, self._b_ref, self._b_ptr)):
            self._bind(stream)
        ld_x, xp, ld_w = _matrix(x, "x", self.dtype, M, self.K, self.device), x.data_ptr(), D.ld_w
        ld_y, yp = _matrix(dy, "dy", self.dtype, M, n, self.device), dy.data_ptr()
        dx = dw = db = dxp = dwp = dbp = None
        # a call takes one distance for the rows of x and dx: where x's rows lie far apart (slices of
        # something larger) dx is a call of its own, in dense rows. That repeats the pass over dz, if there
        # is one (4096 x 2816 x 2048 with GELU: 107 us, 89 in one call; without an activation both 76), so
        # columns of a buffer up to eight times as wide stay in one call
        ld_dx = ld_x if ld_x <= 8 * self.K else self.K
        if "dx" in need:
            dx, dxp = self._view(("dx", ld_dx), self.max_rows, ld_dx, M, self.K, stream)
        if "dw" in need:
            dw, dwp = self._view(("dw", ld_w), n, ld_w, n, self.K, stream)
        if "db" in need and self.bias is not None:
            db, dbp = self._view("db", 1, n, 1, n, stream)
        # dw's product reads x and dz last; dz is dy itself where it is not made first
        own_dz = self.act != 0 or (size == 2 and ld_y % 8 != 0)
        for o, op, rows, ld_o in ((dx, dxp, M, ld_dx), (dw, dwp, n, ld_w), (db, dbp, 1, n)):
            if o is None:
                continue
            end = op + rows * ld_o * size
            if (not own_dz and yp < end and op < yp + M * ld_y * size and _overlap(dy, ld_y, o, ld_o)) or (
                    dw is not None and xp < end and op < xp + M * ld_x * size and _overlap(x, ld_x, o, ld_o)):
                raise ValueError("dy or x: overlaps a result of this layer that is written before it is read (pass a copy)")
        z = self._own("z", self.max_rows, n + 7 & ~7, stream).data_ptr() if self.act != 0 else None
        D.M, D.ld_y, D.ld_res = M, ld_y, 0
        parts = ((ld_x, dxp, dwp, dbp),)
        if ld_dx != ld_x and dx is not None:
            parts = ((ld_dx, dxp, None, None),) + (((ld_x, None, dwp, dbp),) if dw is not None or db is not None else ())
        for D.ld_x, dxp, dwp, dbp in parts:
            st = self._bwd(xp, self._w_ptr, z, yp, self._dims_ref, dxp, dwp, dbp, self.ws.ptr, self.ws.nbytes,
                           _stream(stream, self._index))
            if st:
                N.check(st, "moe_linear_bwd")
        return dict(dx=dx, dw=dw, db=None if db is None else db[0])


class DraftVerifier:
    """Verification of drafted tokens (moe_verify_draft) for up to ``max_batch`` sequences of
    ``n`` drafted tokens each; returns (tokens [B, n+1], accepted [B]), own buffers."""

    def __init__(self, max_batch, n, V, dtype=torch.float32, device="cuda"):
        self.max_batch, self.n, self.V, self.dtype = max_batch, n, V, dtype
        self.dims = N.VerifyDims(0, n, V, _dt(dtype), 0, 0)
        self._tokens = torch.empty(max_batch, n + 1, dtype=torch.int32, device=device)
        self._accepted = torch.empty(max_batch, dtype=torch.int32, device=device)
        self._views = {}
        self._ptrs = self._tokens.data_ptr(), self._accepted.data_ptr()
        self.device, self._index = _device(device)
        self._call, self._dims_ref = N.lib().moe_verify_draft, ctypes.byref(self.dims)

    def _rows(self, t, name, B, rows):
        """Checks probabilities [B, rows, V] whose rows are contiguous and evenly spaced; returns their distance."""
        if t.dtype != self.dtype or t.shape != (B, rows, self.V):
            raise ValueError(f"{name}: expected [{B}, {rows}, {self.V}] of {self.dtype}, got {list(t.shape)} of {t.dtype}")
        if t.device != self.device:
            _elsewhere(name, self.device, t)
        s0, s1, s2 = t.stride()
        ld = s1 if rows > 1 else (s0 if B > 1 else self.V)
        if (self.V > 1 and s2 != 1) or (B > 1 and rows > 0 and s0 != rows * ld) or ld < self.V:
            raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
        return ld

    def verify(self, draft_tokens, draft_probs, target_probs, u_accept, u_sample, draft_len=None, stream=None):
        B, n, dev, dt = draft_tokens.shape[0], self.n, self.device, self.dtype
        v = self._views.get(B)
        if v is None:
            if B > self.max_batch:
                raise ValueError(f"{B} sequences, made for {self.max_batch}")
            v = self._views[B] = ((self._tokens[:B], self._accepted[:B]), (B, n), (B,), (B, n, self.V), (B, n + 1, self.V))
        out, of_tokens, of_rows, of_q, of_p = v
        # (checked here, and said there: a call's host time is near the kernel's own for one sequence)
        t = draft_tokens
        if t.dtype is not torch.int32 or t.shape != of_tokens or not t.is_contiguous() or t.device != dev:
            _dense(t, "draft_tokens", torch.int32, of_tokens, dev)
        t = u_accept
        if t.dtype is not torch.float32 or t.shape != of_tokens or not t.is_contiguous() or t.device != dev:
            _dense(t, "u_accept", torch.float32, of_tokens, dev)
        t = u_sample
        if t.dtype is not torch.float32 or t.shape != of_rows or not t.is_contiguous() or t.device != dev:
            _dense(t, "u_sample", torch.float32, of_rows, dev)
        ld_q = ld_p = self.V
        t = draft_probs
        if t.dtype is not dt or t.shape != of_q or not t.is_contiguous() or t.device != dev:
            ld_q = self._rows(t, "draft_probs", B, n)
        t = target_probs
        if t.dtype is not dt or t.shape != of_p or not t.is_contiguous() or t.device != dev:
            ld_p = self._rows(t, "target_probs", B, n + 1)
        # a result is written while other sequences, and later tokens of its own, are read
        dp, (tp, ap) = draft_tokens.data_ptr(), self._ptrs
        if dp < tp + B * (n + 1) * 4 and tp < dp + B * n * 4 and not (B == 1 and dp == tp):
            raise ValueError("draft_tokens: overlaps the result")
        lp = None
        if draft_len is not None:
            _dense(draft_len, "draft_len", torch.int32, of_rows, dev)
            lp = draft_len.data_ptr()
            if lp != ap and abs(lp - ap) < B * 4:
                raise ValueError("draft_len: overlaps the result and does not lie where it does")
        D = self.dims
        D.B, D.ld_draft, D.ld_target = B, ld_q, ld_p
        st = self._call(dp, lp, draft_probs.data_ptr(), target_probs.data_ptr(), u_accept.data_ptr(), u_sample.data_ptr(),
                        self._dims_ref, tp, ap, _stream(stream, self._index))
        if st:
            N.check(st, "moe_verify_draft")
        return out
