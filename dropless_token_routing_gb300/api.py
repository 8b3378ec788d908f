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
           "OpWorkspace", "MoEDecodeLayer", "Linear", "DraftVerifier", "LayerNorm", "TokenLogprobs", "GradClipper"]


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


def _unchanged(*tensors):
    """Says of the same tensors later on, all in one call, whether types, shapes and strides are the present ones: the
    address alone does not, as the memory there may be another tensor's by then, or the same one's in another order.
    It may say no where none of these has changed (a tensor now requires its gradient, another mode)."""
    try:
        return torch._C._dynamo.guards.TensorGuards(
            *tensors, dynamic_dims_sizes=[list(t.shape) for t in tensors],
            dynamic_dims_strides=[list(t.stride()) for t in tensors]).check
    except Exception:       # (none, or another form of it)
        were = [(t.dtype, t.shape, t.stride()) for t in tensors]
        return lambda *tensors: [(t.dtype, t.shape, t.stride()) for t in tensors] == were


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
        p, there = self.params, []
        for name, ref, ptr in self._bound:
            t = getattr(p, name)
            if t is not ref() or (t.data_ptr() if t is not None else None) != ptr:
                return False
            if t is not None:
                there.append(t)
        return self._like(*there)

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
        there = [getattr(p, name) for name, _, _ in self._weights]
        self._like = _unchanged(*[t for t in there if t is not None])
        self._bound = tuple((name, _ref(t), getattr(c, name)) for (name, _, _), t in zip(self._weights, there))

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
        self._like = _unchanged(w) if bias is None else _unchanged(w, bias)
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
        if not (_same(self.w, self._w_ref, self._w_ptr) and _same(self.bias, self._b_ref, self._b_ptr) and
                (self._like(self.w) if self.bias is None else self._like(self.w, self.bias))):
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
        if not (_same(self.w, self._w_ref, self._w_ptr) and _same(self.bias, self._b_ref, self._b_ptr) and
                (self._like(self.w) if self.bias is None else self._like(self.w, self.bias))):
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


# ------------------------------------------------------------------ around the layer in training
def _in_place(name, t, ld, out, ld_out, what):
    """Refuses an operand that overlaps a result unless it lies just where that does."""
    M = t.shape[0]
    if t.data_ptr() == out.data_ptr() and (ld == ld_out or M == 1):
        return
    if _overlap(t, ld, out, ld_out):
        raise ValueError(f"{name}: overlaps {what} and does not lie where it does")


_KEPT_VIEWS = 1024      # of results and shapes, one for each number of rows that came up


class LayerNorm:
    """y = (s - mean) rstd weight + bias with s = x + residual, and its gradients: moe_norm_fwd /
    moe_norm_bwd on kept buffers for up to ``max_rows`` rows. ``dtype`` is the rows' (default the
    weight's; bf16 rows may have fp32 weights). Every call takes the ``weight`` and ``bias`` that the
    layer holds then.

    ``forward(x, residual=None, save=False)`` returns y [M, N], or (y, s) with a residual: the layer's own
    buffers (written by the next call) unless ``out`` and ``sum_out`` are given, which may be x or the
    residual. With ``save=True`` it keeps what was normed (unchanged until then) for
    ``backward(dy, d_sum=None)``, which returns dict(dx, dw, db) (own buffers too; ``need`` names those to
    compute; ``out`` takes dx and may be dy, d_sum or what was kept, which is then gone). d_sum is the gradient of s by its other
    way; dx is the gradient of x and of the residual. What is kept is x and, in bf16, the residual: the
    rounding of s would show in the gradient of the weight. It is s for fp32 rows (the one returned), and where a result
    has taken the place of x or the residual. Rows may be any distance apart; tensors begin on 16 bytes. Own buffers are
    returned as the same tensors for the same number of rows. One instance serves one stream at a time, which waits
    for the one it was made on.
    """

    def __init__(self, weight, bias=None, eps=1e-5, max_rows=1, dtype=None, device=None, stream=None):
        self.weight, self.bias, self.eps, self.max_rows = weight, bias, eps, max_rows
        self.dtype, self.w_dtype = dtype if dtype is not None else weight.dtype, weight.dtype
        (self.N,) = weight.shape
        self.device, self._index = _device(device if device is not None else weight.device)
        self._size, self._w_size = (torch.empty(0, dtype=t).element_size() for t in (self.dtype, self.w_dtype))
        # one for each direction: a call sets what has changed since its last one
        self.dims, self._bwd_dims = (N.NormDims(int(max_rows), self.N, _dt(self.dtype), _dt(self.w_dtype), eps, 0, 0, 0, 0, 0)
                                     for _ in range(2))
        self._set, self._bwd_set = None, None
        self._bufs, self._views, self._shapes, self._kept = {}, {}, {}, None
        self._bind()
        self._need = N.lib().moe_norm_workspace_bytes(ctypes.byref(self.dims))
        if self._need == 0:
            raise N.MoeError(N.STATUS_CODE["MOE_ERR_BAD_DIMS"], "moe_norm_workspace_bytes")
        self.ws = None
        self._dims_ref, self._bwd_ref = ctypes.byref(self.dims), ctypes.byref(self._bwd_dims)
        self._fwd, self._bwd = N.lib().moe_norm_fwd, N.lib().moe_norm_bwd

    def _bind(self):
        self._w_ref = lambda: self      # none of them, should a check fail
        _dense(self.weight, "weight", self.w_dtype, (self.N,), self.device)
        if self.bias is not None:
            _dense(self.bias, "bias", self.w_dtype, (self.N,), self.device)
        for name, t in (("weight", self.weight), ("bias", self.bias)):
            for buf in self._bufs.values():     # (those made later are other memory)
                if t is not None and buf.numel() and _bytes_meet(buf.view(1, -1), 0, t):
                    raise ValueError(f"{name}: lies in a result of this layer (pass a copy)")
        self._w_ptr, self._b_ptr = self.weight.data_ptr(), _p(self.bias)
        self._like = _unchanged(self.weight) if self.bias is None else _unchanged(self.weight, self.bias)
        self._w_ref, self._b_ref = _ref(self.weight), _ref(self.bias)

    def _view(self, name, M, stream):
        """The first M rows of the layer's buffer ``name`` (all of it: None), made at its first use, of the
        call's stream, and its address."""
        t = self._bufs.get(name)
        if t is None:
            shape, dt = {"stats": ((self.max_rows, 2), torch.float32), "dw": ((self.N,), self.w_dtype),
                         "db": ((self.N,), self.w_dtype)}.get(name, ((self.max_rows, self.N), self.dtype))
            with _on(stream, self.device):
                t = self._bufs[name] = torch.empty(shape, dtype=dt, device=self.device)
        if len(self._views) >= _KEPT_VIEWS:
            self._views.clear()
        v = self._views[(name, M)] = t if M is None else t[:M], t.data_ptr()
        return v

    def _shape(self, M):
        if M > self.max_rows:
            raise ValueError(f"{M} rows, the layer was made for {self.max_rows}")
        if len(self._shapes) >= _KEPT_VIEWS:
            self._shapes.clear()
        s = self._shapes[M] = torch.Size((M, self.N))
        return s

    def _given(self, name, t, M):
        """Checks a result's place that the caller gives; returns the stride between its rows."""
        ld = _matrix(t, name, self.dtype, M, self.N, self.device)
        for wname, w in (("weight", self.weight), ("bias", self.bias)):
            if w is not None and M and _bytes_meet(t, ld, w):
                raise ValueError(f"{name}: overlaps the layer's {wname}")
        return ld

    def forward(self, x, residual=None, save=False, out=None, sum_out=None, stream=None):
        M, n, dev, dt, views = x.shape[0], self.N, self.device, self.dtype, self._views
        # (checked here, and said there: a call's host time is near the kernel's own for one row)
        shape = self._shapes.get(M) or self._shape(M)
        ld_x = n if x.dtype is dt and x.shape == shape and x.is_contiguous() and x.device == dev else _matrix(x, "x", dt, M, n, dev)
        w, b = self.weight, self.bias
        if w is not self._w_ref() or b is not self._b_ref() or w.data_ptr() != self._w_ptr or (
                not self._like(w) if b is None else b.data_ptr() != self._b_ptr or not self._like(w, b)):
            self._bind()
        xp, row = x.data_ptr(), M * self._size     # (row times a stride: the span of rows that far apart)
        if out is None:
            y, yp = views.get(("y", M)) or self._view("y", M, stream)
            ld_y = n
        else:
            y, yp, ld_y = out, out.data_ptr(), self._given("out", out, M)
        if -row * ld_x < xp - yp < row * ld_y:
            _in_place("x", x, ld_x, y, ld_y, "the output")
        sp = rp = stats = None
        ld_s = ld_r = 0
        if residual is not None:
            r = residual
            ld_r = n if r.dtype is dt and r.shape == shape and r.is_contiguous() and r.device == dev else _matrix(r, "residual", dt, M, n, dev)
            rp = r.data_ptr()
            if sum_out is None:
                s, sp = views.get(("sum", M)) or self._view("sum", M, stream)
                ld_s = n
            else:
                s, sp, ld_s = sum_out, sum_out.data_ptr(), self._given("sum_out", sum_out, M)
            if -row * ld_r < rp - yp < row * ld_y:
                _in_place("residual", r, ld_r, y, ld_y, "the output")
            if -row * ld_r < rp - sp < row * ld_s:
                _in_place("residual", r, ld_r, s, ld_s, "the sum")
            if -row * ld_x < xp - sp < row * ld_s:
                _in_place("x", x, ld_x, s, ld_s, "the sum")
            if (out is not None or sum_out is not None) and _overlap(y, ld_y, s, ld_s):
                raise ValueError("out: overlaps the sum")
        elif sum_out is not None:
            raise ValueError("sum_out: there is no residual to add")
        elif save and yp == xp and M:
            raise ValueError("out: x is needed for the backward")
        self._kept = None
        if save:
            stats = (views.get(("stats", M)) or self._view("stats", M, stream))[1]
            if rp is None:
                self._kept = x, xp, ld_x, None, None, 0
            elif self._size == 2 and xp != sp and xp != yp and rp != sp and rp != yp:
                self._kept = x, xp, ld_x, residual, rp, ld_r
            else:
                self._kept = s, sp, ld_s, None, None, 0
        key = M, ld_x, ld_r, ld_s, ld_y
        if key != self._set:
            D = self.dims
            D.M, D.ld_x, D.ld_res, D.ld_sum, D.ld_y = self._set = key
        st = self._fwd(xp, rp, self._w_ptr, self._b_ptr, self._dims_ref, sp, yp, stats,
                       _raw_stream(self._index) if stream is None and _raw_stream is not None else _stream(stream, self._index))
        if st:
            self._kept = None
            N.check(st, "moe_norm_fwd")
        return y if rp is None else (y, s)

    def backward(self, dy, d_sum=None, need=("dx", "dw", "db"), out=None, stream=None):
        if self._kept is None:
            raise ValueError("backward: the last forward did not save (save=True)")
        (x, xp, ld_x, res, rp, ld_r), n, dev, dt, views = self._kept, self.N, self.device, self.dtype, self._views
        M = x.shape[0]
        shape, row = x.shape, M * self._size
        w, b = self.weight, self.bias
        if w is not self._w_ref() or b is not self._b_ref() or w.data_ptr() != self._w_ptr or (
                not self._like(w) if b is None else b.data_ptr() != self._b_ptr or not self._like(w, b)):
            self._bind()
        ld_y = n if dy.dtype is dt and dy.shape == shape and dy.is_contiguous() and dy.device == dev else _matrix(dy, "dy", dt, M, n, dev)
        dx = dw = db = dxp = dwp = dbp = sp = None
        ld_dx = ld_d = 0
        gone = False        # what was kept
        if d_sum is not None:
            d = d_sum
            ld_d = n if d.dtype is dt and d.shape == shape and d.is_contiguous() and d.device == dev else _matrix(d, "d_sum", dt, M, n, dev)
            sp = d.data_ptr()
        yp = dy.data_ptr()
        if "dx" in need:
            if out is None:
                dx, dxp = views.get(("dx", M)) or self._view("dx", M, stream)
                ld_dx = n
            else:
                dx, dxp, ld_dx = out, out.data_ptr(), self._given("out", out, M)
            end = row * ld_dx
            if -row * ld_y < yp - dxp < end:
                _in_place("dy", dy, ld_y, dx, ld_dx, "dx")
            if -row * ld_x < xp - dxp < end:
                _in_place("x", x, ld_x, dx, ld_dx, "dx")
                gone = xp == dxp
            if rp is not None and -row * ld_r < rp - dxp < end:
                _in_place("residual", res, ld_r, dx, ld_dx, "dx")
                gone = gone or rp == dxp
            if sp is not None and -row * ld_d < sp - dxp < end:
                _in_place("d_sum", d_sum, ld_d, dx, ld_dx, "dx")
        if "dw" in need:
            dw, dwp = views.get(("dw", None)) or self._view("dw", None, stream)
        if "db" in need and b is not None:
            db, dbp = views.get(("db", None)) or self._view("db", None, stream)
        if 0 < row <= self._w_size:     # few enough rows to lie in an earlier call's dw or db
            end = n * self._w_size
            for g in (dwp, dbp):
                if g is not None and (-row * ld_x < xp - g < end or -row * ld_y < yp - g < end or (
                        rp is not None and -row * ld_r < rp - g < end) or (sp is not None and -row * ld_d < sp - g < end) or (
                        dxp is not None and -row * ld_dx < dxp - g < end)):
                    raise ValueError("x, residual, dy, d_sum or out: lies in the weight's or bias's gradient (pass a copy)")
        if self.ws is None:
            self.ws = OpWorkspace(self._need, "moe_norm_workspace_bytes", dev, stream)
        key = M, ld_x, ld_r, ld_d, ld_y, ld_dx
        if key != self._bwd_set:
            D = self._bwd_dims
            D.M, D.ld_x, D.ld_res, D.ld_sum, D.ld_y, D.ld_dx = self._bwd_set = key
        st = self._bwd(xp, rp, yp, sp, self._w_ptr, self._bufs["stats"].data_ptr(), self._bwd_ref, dxp, dwp, dbp, self.ws.ptr, self.ws.nbytes,
                       _stream(stream, self._index))
        if st:
            N.check(st, "moe_norm_bwd")
        if gone:
            self._kept = None
        return dict(dx=dx, dw=dw, db=db)


def _bytes_meet(a, ld_a, b):
    """Whether the span of matrix a's rows and the dense tensor b share a byte."""
    end = a.data_ptr() + ((a.shape[0] - 1) * ld_a + a.shape[1]) * a.element_size()
    return a.data_ptr() < b.data_ptr() + b.numel() * b.element_size() and b.data_ptr() < end


class TokenLogprobs:
    """Log probabilities of given tokens under the softmax of rows of scores [M, V], with entropy and
    the ``top`` most probable alternatives, and the gradient of the scores: moe_token_logprob /
    moe_token_logprob_bwd for up to ``max_rows`` rows.

    ``forward(scores, tokens=None, entropy=False, save=False)`` returns a dict of ``logprob`` [M] (with
    tokens), ``entropy`` [M] (if asked for), ``top_idx`` and ``top_logprob`` [M, top] (if top > 0): own
    buffers, written by the next call (they may be changed, the backward does not read them). A token outside
    [0, V) is padding (0). With ``save=True`` it keeps scores and tokens (unchanged until then) for ``backward(d_logprob=None, d_entropy=None)``, which returns the
    gradient of the scores [M, V]: an own buffer unless ``out`` is given, which may be the scores (what was kept is
    then gone). Scores and their gradient begin on 16 bytes, their rows anywhere (fastest where both
    do alike). One instance serves one stream at a time, which waits for the one it was made on.
    """

    def __init__(self, max_rows, V, top=0, dtype=torch.float32, device="cuda", stream=None):
        self.max_rows, self.V, self.top, self.dtype = max_rows, V, top, dtype
        self.dims = N.LogprobDims(int(max_rows), V, top, _dt(dtype), 0, 0, 1)
        if not (0 <= max_rows <= 1 << 30 and 1 <= V <= 1 << 22 and 0 <= top <= 32):
            raise N.MoeError(N.STATUS_CODE["MOE_ERR_BAD_DIMS"], "moe_token_logprob")
        self.device, self._index = _device(device)
        with _on(stream, self.device):
            self._logprob, self._entropy, self._stats = (torch.empty(max_rows, w, dtype=torch.float32, device=device) for w in (1, 1, 4))
            top_idx = torch.empty(max_rows, top, dtype=torch.int32, device=device)
            top_logprob = torch.empty(max_rows, top, dtype=torch.float32, device=device)
        self._top = top_idx, top_logprob
        self._own = tuple((t.data_ptr(), 4 * t.numel()) for t in (self._logprob, self._entropy, top_idx, top_logprob) if t.numel())
        self._most = 4 * max_rows * max(1, top)     # bytes of the largest of them
        self._size = 2 if self.dims.dtype == N.MOE_BF16 else 4
        self._ptrs = (self._logprob.data_ptr(), self._entropy.data_ptr(), self._stats.data_ptr(),
                      top_idx.data_ptr() if top else None, top_logprob.data_ptr() if top else None)
        self._grad, self._views, self._saved, self._set = None, {}, None, None
        self._dims_ref = ctypes.byref(self.dims)
        self._fwd, self._bwd = N.lib().moe_token_logprob, N.lib().moe_token_logprob_bwd

    def forward(self, scores, tokens=None, entropy=False, save=False, stream=None):
        M, dev = scores.shape[0], self.device
        v = self._views.get(M)
        if v is None:
            if M > self.max_rows:
                raise ValueError(f"{M} rows, made for {self.max_rows}")
            if len(self._views) >= _KEPT_VIEWS:
                self._views.clear()
            v = self._views[M] = (torch.Size((M, self.V)), torch.Size((M,)), self._logprob[:M, 0], self._entropy[:M, 0],
                                  self._top[0][:M], self._top[1][:M])
        shape, of_rows, logprob, ent, top_idx, top_logprob = v
        t = scores
        ld = self.V if t.dtype is self.dtype and t.shape == shape and t.is_contiguous() and t.device == dev else _matrix(
            t, "scores", self.dtype, M, self.V, dev)
        if 0 < M * self.V * self._size <= self._most:   # small enough to lie in an earlier call's results
            xp, span = scores.data_ptr(), M * ld * self._size
            for p, size in self._own:
                if p - span < xp < p + size:
                    raise ValueError("scores: lies in a result, or overlaps it (pass a copy)")
        out = {}
        lp, ep, sp, ip, vp = self._ptrs
        if tokens is not None:
            t = tokens
            if t.dtype is not torch.int32 or t.shape != of_rows or not t.is_contiguous() or t.device != dev:
                _dense(t, "tokens", torch.int32, of_rows, dev)
            out["logprob"], tp = logprob, t.data_ptr()
            if ip is not None and -4 * M < tp - ip < 4 * M * self.top and (save or tp != ip or self.top > 1):
                raise ValueError("tokens: overlaps the result" + (", and is needed for the backward" if save else ""))
        else:
            tp = lp = None
        if entropy:
            out["entropy"] = ent
        else:
            ep = None
        if ip is not None:
            out["top_idx"], out["top_logprob"] = top_idx, top_logprob
        self._saved = (scores, ld, tokens, entropy) if save else None
        key = M, ld
        if key != self._set:
            D = self.dims
            D.M, D.ld = self._set = key
        st = self._fwd(scores.data_ptr(), tp, self._dims_ref, lp, ep, sp if save else None, ip, vp,
                       _raw_stream(self._index) if stream is None and _raw_stream is not None else _stream(stream, self._index))
        if st:
            self._saved = None
            N.check(st, "moe_token_logprob")
        return out

    def backward(self, d_logprob=None, d_entropy=None, out=None, stream=None):
        if self._saved is None:
            raise ValueError("backward: the last forward did not save (save=True)")
        (scores, ld, tokens, entropy), D, dev = self._saved, self.dims, self.device
        M = scores.shape[0]
        if d_logprob is not None:
            if tokens is None:
                raise ValueError("d_logprob: the last forward had no tokens")
            _dense(d_logprob, "d_logprob", torch.float32, (M,), dev)
        if d_entropy is not None:
            if not entropy:
                raise ValueError("d_entropy: the last forward took no entropy")
            _dense(d_entropy, "d_entropy", torch.float32, (M,), dev)
        if out is None:
            if self._grad is None:
                with _on(stream, dev):
                    self._grad = torch.empty(self.max_rows, self.V, dtype=self.dtype, device=dev)
            out, ld_g = self._grad[:M], self.V
        else:
            ld_g = _matrix(out, "out", self.dtype, M, self.V, dev)
        gp = out.data_ptr()     # (the own one may hold an earlier gradient, whose numbers are these)
        end = gp + M * ld_g * self._size
        for name, t in (("tokens", tokens), ("d_logprob", d_logprob), ("d_entropy", d_entropy)):
            if t is not None and gp - 4 * M < t.data_ptr() < end and M and _bytes_meet(out, ld_g, t):
                raise ValueError(f"{name}: overlaps the scores' gradient")
        _in_place("scores", scores, ld, out, ld_g, "their gradient")
        D.M, D.ld, D.ld_grad = M, ld, ld_g
        self._set = M, ld
        st = self._bwd(scores.data_ptr(), _p(tokens), self._stats.data_ptr(), None, _p(d_logprob), _p(d_entropy),
                       self._dims_ref, out.data_ptr(), _stream(stream, self._index))
        if st:
            N.check(st, "moe_token_logprob_bwd")
        if out.data_ptr() == scores.data_ptr():
            self._saved = None
        return out


_addresses_are = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", None)


class _Places:
    """Where contiguous tensors lie, how large they are and their types.

    To ask hundreds of tensors takes as long as the kernels run (300 gradients clipped into as many others in 105 us: 124 us
    of host time with calls for each tensor and property), so torch is asked for all of them at once where it can be (73
    us), and for each when that says no.
    """

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.addresses, self.every = [t.data_ptr() for t in tensors], list(range(len(tensors)))
        self.sizes, self.types = [t.numel() for t in tensors], [t.dtype for t in tensors]
        self.unchanged = _unchanged(*tensors)

    def hold(self):
        ts = self.tensors
        if _addresses_are is not None:
            if not _addresses_are(ts, self.addresses, self.every):
                return False
        elif [t.data_ptr() for t in ts] != self.addresses:
            return False
        return self.unchanged(*ts) or ([t.numel() for t in ts] == self.sizes and [t.dtype for t in ts] == self.types and
                                       all(t.is_contiguous() for t in ts))


class GradClipper:
    """The global norm of a list (or dict) of gradients, and their clipping: moe_clip_grads on a kept list
    (contiguous fp32 or bf16 tensors; those of None are left out).

    ``norm()`` returns the norm, ``clip(max_norm)`` also scales the gradients by min(1, max_norm / (norm +
    1e-6)), in place, or into ``out`` (a list of the same shape and types). Both return a tensor of one number
    without waiting for it, an own buffer that the next call writes; ``scale`` holds the factor of the
    last call. A tensor that has moved (``t.data = ...``) is taken where and as it is then, another tensor in its place (a
    parameter's new ``grad``) is not; a captured graph takes those of the capture. One instance serves one stream at a time, which waits for the one it was made on.
    """

    def __init__(self, grads, out=None, device=None, stream=None):
        grads = list(grads.values() if isinstance(grads, dict) else grads)
        outs = grads if out is None else list(out.values() if isinstance(out, dict) else out)
        if len(outs) != len(grads):
            raise ValueError(f"out: {len(outs)} tensors for {len(grads)} gradients")
        if any((g is None) != (o is None) for g, o in zip(grads, outs)):
            raise ValueError("out: None where a gradient is not, or the other way round")
        self.grads = [g for g in grads if g is not None]
        self.out = self.grads if out is None else [o for o in outs if o is not None]
        if device is None:
            device = self.grads[0].device if self.grads else "cuda"
        self.device, self._index = _device(device)
        self._places = None
        n = len(self.grads)
        self.ws = OpWorkspace(N.lib().moe_clip_workspace_bytes(n), "moe_clip_workspace_bytes", self.device, stream)
        with _on(stream, self.device):
            self._result = torch.empty(2, dtype=torch.float32, device=self.device)
        self._norm, self.scale = self._result[0], self._result[1]
        self._np, self._sp = self._norm.data_ptr(), self.scale.data_ptr()
        self._clip_table, self._norm_table = (N.Grad * max(n, 1))(), (N.Grad * max(n, 1))()
        self._call = N.lib().moe_clip_grads
        self._bind()

    def _bind(self):
        """Checks the tensors and takes their present places."""
        self._places = None
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for name, t in (("gradient", g), ("out", o)):
                if not t.is_contiguous() or t.dtype not in (torch.float32, torch.bfloat16):
                    raise ValueError(f"{name} {i}: expected a contiguous fp32 or bf16 tensor, got {list(t.shape)} of {t.dtype}, "
                                     f"strides {t.stride()}")
                if t.device != self.device:
                    _elsewhere(f"{name} {i}", self.device, t)
            if o.dtype != g.dtype or o.shape != g.shape:
                raise ValueError(f"out {i}: expected {list(g.shape)} of {g.dtype}, got {list(o.shape)} of {o.dtype}")
            self._clip_table[i] = N.Grad(g.data_ptr(), o.data_ptr(), g.numel(), _dt(g.dtype))
            self._norm_table[i] = N.Grad(g.data_ptr(), None, g.numel(), _dt(g.dtype))
        self._check_places()
        self._places = _Places(self.grads)
        self._out_places = self._places if self.out is self.grads else _Places(self.out)

    def _check_places(self):
        """No result may overlap another one, or a gradient other than its own (that one only as a whole)."""
        spans = []      # (first byte, behind the last, result's name or None, gradient's name)
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            a, b, size = g.data_ptr(), o.data_ptr(), g.numel() * g.element_size()
            if size:
                spans.append((b, b + size, f"out {i}", None))
                if a != b:
                    spans.append((a, a + size, None, f"gradient {i}"))
        spans.sort(key=lambda s: s[0])
        read = written = (0, None)      # the end that reaches furthest, and whose
        for a, b, result, gradient in spans:
            for end, name in ((written,) if gradient else (written, read)):
                if a < end:
                    raise ValueError(f"{result or gradient}: overlaps {name}")
            if result:
                written = max(written, (b, result))
            else:
                read = max(read, (b, gradient))

    def _run(self, table, max_norm, stream):
        st = self._call(table, len(self.grads), max_norm, self._np, self._sp, self.ws.ptr, self.ws.nbytes,
                        _stream(stream, self._index))
        if st:
            N.check(st, "moe_clip_grads")
        return self._norm

    def norm(self, stream=None):
        if self._places is None or not self._places.hold():
            self._bind()
        return self._run(self._norm_table, float("inf"), stream)

    def clip(self, max_norm, stream=None):
        if self._places is None or not self._places.hold() or not (
                self._out_places is self._places or self._out_places.hold()):
            self._bind()
        return self._run(self._clip_table, max_norm, stream)
