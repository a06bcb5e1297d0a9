"""The operators around the tree verify (``include/gdn_layer.h``): the delta
rule over packed prompts and over single tokens, the norms around the layer,
and its projections.

Argument marshalling only, as in the rest of the binding: tensors are checked,
outputs are allocated where none is passed, and the HIP kernels of
``libgdn_tree.so`` do the work on the current stream (or on ``stream``).
Rows may be slices of wider tensors: only what one row holds has to be dense.
"""
from __future__ import annotations

import ctypes

from . import GDN_BF16, GDN_F32, GdnError, load_library

LAYER_EXPORTS = ["gdn_prefill_workspace_bytes", "gdn_prefill", "gdn_decode", "gdn_add_norm", "gdn_gated_norm",
                 "gdn_linear_workspace_bytes", "gdn_linear"]
ACTS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class SeqDims(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("H_k", _i32), ("H_v", _i32), ("d_k", _i32), ("d_v", _i32),
                ("qkv_dtype", _i32), ("o_dtype", _i32), ("n_slots", _i32), ("qk_l2norm", _i32), ("q_scale", _f32),
                ("l2_eps", _f32), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64)]


class AddNormDims(ctypes.Structure):
    _fields_ = [("T", _i32), ("D", _i32), ("x_dtype", _i32), ("res_dtype", _i32), ("y_dtype", _i32), ("scale", _f32),
                ("eps", _f32), ("weight_offset", _f32), ("x_stride", _i64), ("res_stride", _i64), ("h_stride", _i64),
                ("y_stride", _i64)]


class GatedNormDims(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("d", _i32), ("o_dtype", _i32), ("z_dtype", _i32), ("y_dtype", _i32),
                ("gate", _i32), ("eps", _f32), ("o_stride", _i64), ("z_stride", _i64), ("y_stride", _i64)]


class LinearDims(ctypes.Structure):
    _fields_ = [("M", _i32), ("N", _i32), ("K", _i32), ("res_dtype", _i32), ("y_dtype", _i32), ("act", _i32),
                ("scale", _f32), ("x_stride", _i64), ("w_stride", _i64), ("res_stride", _i64), ("y_stride", _i64)]


_lib = None
_torch = None
_codes = {}  # torch dtype -> gdn_dtype


def layer_library():
    """The HIP library with this header's entry points declared."""
    global _lib, _torch
    if _lib is None:
        lib = load_library()
        import torch
        size = ctypes.c_size_t
        ptr = ctypes.POINTER
        lib.gdn_prefill_workspace_bytes.argtypes = [ptr(SeqDims)]
        lib.gdn_prefill_workspace_bytes.restype = size
        lib.gdn_prefill.argtypes = [ptr(SeqDims)] + [_vp] * 12 + [size, _vp]
        lib.gdn_decode.argtypes = [ptr(SeqDims)] + [_vp] * 9
        lib.gdn_add_norm.argtypes = [ptr(AddNormDims)] + [_vp] * 8
        lib.gdn_gated_norm.argtypes = [ptr(GatedNormDims)] + [_vp] * 5
        lib.gdn_linear_workspace_bytes.argtypes = [ptr(LinearDims)]
        lib.gdn_linear_workspace_bytes.restype = size
        lib.gdn_linear.argtypes = [ptr(LinearDims)] + [_vp] * 6 + [size, _vp]
        for name in ("gdn_prefill", "gdn_decode", "gdn_add_norm", "gdn_gated_norm", "gdn_linear"):
            getattr(lib, name).restype = ctypes.c_int
        _codes.update({torch.bfloat16: GDN_BF16, torch.float32: GDN_F32})
        _torch = torch
        _lib = lib
    return _lib


def _code(dtype, name):
    try:
        return _codes[dtype]
    except KeyError:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}") from None


def _rows(t, name, shape, device, dtype=None):
    """Checks a tensor [rows][...] whose rows are dense; returns the stride
    between rows (0 where there is one row)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return t.numel() // shape[0] if shape[0] > 0 else 0
    stride, want = t.stride(), 1
    for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
        if n != 1 and s != want:
            raise ValueError(f"{name}: the elements of a row must be dense")
        want *= n
    return stride[0] if shape[0] > 1 else 0


def _dense(t, name, shape, device, dtype):
    if t is None:
        return None
    _rows(t, name, shape, device, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_device(t, name):
    layer_library()
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


class _Launch:
    """The call's device and stream.  Memory allocated here for work on a
    stream other than the current one is marked as used there."""

    def __init__(self, device, stream):
        self.device, self.current = device, _torch.cuda.current_stream(device)
        self.other = None
        if stream is None:
            self.raw = self.current.cuda_stream
        else:
            self.raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            if self.raw != self.current.cuda_stream:
                self.other = _torch.cuda.ExternalStream(self.raw, device=device)

    def empty(self, shape, dtype):
        t = _torch.empty(shape, dtype=dtype, device=self.device)
        if self.other is not None:
            t.record_stream(self.other)
        return t

    def run(self, fn, *args):
        if _torch.cuda.current_device() != self.device.index:
            with _torch.cuda.device(self.device):
                code = fn(*args, self.raw)
        else:
            code = fn(*args, self.raw)
        if code != 0:
            raise GdnError(code, _lib.gdn_last_error().decode())


def _seq_dims(q, k, v, g, beta, S, slot, n, device, q_scale, qk_l2norm, l2_eps, o_dtype):
    if q.dim() != 3 or v.dim() != 3 or S.dim() != 4:
        raise ValueError("q, k and v must have 3 dimensions, S 4")
    rows, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    if n is None:
        n = rows
    qs = _rows(q, "q", (rows, Hk, dk), device)
    ks = _rows(k, "k", (rows, Hk, dk), device, q.dtype)
    vs = _rows(v, "v", (rows, Hv, dv), device, q.dtype)
    _dense(g, "g", (rows, Hv), device, _torch.float32)
    _dense(beta, "beta", (rows, Hv), device, _torch.float32)
    _dense(S, "S", (S.shape[0], Hv, dv, dk), device, _torch.float32)
    _dense(slot, "slot", (n,), device, _torch.int32)
    return SeqDims(n, rows, Hk, Hv, dk, dv, _code(q.dtype, "q"), _code(o_dtype, "o_dtype"), S.shape[0],
                   int(bool(qk_l2norm)), q_scale, l2_eps, qs, ks, vs)


def _ptr(t):
    return None if t is None else t.data_ptr()


def gdn_prefill(q, k, v, g, beta, cu_seqlens, S, slot=None, has_state=None, q_scale=1.0, qk_l2norm=False, l2_eps=1e-6,
                o=None, o_dtype=None, seq_status=None, workspace=None, stream=None):
    """The delta rule over packed sequences: q, k [T][H_k][d_k], v
    [T][H_v][d_v], g and beta [T][H_v], cu_seqlens [B + 1] int32, the state
    pool S [n][H_v][d_v][d_k] updated in place (sequence b at slot[b], or at
    b).  has_state[b] == 0 starts sequence b from zero.  Returns o
    [T][H_v][d_v] (q's dtype unless ``o`` or ``o_dtype`` says otherwise).
    ``workspace``: a uint8 device tensor of at least
    :func:`gdn_prefill_workspace_bytes` bytes to allocate nothing here."""
    device = _on_device(q, "q")
    n = cu_seqlens.shape[0] - 1
    o_dtype = o.dtype if o is not None else o_dtype or q.dtype
    dims = _seq_dims(q, k, v, g, beta, S, slot, n, device, q_scale, qk_l2norm, l2_eps, o_dtype)
    _dense(cu_seqlens, "cu_seqlens", (n + 1,), device, _torch.int32)
    _dense(has_state, "has_state", (n,), device, _torch.int32)
    _dense(seq_status, "seq_status", (n,), device, _torch.int32)
    at = _Launch(device, stream)
    if o is None:
        o = at.empty(v.shape, o_dtype)
    else:
        _dense(o, "o", v.shape, device, o_dtype)
    need = _lib.gdn_prefill_workspace_bytes(dims)
    if workspace is None and need:
        workspace = at.empty((need,), _torch.uint8)
    at.run(_lib.gdn_prefill, dims, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
           cu_seqlens.data_ptr(), _ptr(slot), _ptr(has_state), S.data_ptr(), o.data_ptr(), _ptr(seq_status),
           _ptr(workspace), 0 if workspace is None else workspace.numel())
    return o


def gdn_prefill_workspace_bytes(q, v, cu_seqlens):
    """Bytes of workspace :func:`gdn_prefill` needs for tensors of these shapes."""
    lib = layer_library()
    return lib.gdn_prefill_workspace_bytes(SeqDims(
        cu_seqlens.shape[0] - 1, q.shape[0], q.shape[1], v.shape[1], q.shape[2], v.shape[2],
        _code(q.dtype, "q"), GDN_F32, 0, 0, 1.0, 0.0, 0, 0, 0))


def gdn_decode(q, k, v, g, beta, S, slot=None, q_scale=1.0, qk_l2norm=False, l2_eps=1e-6, o=None, o_dtype=None,
               stream=None):
    """One token per sequence: q, k [B][H_k][d_k], v [B][H_v][d_v], g and beta
    [B][H_v]; the states in the pool S are updated in place.  A row whose
    slot is outside the pool is idle (o = 0).  Returns o [B][H_v][d_v]."""
    device = _on_device(q, "q")
    o_dtype = o.dtype if o is not None else o_dtype or q.dtype
    dims = _seq_dims(q, k, v, g, beta, S, slot, None, device, q_scale, qk_l2norm, l2_eps, o_dtype)
    at = _Launch(device, stream)
    if o is None:
        o = at.empty(v.shape, o_dtype)
    else:
        _dense(o, "o", v.shape, device, o_dtype)
    at.run(_lib.gdn_decode, dims, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(slot),
           S.data_ptr(), o.data_ptr())
    return o


def gdn_add_norm(x, residual, weight, scale=1.0, chan_scale=None, post_weight=None, eps=1e-6, weight_offset=0.0,
                 h=None, y=None, y_dtype=None, stream=None):
    """(y, h): the residual sum h = residual + scale * p and its RMS norm y,
    where p is x, or with ``post_weight`` x's own RMS norm, times
    ``chan_scale`` if given.  x [T][D]; h has the residual's dtype (x's where
    there is no residual) and may be the residual itself."""
    device = _on_device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have 2 dimensions")
    T, D = shape = x.shape
    xs = _rows(x, "x", shape, device)
    rs = 0 if residual is None else _rows(residual, "residual", shape, device)
    h_dtype = x.dtype if residual is None else residual.dtype
    f32 = _torch.float32
    _dense(weight, "weight", (D,), device, f32)
    _dense(chan_scale, "chan_scale", (D,), device, f32)
    _dense(post_weight, "post_weight", (D,), device, f32)
    at = _Launch(device, stream)
    if h is None:
        h, hs = at.empty(shape, h_dtype), D
    else:
        hs = _rows(h, "h", shape, device, h_dtype)
    if y is None:
        y, ys = at.empty(shape, y_dtype or _torch.bfloat16), D
    else:
        ys = _rows(y, "y", shape, device, y_dtype)
    dims = AddNormDims(T, D, _code(x.dtype, "x"), _code(h_dtype, "residual"), _code(y.dtype, "y"), scale, eps,
                       weight_offset, xs, rs, hs, ys)
    at.run(_lib.gdn_add_norm, dims, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(post_weight),
           _ptr(chan_scale), h.data_ptr(), y.data_ptr())
    return y, h


def gdn_gated_norm(o, z, weight, eps=1e-6, gate="silu", y=None, y_dtype=None, stream=None):
    """y = rms(o) * weight * gate(z) over each head of o and z [T][H][d];
    ``gate`` is "silu" or "sigmoid"."""
    device = _on_device(o, "o")
    if o.dim() != 3:
        raise ValueError("o must have 3 dimensions")
    T, H, d = shape = o.shape
    os_ = _rows(o, "o", shape, device)
    zs = _rows(z, "z", shape, device)
    _dense(weight, "weight", (d,), device, _torch.float32)
    at = _Launch(device, stream)
    if y is None:
        y, ys = at.empty(shape, y_dtype or _torch.bfloat16), H * d
    else:
        ys = _rows(y, "y", shape, device, y_dtype)
    if gate not in ("silu", "sigmoid"):
        raise ValueError('gate must be "silu" or "sigmoid"')
    dims = GatedNormDims(T, H, d, _code(o.dtype, "o"), _code(z.dtype, "z"), _code(y.dtype, "y"), ACTS[gate], eps, os_,
                         zs, ys)
    at.run(_lib.gdn_gated_norm, dims, o.data_ptr(), z.data_ptr(), weight.data_ptr(), y.data_ptr())
    return y


def gdn_linear(x, w, bias=None, act="none", residual=None, scale=1.0, y=None, y_dtype=None, workspace=None,
               stream=None):
    """y = residual + scale * act(x w^T + bias): x [M][K] and w [N][K]
    bfloat16, bias [N] float32, residual and y [M][N]; ``act`` is "none",
    "silu", "gelu" or "sigmoid".  ``y`` may be the residual itself."""
    device = _on_device(x, "x")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must have 2 dimensions")
    M, K = x.shape
    N = w.shape[0]
    bf16 = _torch.bfloat16
    xs = _rows(x, "x", (M, K), device, bf16)
    ws = _rows(w, "w", (N, K), device, bf16)
    _dense(bias, "bias", (N,), device, _torch.float32)
    rs = 0 if residual is None else _rows(residual, "residual", (M, N), device)
    at = _Launch(device, stream)
    if y is None:
        y, ys = at.empty((M, N), y_dtype or bf16), N
    else:
        ys = _rows(y, "y", (M, N), device, y_dtype)
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    dims = LinearDims(M, N, K, GDN_BF16 if residual is None else _code(residual.dtype, "residual"),
                      _code(y.dtype, "y"), ACTS[act], scale, xs, ws, rs, ys)
    need = _lib.gdn_linear_workspace_bytes(dims)
    if workspace is None and need:
        workspace = at.empty((need,), _torch.uint8)
    at.run(_lib.gdn_linear, dims, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(),
           _ptr(workspace), 0 if workspace is None else workspace.numel())
    return y
