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

from . import GDN_BF16, GDN_F32, GdnError, _torch_stream, load_library

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
_Tensor = _raw_stream = _current_device = _empty_like = None  # from torch, bound on first use
_codes = {}  # torch dtype -> gdn_dtype


def layer_library():
    """The HIP library with this header's entry points declared."""
    global _lib, _torch, _Tensor, _raw_stream, _current_device, _empty_like
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
        _torch, _Tensor, _empty_like = torch, torch.Tensor, torch.empty_like
        _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _lib = lib
    return _lib


def _code(dtype, name):
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    return code


def _device(t, name):
    """The index of the device that the call runs on."""
    if _lib is None:
        layer_library()
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a device tensor")
    return index


def _rows(t, name, shape, index, dtype=None):
    """Checks a tensor [rows][...] whose rows are dense; returns the stride
    between rows."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    stride = t.stride()
    if not t.is_contiguous():
        want = 1
        for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
            if n != 1 and s != want:
                raise ValueError(f"{name}: the elements of a row must be dense")
            want *= n
    return stride[0]


def _dense(t, name, shape, index, dtype):
    """The address of a contiguous tensor, None for None."""
    if t is None:
        return None
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index or t.dtype != dtype or not t.is_contiguous():
        raise (TypeError if t.dtype != dtype else ValueError)(f"{name} must be a contiguous {dtype} tensor on device {index}")
    return t.data_ptr()


def _workspace(t, index):
    """The address and size of a caller's workspace."""
    if not isinstance(t, _Tensor):
        raise TypeError("workspace must be a torch tensor")
    if t.dtype != _torch.uint8:
        raise TypeError(f"workspace must be {_torch.uint8}, got {t.dtype}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on device {index}")
    return t.data_ptr(), t.numel()


def _stream(stream, index):
    """The raw handle of the call's stream."""
    if stream is None:
        return _raw_stream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(like, shape, dtype, index, raw, stream, keep=True):
    """Memory for an output, or with ``keep`` false for this call alone.  The
    allocator hands out what is free in the order of one stream, so a call on
    another stream than the current one allocates there; what its caller keeps
    is marked as used on the current stream as well."""
    if stream is not None and raw != _raw_stream(index):
        with _torch.cuda.stream(_torch_stream(stream, index)):
            t = like.new_empty(shape, dtype=dtype)
        if keep:
            t.record_stream(_torch.cuda.current_stream(index))
        return t
    if like.shape == shape and like.is_contiguous():  # 0.5 us less than from a shape
        return _empty_like(like, dtype=dtype)
    return like.new_empty(shape, dtype=dtype)


def _run(index, fn, *args):
    if _current_device() == index:
        code = fn(*args)
    else:
        with _torch.cuda.device(index):
            code = fn(*args)
    if code != 0:
        raise GdnError(code, _lib.gdn_last_error().decode())


def _seq_dims(q, k, v, g, beta, S, n, index, q_scale, qk_l2norm, l2_eps, o_dtype):
    if q.dim() != 3 or v.dim() != 3 or S.dim() != 4:
        raise ValueError("q, k and v must have 3 dimensions, S 4")
    rows, Hk, dk = shape = q.shape
    Hv, dv = v.shape[1:]
    dtype = q.dtype
    qs = _rows(q, "q", shape, index)
    ks = _rows(k, "k", shape, index, dtype)
    vs = _rows(v, "v", (rows, Hv, dv), index, dtype)
    if rows <= 1:  # one row has no stride
        qs = ks = vs = 0
    f32 = _torch.float32
    slots = S.shape[0]
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _dense(g, "g", (rows, Hv), index, f32),
            _dense(beta, "beta", (rows, Hv), index, f32), _dense(S, "S", (slots, Hv, dv, dk), index, f32))
    return SeqDims(rows if n is None else n, rows, Hk, Hv, dk, dv, _code(dtype, "q"), _code(o_dtype, "o_dtype"), slots,
                   bool(qk_l2norm), q_scale, l2_eps, qs, ks, vs), ptrs


def gdn_prefill(q, k, v, g, beta, cu_seqlens, S, slot=None, has_state=None, q_scale=1.0, qk_l2norm=False, l2_eps=1e-6,
                o=None, o_dtype=None, seq_status=None, workspace=None, stream=None):
    """The delta rule over packed sequences: q, k [T][H_k][d_k], v
    [T][H_v][d_v], g and beta [T][H_v], cu_seqlens [B + 1] int32, the state
    pool S [n][H_v][d_v][d_k] updated in place (sequence b at slot[b], or at
    b).  has_state[b] == 0 starts sequence b from zero.  Returns o
    [T][H_v][d_v] (q's dtype unless ``o`` or ``o_dtype`` says otherwise).
    ``workspace``: a uint8 device tensor of at least
    :func:`gdn_prefill_workspace_bytes` bytes to allocate nothing here."""
    index = _device(q, "q")
    n = cu_seqlens.shape[0] - 1
    o_dtype = o.dtype if o is not None else o_dtype or q.dtype
    dims, (qp, kp, vp, gp, bp, sp) = _seq_dims(q, k, v, g, beta, S, n, index, q_scale, qk_l2norm, l2_eps, o_dtype)
    i32 = _torch.int32
    cu = _dense(cu_seqlens, "cu_seqlens", (n + 1,), index, i32)
    slot = _dense(slot, "slot", (n,), index, i32)
    has_state = _dense(has_state, "has_state", (n,), index, i32)
    seq_status = _dense(seq_status, "seq_status", (n,), index, i32)
    raw = _stream(stream, index)
    if o is None:
        o = _empty(v, v.shape, o_dtype, index, raw, stream)
        op = o.data_ptr()
    else:
        op = _dense(o, "o", v.shape, index, o_dtype)
    if workspace is None:
        need = _lib.gdn_prefill_workspace_bytes(dims)
        workspace = _empty(q, (need,), _torch.uint8, index, raw, stream, keep=False)
    wp, nbytes = _workspace(workspace, index)
    _run(index, _lib.gdn_prefill, dims, qp, kp, vp, gp, bp, cu, slot, has_state, sp, op, seq_status, wp, nbytes, raw)
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
    index = _device(q, "q")
    o_dtype = o.dtype if o is not None else o_dtype or q.dtype
    dims, (qp, kp, vp, gp, bp, sp) = _seq_dims(q, k, v, g, beta, S, None, index, q_scale, qk_l2norm, l2_eps, o_dtype)
    slot = _dense(slot, "slot", (q.shape[0],), index, _torch.int32)
    raw = _stream(stream, index)
    if o is None:
        o = _empty(v, v.shape, o_dtype, index, raw, stream)
        op = o.data_ptr()
    else:
        op = _dense(o, "o", v.shape, index, o_dtype)
    _run(index, _lib.gdn_decode, dims, qp, kp, vp, gp, bp, slot, sp, op, raw)
    return o


def gdn_add_norm(x, residual, weight, scale=1.0, chan_scale=None, post_weight=None, eps=1e-6, weight_offset=0.0,
                 h=None, y=None, y_dtype=None, stream=None):
    """(y, h): the residual sum h = residual + scale * p and its RMS norm y,
    where p is x, or with ``post_weight`` x's own RMS norm, times
    ``chan_scale`` if given.  x [T][D]; h has the residual's dtype (x's where
    there is no residual) and may be the residual itself; y is bfloat16
    unless ``y`` or ``y_dtype`` says otherwise."""
    index = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have 2 dimensions")
    T, D = shape = x.shape
    xs = _rows(x, "x", shape, index)
    if residual is None:
        rs, rp, h_dtype = 0, None, x.dtype
    else:
        rs, rp, h_dtype = _rows(residual, "residual", shape, index), residual.data_ptr(), residual.dtype
    f32 = _torch.float32
    raw = _stream(stream, index)
    if h is None:
        h, hs = _empty(x, shape, h_dtype, index, raw, stream), D
    else:
        hs = _rows(h, "h", shape, index, h_dtype)
    if y is None:
        y, ys = _empty(x, shape, y_dtype or _torch.bfloat16, index, raw, stream), D
    else:
        ys = _rows(y, "y", shape, index, y_dtype)
    dims = AddNormDims(T, D, _code(x.dtype, "x"), _code(h_dtype, "residual"), _code(y.dtype, "y"), scale, eps,
                       weight_offset, xs, rs, hs, ys)
    _run(index, _lib.gdn_add_norm, dims, x.data_ptr(), rp, _dense(weight, "weight", (D,), index, f32),
         _dense(post_weight, "post_weight", (D,), index, f32), _dense(chan_scale, "chan_scale", (D,), index, f32),
         h.data_ptr(), y.data_ptr(), raw)
    return y, h


def gdn_gated_norm(o, z, weight, eps=1e-6, gate="silu", y=None, y_dtype=None, stream=None):
    """y = rms(o) * weight * gate(z) over each head of o and z [T][H][d];
    ``gate`` is "silu" or "sigmoid"; y is bfloat16 unless ``y`` or
    ``y_dtype`` says otherwise, and may be o or z itself."""
    index = _device(o, "o")
    if o.dim() != 3:
        raise ValueError("o must have 3 dimensions")
    T, H, d = shape = o.shape
    os_ = _rows(o, "o", shape, index)
    zs = _rows(z, "z", shape, index)
    raw = _stream(stream, index)
    if y is None:
        y, ys = _empty(o, shape, y_dtype or _torch.bfloat16, index, raw, stream), H * d
    else:
        ys = _rows(y, "y", shape, index, y_dtype)
    if gate not in ("silu", "sigmoid"):
        raise ValueError('gate must be "silu" or "sigmoid"')
    dims = GatedNormDims(T, H, d, _code(o.dtype, "o"), _code(z.dtype, "z"), _code(y.dtype, "y"), ACTS[gate], eps, os_,
                         zs, ys)
    _run(index, _lib.gdn_gated_norm, dims, o.data_ptr(), z.data_ptr(),
         _dense(weight, "weight", (d,), index, _torch.float32), y.data_ptr(), raw)
    return y


def gdn_linear(x, w, bias=None, act="none", residual=None, scale=1.0, y=None, y_dtype=None, workspace=None,
               stream=None):
    """y = residual + scale * act(x w^T + bias): x [M][K] and w [N][K]
    bfloat16, bias [N] float32, residual and y [M][N]; ``act`` is "none",
    "silu", "gelu" or "sigmoid"; y is bfloat16 unless ``y`` or ``y_dtype``
    says otherwise, and may be the residual itself."""
    index = _device(x, "x")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must have 2 dimensions")
    M, K = x.shape
    N = w.shape[0]
    bf16 = _torch.bfloat16
    xs = _rows(x, "x", (M, K), index, bf16)
    ws = _rows(w, "w", (N, K), index, bf16)
    if residual is None:
        rs, rp, r_code = 0, None, GDN_BF16
    else:
        rs, rp, r_code = _rows(residual, "residual", (M, N), index), residual.data_ptr(), _code(residual.dtype, "residual")
    raw = _stream(stream, index)
    if y is None:
        y, ys = _empty(x if residual is None else residual, (M, N), y_dtype or bf16, index, raw, stream), N
    else:
        ys = _rows(y, "y", (M, N), index, y_dtype)
    act_code = ACTS.get(act)
    if act_code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    dims = LinearDims(M, N, K, r_code, _code(y.dtype, "y"), act_code, scale, xs, ws, rs, ys)
    if workspace is None:
        need = _lib.gdn_linear_workspace_bytes(dims)
        if need:
            workspace = _empty(x, (need,), _torch.uint8, index, raw, stream, keep=False)
    wp, nbytes = (None, 0) if workspace is None else _workspace(workspace, index)
    _run(index, _lib.gdn_linear, dims, x.data_ptr(), w.data_ptr(), _dense(bias, "bias", (N,), index, _torch.float32), rp,
         y.data_ptr(), wp, nbytes, raw)
    return y
