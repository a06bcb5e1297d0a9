"""The softmax attention layers between Gated DeltaNet layers
(``include/gdn_attn.h``): a paged cache of keys and values, what appends to it
and commits in it, and the attention of prompts, single tokens and whole trees
over it.

Argument marshalling only, as in the rest of the binding: tensors are checked,
outputs are allocated where none is passed, and the HIP kernels of
``libgdn_tree.so`` do the work on the current stream (or on ``stream``).
"""
from __future__ import annotations

import ctypes

from . import GDN_BF16
from . import layer as _layer
from .layer import _dense, _device, _empty, _run, _stream, _workspace

ATTN_EXPORTS = ["gdn_kv_append", "gdn_attn_prefill_workspace_bytes", "gdn_attn_decode_workspace_bytes",
                "gdn_attn_verify_workspace_bytes", "gdn_attn_decode", "gdn_attn_prefill", "gdn_attn_verify",
                "gdn_kv_commit"]
GDN_E4M3 = 2

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("n_pages", _i32), ("page_size", _i32),
                ("H_kv", _i32), ("d", _i32), ("dtype", _i32), ("reserved", _i32), ("k_page_stride", _i64),
                ("k_row_stride", _i64), ("k_head_stride", _i64), ("v_page_stride", _i64), ("v_row_stride", _i64),
                ("v_head_stride", _i64)]


class AppendDims(ctypes.Structure):
    _fields_ = [("T", _i32), ("H_q", _i32), ("in_dtype", _i32), ("rot", _i32), ("interleaved", _i32), ("eps", _f32),
                ("weight_offset", _f32), ("reserved", _i32), ("q_stride", _i64), ("q_head_stride", _i64),
                ("k_stride", _i64), ("k_head_stride", _i64), ("v_stride", _i64), ("v_head_stride", _i64)]


class AttnDims(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("H_q", _i32), ("max_pages", _i32), ("scale", _f32), ("reserved", _i32),
                ("q_stride", _i64), ("gate_stride", _i64), ("gate_head_stride", _i64), ("table_stride", _i64)]


class CommitDims(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("max_pages", _i32), ("reserved", _i32), ("table_stride", _i64)]


_lib = None
_torch = None
_Tensor = _bf16 = _int32 = None


def attn_library():
    """The HIP library with this header's entry points declared."""
    global _lib, _torch, _Tensor, _bf16, _int32
    if _lib is None:
        lib = _layer.layer_library()
        import torch
        size, ptr = ctypes.c_size_t, ctypes.POINTER
        cache = ptr(KvCacheStruct)
        lib.gdn_kv_append.argtypes = [ptr(AppendDims), cache] + [_vp] * 10
        lib.gdn_attn_decode.argtypes = [ptr(AttnDims), cache] + [_vp] * 7 + [size, _vp]
        lib.gdn_attn_prefill.argtypes = [ptr(AttnDims), cache] + [_vp] * 8 + [size, _vp]
        lib.gdn_attn_verify.argtypes = [ptr(AttnDims), cache] + [_vp] * 8 + [size, _vp]
        lib.gdn_kv_commit.argtypes = [ptr(CommitDims), cache, _i32] + [_vp] * 7
        for name in ("gdn_kv_append", "gdn_attn_decode", "gdn_attn_prefill", "gdn_attn_verify", "gdn_kv_commit"):
            getattr(lib, name).restype = ctypes.c_int
        for name in ("prefill", "decode", "verify"):
            fn = getattr(lib, f"gdn_attn_{name}_workspace_bytes")
            fn.argtypes, fn.restype = [ptr(AttnDims), cache], size
        _torch, _Tensor, _bf16, _int32 = torch, torch.Tensor, torch.bfloat16, torch.int32
        _lib = lib
    return _lib


class GdnKvCache:
    """One layer's cache: pools of keys and values [n_pages][page_size][H_kv][d],
    bfloat16 or float8_e4m3fn, of any strides whose heads are dense (views of
    pools in another order, or of one pool of both).  ``k_scale`` and
    ``v_scale`` [H_kv] float32: what is stored stands for itself times its
    head's scale.  Holds the tensors, and their addresses for every call."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if _lib is None:
            attn_library()
        index = _device(k, "k")
        if k.dim() != 4:
            raise ValueError("k must have 4 dimensions")
        if not isinstance(v, _Tensor):
            raise TypeError("v must be a torch tensor")
        if v.shape != k.shape:
            raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
        if v.get_device() != index:
            raise ValueError(f"v must be on device {index}, got {v.device}")
        if k.dtype not in (_bf16, _torch.float8_e4m3fn):
            raise TypeError(f"k must be bfloat16 or float8_e4m3fn, got {k.dtype}")
        if v.dtype != k.dtype:
            raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
        n, page, H, d = k.shape
        for t, name in ((k, "k"), (v, "v")):
            if t.stride(3) != 1:
                raise ValueError(f"{name}: the elements of a head must be dense")
        scales = [_dense(s, name, (H,), index, _torch.float32) for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self.k, self.v, self.k_scale, self.v_scale, self.index = k, v, k_scale, v_scale, index
        self.heads, self.d = H, d
        strides = [t.stride(i) if t.shape[i] > 1 else 0 for t in (k, v) for i in range(3)]  # one page, row or head has none
        self.struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), *scales, n, page, H, d,
                                    GDN_BF16 if k.dtype == _bf16 else GDN_E4M3, 0, *strides)
        self.raw = bytes(self.struct)  # an array of these is joined, 6 us sooner than built of 12 structs


def _cache(cache):
    if not isinstance(cache, GdnKvCache):
        raise TypeError("cache must be a GdnKvCache")
    return cache.index


def _heads(t, name, shape, index, dtype):
    """Checks [rows][heads][d] with dense heads; returns the strides of rows and heads."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    stride = t.stride()
    if stride[2] != 1:
        raise ValueError(f"{name}: the elements of a head must be dense")
    return (stride[0] if shape[0] > 1 else 0), (stride[1] if shape[1] > 1 else 0)


def gdn_kv_append(cache, k, v, slot, position=None, inv_freq=None, q=None, q_weight=None, k_weight=None, eps=1e-6,
                  weight_offset=0.0, interleaved=False, q_out=None, stream=None):
    """Norm (where there are weights) and rotation of new queries and keys;
    keys and values go into ``cache``: token t to row slot[t] % page_size of
    page slot[t] // page_size (nowhere if outside).  k, v [T][H_kv][d] and q
    [T][H_q][d] bfloat16 or float32, slices of wider rows or not; inv_freq
    [rot / 2] float32 rotates the first rot elements of every head by
    position[t] * inv_freq, in pairs of neighbours if ``interleaved``, else
    of halves.  Returns q_out [T][H_q][d] bfloat16, None without q."""
    index = _cache(cache)
    d, H = cache.d, cache.heads
    if not isinstance(k, _Tensor):
        raise TypeError("k must be a torch tensor")
    if k.dim() != 3:
        raise ValueError("k must have 3 dimensions")
    T, dtype = k.shape[0], k.dtype
    code = GDN_BF16 if dtype == _bf16 else _layer._code(dtype, "k")
    kt, kh = _heads(k, "k", (T, H, d), index, dtype)
    vt, vh = _heads(v, "v", (T, H, d), index, dtype)
    raw = _stream(stream, index)
    H_q = qt = qh = 0
    qp = op = None
    if q is not None:
        if not isinstance(q, _Tensor):
            raise TypeError("q must be a torch tensor")
        if q.dim() != 3:
            raise ValueError("q must have 3 dimensions")
        H_q = q.shape[1]
        qt, qh = _heads(q, "q", (T, H_q, d), index, dtype)
        qp = q.data_ptr()
        if q_out is None:
            q_out = _empty(q, (T, H_q, d), _bf16, index, raw, stream)
            op = q_out.data_ptr()
        else:
            op = _dense(q_out, "q_out", (T, H_q, d), index, _bf16)
            if op == qp:  # strides of single tokens or heads count as dense
                qt, qh = qt or H_q * d, qh or d
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, _Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a tensor of 1 dimension")
        rot = 2 * inv_freq.shape[0]
    f32 = _torch.float32
    dims = AppendDims(T, H_q, code, rot, bool(interleaved), eps, weight_offset, 0, qt, qh, kt, kh, vt, vh)
    _run(index, _lib.gdn_kv_append, dims, cache.struct, qp, k.data_ptr(), v.data_ptr(),
         _dense(q_weight, "q_weight", (d,), index, f32), _dense(k_weight, "k_weight", (d,), index, f32),
         _dense(inv_freq, "inv_freq", (rot // 2,), index, f32), _dense(position, "position", (T,), index, _int32),
         _dense(slot, "slot", (T,), index, _int32), op, raw)
    return q_out


def _table(table, index, B):
    if not isinstance(table, _Tensor):
        raise TypeError("table must be a torch tensor")
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError(f"table must have shape ({B}, pages), got {tuple(table.shape)}")
    if table.get_device() != index:
        raise ValueError(f"table must be on device {index}, got {table.device}")
    if table.dtype != _int32:
        raise TypeError(f"table must be {_int32}, got {table.dtype}")
    if table.shape[1] > 1 and table.stride(1) != 1:
        raise ValueError("table: the elements of a row must be dense")
    return table.data_ptr(), table.shape[1], (table.stride(0) if B > 1 else 0)


def _attend(fn, need_fn, cache, q, extra, B, T, table, length, scale, gate, o, seq_status, workspace, stream):
    """The calls' common part; q [rows][H_q][d], or [B][N][H_q][d] with dense rows of a tree."""
    index = cache.index
    shape = q.shape
    H_q, d = shape[-2:]
    tree = len(shape) == 4
    rows = shape[0] * shape[1] if tree else shape[0]
    if d != cache.d:
        raise ValueError(f"q must have heads of {cache.d} elements, got {d}")
    if q.get_device() != index:
        raise ValueError(f"q must be on device {index}, got {q.device}")
    if q.dtype != _bf16:
        raise TypeError(f"q must be {_bf16}, got {q.dtype}")
    st = q.stride()
    if q.is_contiguous():
        qs = H_q * d if rows > 1 else 0
    else:
        if st[-1] != 1 or (H_q > 1 and st[-2] != d):
            raise ValueError("q: the elements of a row must be dense")
        if tree and shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError("q: the nodes of all trees must be equally far apart")
        qs = 0 if rows <= 1 else st[0] if not tree or shape[1] == 1 else st[1]
    gs = gh = 0
    gp = None
    if gate is not None:
        if not isinstance(gate, _Tensor):
            raise TypeError("gate must be a torch tensor")
        if gate.shape != shape:
            raise ValueError(f"gate must have shape {tuple(shape)}, got {tuple(gate.shape)}")
        if gate.get_device() != index:
            raise ValueError(f"gate must be on device {index}, got {gate.device}")
        if gate.dtype != _bf16:
            raise TypeError(f"gate must be {_bf16}, got {gate.dtype}")
        zt = gate.stride()
        if zt[-1] != 1:
            raise ValueError("gate: the elements of a head must be dense")
        if tree and shape[0] > 1 and shape[1] > 1 and zt[0] != shape[1] * zt[1]:
            raise ValueError("gate: the nodes of all trees must be equally far apart")
        gs = 0 if rows <= 1 else zt[0] if not tree or shape[1] == 1 else zt[1]
        gh = zt[-2] if H_q > 1 else 0
        gp = gate.data_ptr()
    tp, pages, ts = _table(table, index, B)
    dims = AttnDims(B, T, H_q, pages, d ** -0.5 if scale is None else scale, 0, qs, gs, gh, ts)
    raw = _stream(stream, index)
    if o is None:
        o = _empty(q, shape, _bf16, index, raw, stream)
        op = o.data_ptr()
    else:
        op = _dense(o, "o", shape, index, _bf16)
    lp = _dense(length, "length", (B,), index, _int32)
    sp = _dense(seq_status, "seq_status", (B,), index, _int32)
    if workspace is None:
        need = need_fn(dims, cache.struct)
        if need:
            workspace = _empty(q, (need,), _torch.uint8, index, raw, stream, keep=False)
    wp, nbytes = (None, 0) if workspace is None else _workspace(workspace, index)
    _run(index, fn, dims, cache.struct, q.data_ptr(), *extra, tp, lp, gp, op, sp, wp, nbytes, raw)
    return o


def _query(q, dims):
    if not isinstance(q, _Tensor):
        raise TypeError("q must be a torch tensor")
    if q.dim() != dims:
        raise ValueError(f"q must have {dims} dimensions")


def gdn_attn_decode(cache, q, table, length, scale=None, gate=None, o=None, seq_status=None, workspace=None, stream=None):
    """One token per sequence: q [B][H_q][d] bfloat16 over tokens 0 ..
    length[b] - 1 of the cache, whose pages are table[b]; times
    sigmoid(gate) if there is a gate.  ``scale`` is d ** -0.5 unless given.
    Returns o [B][H_q][d] bfloat16.  ``workspace``: a uint8 device tensor of
    at least :func:`gdn_attn_workspace_bytes` bytes to allocate nothing here."""
    _cache(cache)
    _query(q, 3)
    return _attend(_lib.gdn_attn_decode, _lib.gdn_attn_decode_workspace_bytes, cache, q, (), q.shape[0], 0, table, length,
                   scale, gate, o, seq_status, workspace, stream)


def gdn_attn_prefill(cache, q, cu_seqlens, table, length, scale=None, gate=None, o=None, seq_status=None, workspace=None,
                     stream=None):
    """Packed prompts: rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q
    [T][H_q][d] are the last of the length[b] tokens that the cache holds of
    sequence b, and see the tokens up to their own.  Returns o [T][H_q][d]."""
    index = _cache(cache)
    _query(q, 3)
    if not isinstance(cu_seqlens, _Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor of 1 dimension, at least 1 long")
    B = cu_seqlens.shape[0] - 1
    cu = _dense(cu_seqlens, "cu_seqlens", (B + 1,), index, _int32)
    return _attend(_lib.gdn_attn_prefill, _lib.gdn_attn_prefill_workspace_bytes, cache, q, (cu,), B, q.shape[0], table,
                   length, scale, gate, o, seq_status, workspace, stream)


def gdn_attn_verify(cache, q, anc, table, length, scale=None, gate=None, o=None, seq_status=None, workspace=None,
                    stream=None):
    """Every node of a tree: q [B][N][H_q][d] over the prefix (tokens 0 ..
    length[b] - 1 of the cache) and the nodes (node i as token length[b] + i)
    whose bits anc [B][N][ceil(N / 32)] int32 has, as
    :func:`gdn_tree_ancestors` returns them.  Returns o [B][N][H_q][d]."""
    index = _cache(cache)
    _query(q, 4)
    B, N = q.shape[:2]
    bits = _dense(anc, "anc", (B, N, max((N + 31) // 32, 1)), index, _int32)
    return _attend(_lib.gdn_attn_verify, _lib.gdn_attn_verify_workspace_bytes, cache, q, (bits,), B, N, table, length,
                   scale, gate, o, seq_status, workspace, stream)


def gdn_attn_workspace_bytes(kind, cache, B, T, H_q, max_pages):
    """Bytes of workspace of a call of ``kind`` "decode", "prefill" or "verify"
    with B sequences, T rows of q (nodes of a tree) and a table of max_pages.
    A workspace of that many serves calls with fewer of them too (not one of 0
    bytes for trees)."""
    _cache(cache)
    need = {"decode": _lib.gdn_attn_decode_workspace_bytes, "prefill": _lib.gdn_attn_prefill_workspace_bytes,
            "verify": _lib.gdn_attn_verify_workspace_bytes}.get(kind)
    if need is None:
        raise ValueError('kind must be "decode", "prefill" or "verify"')
    return need(AttnDims(B, T, H_q, max_pages, 1.0, 0, 0, 0, 0, 0), cache.struct)


def gdn_kv_commit(caches, anc, accepted, table, length, new_length=None, seq_status=None, stream=None):
    """After a tree's verify: in all of ``caches`` (a GdnKvCache, or a list of
    equal ones; layers may share one) the keys and values of the path to node accepted[b] move to
    tokens length[b], length[b] + 1, ...; -1 moves nothing.  Returns
    new_length [B] int32: length[b] + tokens of the path."""
    caches = [caches] if isinstance(caches, GdnKvCache) else list(caches)
    if not caches:
        raise ValueError("caches must hold at least one GdnKvCache")
    index = _cache(caches[0])
    for cache in caches:
        if not isinstance(cache, GdnKvCache):
            raise TypeError("cache must be a GdnKvCache")
        if cache.index != index:
            raise ValueError("caches must be on one device")
    if not isinstance(anc, _Tensor) or anc.dim() != 3:
        raise ValueError("anc must be a tensor of 3 dimensions")
    B, N = anc.shape[:2]
    bits = _dense(anc, "anc", (B, N, max((N + 31) // 32, 1)), index, _int32)
    raw = _stream(stream, index)
    lp = _dense(length, "length", (B,), index, _int32)
    if new_length is None:
        new_length = _empty(length, (B,), _int32, index, raw, stream)
    tp, pages, ts = _table(table, index, B)
    structs = (KvCacheStruct * len(caches)).from_buffer_copy(b"".join([c.raw for c in caches]))
    _run(index, _lib.gdn_kv_commit, CommitDims(B, N, pages, 0, ts), structs, len(caches), bits,
         _dense(accepted, "accepted", (B,), index, _int32), tp, lp, _dense(new_length, "new_length", (B,), index, _int32),
         _dense(seq_status, "seq_status", (B,), index, _int32), raw)
    return new_length
