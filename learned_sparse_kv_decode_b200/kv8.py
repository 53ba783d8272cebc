"""ctypes binding of include/lsa_kv8.h: the 8-bit K/V cache and its decode path.

As in ``abi``, every function has the name of the C entry point it calls and all work runs in the CUDA
kernels. Before the call it checks what the C side cannot see: types, shapes, strides and the device of
the tensors (``ValueError`` / ``TypeError``).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import abi
from .abi import LSA_BF16, LSA_HEAD_DIM, _check, lib

HEADER = os.path.join(os.path.dirname(abi.HEADER), "lsa_kv8.h")


class _Cache(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("scale_block", ctypes.c_int32),
                ("K8", ctypes.c_void_p), ("V8", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _Prep(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


def _signatures():
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    dp, cp, pp = ctypes.POINTER(abi._Dims), ctypes.POINTER(_Cache), ctypes.POINTER(_Prep)
    sig = {
        "lsa_kv8_workspace_size": [dp, cp, ctypes.POINTER(sz)],
        "lsa_qk_norm_rope": [dp, i32, pp, i64, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp],
        "lsa_kv8_append": [dp, cp, pp, i32, vp, i64, vp, i64, vp, vp, vp, sz, vp],
        "lsa_kv8_gather": [dp, cp, vp, vp, vp, vp, vp, sz, vp],
        "lsa_kv8_decode_attn": [dp, cp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "lsa_decode_step_kv8": [dp, cp, pp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_signatures()


def _view(address, n):
    """The n bytes at an address, for comparisons."""
    return (ctypes.c_char * n).from_address(address)


class _Shape:
    """What the checks need of a Dims, with the bytes of the lsa_dims and its arrays that it was worked out from."""

    def __init__(self, dims):
        c = self.c = dims.c
        if not 1 <= c.B <= abi.LSA_MAX_BATCH:
            raise abi.LsaError(abi.LSA_ERR_INVALID_ARG, "Dims")
        self.ptr = dims.ptr
        views = [_view(ctypes.addressof(c), ctypes.sizeof(c))]
        if c.chunk_offsets:
            views.append(_view(ctypes.addressof(c.chunk_offsets.contents), 8 * (c.B + 1)))
        if c.k_per_seq:
            views.append(_view(ctypes.addressof(c.k_per_seq.contents), 4 * c.B))
        views += views[:1] * (3 - len(views))
        self.v0, self.v1, self.v2 = views
        self.b0, self.b1, self.b2 = (v.raw for v in views)
        self.B, self.H, self.C = c.B, c.H, c.chunk_len
        self.dtype = torch.bfloat16 if c.kv_dtype == LSA_BF16 else torch.float32
        self.emb_dtype = torch.bfloat16 if c.emb_dtype == LSA_BF16 else torch.float32
        self.chunks = int(c.chunk_offsets[c.B]) if c.chunk_offsets else c.B * c.N
        self.kept = sum(c.k_per_seq[b] for b in range(c.B)) if c.k_per_seq else c.B * c.k


def _shape(dims):
    """The sizes that the C side will read from `dims`: worked out again when it was changed in place."""
    s = getattr(dims, "_kv8_shape", None)
    if s is None or s.c is not dims.c or s.v0.raw != s.b0 or s.v1.raw != s.b1 or s.v2.raw != s.b2:
        s = dims._kv8_shape = _Shape(dims)
    return s


def _where(index):
    return "the CPU" if index < 0 else f"cuda:{index}"


def _refuse(t, name, dtype, device):
    """Raise for a tensor of another type or place than the call needs."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on {_where(device)}, got one on {_where(t.get_device())}")


def _ptr(t, name, dtype, numel, device):
    """Data pointer of a contiguous tensor of `numel` elements on CUDA device `device`."""
    if t.dtype is dtype and t.get_device() == device and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")


def _opt(t, name, dtype, numel, device):
    return None if t is None else _ptr(t, name, dtype, numel, device)


def _rows(t, name, dtype, rows, heads, device):
    """(pointer, elements from one row to the next) of rows [...][heads][Dh] whose heads lie side by side."""
    if t.dtype is not dtype or t.get_device() != device:
        _refuse(t, name, dtype, device)
    shape, row = t.shape, heads * LSA_HEAD_DIM
    n = len(shape)
    if n < 3 or t.numel() != rows * row or shape[n - 1] != LSA_HEAD_DIM or shape[n - 2] != heads:
        raise ValueError(f"{name}: expected {rows} rows of [{heads}][{LSA_HEAD_DIM}], got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), row
    stride = t.stride()
    if stride[n - 1] != 1 or (heads > 1 and stride[n - 2] != LSA_HEAD_DIM):
        raise ValueError(f"{name}: the values of a row must lie side by side")
    step, span = row, 1
    for i in range(n - 3, -1, -1):
        size = shape[i]
        if size == 1:
            continue
        if span == 1:
            step = stride[i]
        elif stride[i] != step * span:
            raise ValueError(f"{name}: the rows must be evenly spaced")
        span *= size
    return t.data_ptr(), step


# The current stream's handle without building a Stream object (a third of a small call's time), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, device):
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _device(t):
    """Index of the tensor's CUDA device, which has to be the current one."""
    d = t.get_device()
    if d < 0:
        raise ValueError("expected CUDA tensors")
    if d != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{d}, but the current device is cuda:{torch.cuda.current_device()}")
    return d


def _ws(ws, device):
    if ws.get_device() != device:
        raise ValueError(f"ws: expected a tensor on {_where(device)}, got one on {_where(ws.get_device())}")
    if not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


class _Fixed:
    """Attributes are set once. The struct that a call takes holds addresses and sizes, which another value would leave as
    they are, while the memory behind them could go."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be changed: make a new {type(self).__name__}")
        super().__setattr__(name, value)


class Kv8Cache(_Fixed):
    """lsa_kv8_cache and the tensors it points to (kept alive with it).

    K8, V8: [sum N_b][n_kv_heads][chunk_len][Dh] float8_e4m3fn (or the same bytes as uint8);
    k_scale, v_scale: [sum N_b][n_kv_heads][chunk_len / scale_block] float32."""

    def __init__(self, dims, n_kv_heads, scale_block, K8, V8, k_scale, v_scale):
        s = _shape(dims)
        self.n_kv_heads, self.scale_block = int(n_kv_heads), int(scale_block)
        if self.n_kv_heads < 1 or self.scale_block < 1:
            raise abi.LsaError(abi.LSA_ERR_UNSUPPORTED, "Kv8Cache")
        self.chunks, self.C = s.chunks, s.C
        self.device = K8.get_device()
        if self.device < 0:
            raise ValueError("expected CUDA tensors")
        n = s.chunks * self.n_kv_heads * s.C
        ptrs = []
        for name, t in (("K8", K8), ("V8", V8)):
            ptrs.append(_ptr(t, name, torch.uint8 if t.dtype is torch.uint8 else torch.float8_e4m3fn,
                             n * LSA_HEAD_DIM, self.device))
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            ptrs.append(_ptr(t, name, torch.float32, n // self.scale_block, self.device))
        self.K8, self.V8, self.k_scale, self.v_scale = K8, V8, k_scale, v_scale
        self.c = _Cache(self.n_kv_heads, self.scale_block, *ptrs)
        self.ptr = ctypes.byref(self.c)

    def check(self, s):
        if s.chunks != self.chunks or s.C != self.C:
            raise ValueError(f"the cache holds {self.chunks} chunks of {self.C} tokens, the call's dims name "
                             f"{s.chunks} of {s.C}")
        return _device(self.K8)


def alloc_kv8_cache(dims, n_kv_heads, scale_block=64, device=None):
    """A zeroed 8-bit cache for ``dims``."""
    s = _shape(dims)
    if scale_block < 1 or s.C % scale_block:
        raise abi.LsaError(abi.LSA_ERR_UNSUPPORTED, "alloc_kv8_cache")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    codes = (s.chunks, n_kv_heads, s.C, LSA_HEAD_DIM)
    scales = (s.chunks, n_kv_heads, s.C // scale_block)
    k8, v8 = (torch.zeros(codes, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(scales, dtype=torch.float32, device=device) for _ in range(2))
    return Kv8Cache(dims, n_kv_heads, scale_block, k8, v8, ks, vs)


class QkPrep(_Fixed):
    """lsa_qk_prep and the tensors it points to (kept alive with it): inv_freq [rot_dim/2], q_weight and
    k_weight [Dh] float32; a weight of None leaves those rows without a norm."""

    def __init__(self, rot_dim, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False):
        ref = next((t for t in (inv_freq, q_weight, k_weight) if t is not None), None)
        self.device = None if ref is None else ref.get_device()
        if ref is not None and self.device < 0:
            raise ValueError("expected CUDA tensors")
        f32 = torch.float32
        self.tensors = (inv_freq, q_weight, k_weight)
        self.c = _Prep(int(rot_dim), int(bool(interleaved)), float(eps),
                       _opt(inv_freq, "inv_freq", f32, int(rot_dim) // 2, self.device),
                       _opt(q_weight, "q_weight", f32, LSA_HEAD_DIM, self.device),
                       _opt(k_weight, "k_weight", f32, LSA_HEAD_DIM, self.device))
        self.ptr = ctypes.byref(self.c)

    def check(self, device):
        if self.device is not None and self.device != device:
            raise ValueError(f"prep: expected tensors on {_where(device)}, got some on {_where(self.device)}")
        return self.ptr


def kv8_header_symbols() -> list:
    """Names of the entry points declared in include/lsa_kv8.h."""
    import re
    with open(HEADER) as f:
        return re.findall(r"LSA_API\s+[\w\s\*]*?\b(lsa_\w+)\s*\(", f.read())


def lsa_kv8_workspace_size(dims, cache) -> int:
    n = ctypes.c_size_t(0)
    _check(lib.lsa_kv8_workspace_size(dims.ptr, cache.ptr, ctypes.byref(n)), "lsa_kv8_workspace_size")
    return n.value


def lsa_qk_norm_rope(dims, prep, positions, q, k, q_out, k_out, stream=None) -> None:
    s = _shape(dims)
    d = _device(positions)
    n = positions.numel()
    qp = qs = kp = ks = qo = qos = ko = kos = hkv = None
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("q or k or both, each with its output")
    if q is not None:
        qp, qs = _rows(q, "q", s.dtype, n, s.H, d)
        qo, qos = _rows(q_out, "q_out", s.dtype, n, s.H, d)
    if k is not None:
        hkv = k.shape[-2] if k.dim() > 1 else 0
        kp, ks = _rows(k, "k", s.dtype, n, hkv, d)
        ko, kos = _rows(k_out, "k_out", s.dtype, n, hkv, d)
    _check(lib.lsa_qk_norm_rope(s.ptr, hkv or 1, prep.check(d), n, _ptr(positions, "positions", torch.int32, n, d),
                                qp, qs or 0, kp, ks or 0, qo, qos or 0, ko, kos or 0, _stream(stream, d)),
           "lsa_qk_norm_rope")


def lsa_kv8_append(dims, cache, prep, k, v, start, new_count, ws, stream=None) -> None:
    s = _shape(dims)
    d = cache.check(s)
    if k.dim() != 4 or k.shape[0] != s.B:
        raise ValueError(f"k: expected [{s.B}][n_new][{cache.n_kv_heads}][{LSA_HEAD_DIM}], got {tuple(k.shape)}")
    n = k.shape[1]
    kp, ks = _rows(k, "k", s.dtype, s.B * n, cache.n_kv_heads, d)
    vp, vs = _rows(v, "v", s.dtype, s.B * n, cache.n_kv_heads, d)
    wp, wn = _ws(ws, d)
    _check(lib.lsa_kv8_append(s.ptr, cache.ptr, None if prep is None else prep.check(d), n, kp, ks, vp, vs,
                              _opt(start, "start", torch.int32, s.B, d),
                              _opt(new_count, "new_count", torch.int32, s.B, d), wp, wn, _stream(stream, d)),
           "lsa_kv8_append")


def lsa_kv8_gather(dims, cache, chunk_ids, seq_len, K_res, V_res, ws, stream=None) -> None:
    s = _shape(dims)
    d = cache.check(s)
    n = (s.chunks if chunk_ids is None else s.kept) * s.C * cache.n_kv_heads * LSA_HEAD_DIM
    wp, wn = _ws(ws, d)
    _check(lib.lsa_kv8_gather(s.ptr, cache.ptr, _opt(chunk_ids, "chunk_ids", torch.int32, s.kept, d),
                              _opt(seq_len, "seq_len", torch.int32, s.B, d), _ptr(K_res, "K_res", s.dtype, n, d),
                              _ptr(V_res, "V_res", s.dtype, n, d), wp, wn, _stream(stream, d)), "lsa_kv8_gather")


def lsa_kv8_decode_attn(dims, cache, q, chunk_ids, kept_count, seq_len, out, lse, ws, stream=None) -> None:
    s = _shape(dims)
    d = cache.check(s)
    n = s.B * s.H
    wp, wn = _ws(ws, d)
    _check(lib.lsa_kv8_decode_attn(s.ptr, cache.ptr, _ptr(q, "q", s.dtype, n * LSA_HEAD_DIM, d),
                                   _opt(chunk_ids, "chunk_ids", torch.int32, s.kept, d),
                                   _opt(kept_count, "kept_count", torch.int32, s.B, d),
                                   _opt(seq_len, "seq_len", torch.int32, s.B, d),
                                   _ptr(out, "out", torch.float32, n * LSA_HEAD_DIM, d),
                                   _opt(lse, "lse", torch.float32, n, d), wp, wn, _stream(stream, d)),
           "lsa_kv8_decode_attn")


def lsa_decode_step_kv8(dims, cache, prep, q_emb, chunk_emb, q, k, v, seq_len, chunk_ids_out, out, lse, ws,
                        stream=None) -> None:
    s = _shape(dims)
    d = cache.check(s)
    n = s.B * s.H
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    qp, qs = _rows(q, "q", s.dtype, s.B, s.H, d)
    kp = ks = vp = vs = None
    if k is not None:
        kp, ks = _rows(k, "k", s.dtype, s.B, cache.n_kv_heads, d)
        vp, vs = _rows(v, "v", s.dtype, s.B, cache.n_kv_heads, d)
    wp, wn = _ws(ws, d)
    c = dims.c
    _check(lib.lsa_decode_step_kv8(s.ptr, cache.ptr, None if prep is None else prep.check(d),
                                   _ptr(q_emb, "q_emb", s.emb_dtype, s.B * c.Q * c.E, d),
                                   _ptr(chunk_emb, "chunk_emb", s.emb_dtype, s.chunks * c.E, d), qp, qs, kp, ks or 0,
                                   vp, vs or 0, _opt(seq_len, "seq_len", torch.int32, s.B, d),
                                   _ptr(chunk_ids_out, "chunk_ids_out", torch.int32, s.kept, d),
                                   _ptr(out, "out", torch.float32, n * LSA_HEAD_DIM, d),
                                   _opt(lse, "lse", torch.float32, n, d), wp, wn, _stream(stream, d)),
           "lsa_decode_step_kv8")
