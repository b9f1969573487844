"""Thin Python binding of liblosa.so (include/losa.h).

Argument marshalling only: tensors supply device memory, the current torch
CUDA stream supplies the stream, and every step of the computation runs in
the library's kernels. There is no fallback: if liblosa.so is missing or
fails to load, importing this package raises.

    import block_sparse_attention_losa_b200 as losa
    o, lse, mass = losa.dense_mass(q, k, v, L, block)        # construction step
    pat = losa.select(mass, block, tau=0.99)                   # frozen pattern
    o2, lse2 = losa.sparse_attn(q2, k2, v2, L, pat)            # every later step

Training and the layout around it:

    rope = losa.Rope((T, H, W), dims=(44, 42, 42))             # axes of the token grid
    q, k, v = losa.rope_pack(xq, xk, xv, block, rope)          # [B, L, heads, d] -> packed
    pat.prepare_backward()                                     # once per pattern
    dq, dk, dv = losa.sparse_attn_bwd(q, k, v, o, lse, do, L, pat)
    dxq, dxk, dxv = losa.rope_unpack(dq, dk, dv, L, rope)      # packed -> [B, L, heads, d]

    out, state = losa.layer_attn(xq, xk, xv, rope, pat)        # the same in one call each way
    dxq, dxk, dxv = losa.layer_attn_bwd(dout, state)

rope_pack, sparse_attn, rope_unpack and layer_attn also take part in autograd:
on tensors that require gradients they return results with a graph, whose
backward pass makes the calls above (results written into tensors that the
caller gives stay outside it, and so do the masses and every lse).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblosa.so")

LOSA_BF16, LOSA_FP32 = 0, 1
LOSA_OK = 0
STATUS = {0: "LOSA_OK", -1: "LOSA_ERR_ARG", -2: "LOSA_ERR_CUDA", -3: "LOSA_ERR_NOMEM",
          -4: "LOSA_ERR_TIMEOUT", -5: "LOSA_ERR_MASS", -6: "LOSA_ERR_UNSUPPORTED"}

# Every symbol include/losa.h declares.
EXPORTS = ("losa_dense_mass", "losa_select", "losa_dense_mass_select", "losa_pattern_info",
           "losa_pattern_export",
           "losa_pattern_import", "losa_select_noalloc", "losa_sparse_attn", "losa_free",
           "losa_pattern_prepare_bwd", "losa_pattern_export_bwd", "losa_sparse_attn_bwd",
           "losa_sparse_attn_bwd_workspace", "losa_rope_pack", "losa_rope_unpack",
           "losa_check_status", "losa_selftest_wait", "losa_set_wait_limit", "losa_exp2_eval",
           "losa_strerror", "losa_version")
NOALLOC_MAX_ROWS = 65536  # LOSA_NOALLOC_MAX_ROWS


class LosaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} "
                         f"({_lib.losa_strerror(status).decode()})")


class PatternView(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("n_blocks", ctypes.c_int),
                ("block", ctypes.c_int), ("nnz", ctypes.c_int64),
                ("row_ptr", ctypes.c_void_p), ("col_idx", ctypes.c_void_p),
                ("retained_fx", ctypes.c_void_p), ("total_fx", ctypes.c_void_p),
                ("n_tiles", ctypes.c_int64), ("tile_entries", ctypes.c_int64),
                ("tile_ptr", ctypes.c_void_p), ("tile_entry", ctypes.c_void_p),
                ("tile_order", ctypes.c_void_p)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int), ("grid", ctypes.c_int * 3), ("dim", ctypes.c_int * 3),
                ("start", ctypes.c_int * 3), ("scale", ctypes.c_double * 3),
                ("theta", ctypes.c_double), ("n_text", ctypes.c_int), ("pairing", ctypes.c_int)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python block_sparse_attention_losa_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, f64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double
    lib.losa_dense_mass.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32,
                                    vp, i32, vp, vp, vp]
    lib.losa_dense_mass.restype = i32
    lib.losa_select.argtypes = [vp, i32, i32, i32, i32, f64, ctypes.POINTER(vp), vp]
    lib.losa_select.restype = i32
    lib.losa_dense_mass_select.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32,
                                           f64, vp, i32, vp, vp, ctypes.POINTER(vp), vp]
    lib.losa_dense_mass_select.restype = i32
    lib.losa_pattern_info.argtypes = [vp, ctypes.POINTER(PatternView)]
    lib.losa_pattern_info.restype = i32
    lib.losa_pattern_export.argtypes = [vp] * 9
    lib.losa_pattern_export.restype = i32
    lib.losa_pattern_import.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32,
                                        ctypes.POINTER(vp), vp]
    lib.losa_pattern_import.restype = i32
    i64 = ctypes.c_int64
    lib.losa_select_noalloc.argtypes = [vp, i32, i32, i32, f64, vp, vp, i64, vp, vp, vp]
    lib.losa_select_noalloc.restype = i32
    lib.losa_sparse_attn.argtypes = [vp, vp, vp, i32, i32, i32, f32, vp, vp, i32, vp, vp]
    lib.losa_sparse_attn.restype = i32
    lib.losa_pattern_prepare_bwd.argtypes = [vp, vp]
    lib.losa_pattern_prepare_bwd.restype = i32
    lib.losa_pattern_export_bwd.argtypes = [vp, ctypes.POINTER(i64), vp, vp, vp, vp]
    lib.losa_pattern_export_bwd.restype = i32
    lib.losa_sparse_attn_bwd.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, f32, vp,
                                         vp, vp, vp, i32, vp, i64, vp]
    lib.losa_sparse_attn_bwd.restype = i32
    lib.losa_sparse_attn_bwd_workspace.argtypes = [vp, i32, i32, i32]
    lib.losa_sparse_attn_bwd_workspace.restype = i64
    spec = ctypes.POINTER(RopeSpec)
    lib.losa_rope_pack.argtypes = [vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, spec, vp, vp, vp,
                                   vp, i32, vp]
    lib.losa_rope_pack.restype = i32
    lib.losa_rope_unpack.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, spec, vp, vp, vp,
                                     vp, i32, vp, vp]
    lib.losa_rope_unpack.restype = i32
    lib.losa_free.argtypes = [vp]
    lib.losa_free.restype = None
    lib.losa_check_status.argtypes = [vp]
    lib.losa_check_status.restype = i32
    lib.losa_selftest_wait.argtypes = [i64, vp]
    lib.losa_selftest_wait.restype = i32
    lib.losa_set_wait_limit.argtypes = [i64]
    lib.losa_set_wait_limit.restype = i32
    lib.losa_exp2_eval.argtypes = [vp, vp, i64, vp]
    lib.losa_exp2_eval.restype = i32
    lib.losa_strerror.argtypes = [i32]
    lib.losa_strerror.restype = ctypes.c_char_p
    lib.losa_version.argtypes = []
    lib.losa_version.restype = ctypes.c_char_p
    return lib


_lib = _load()


def lib():
    return _lib


def _check(fn, status):
    if status != LOSA_OK:
        raise LosaError(fn, status)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code_of(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return LOSA_BF16
    if dtype == torch.float32:
        return LOSA_FP32
    raise TypeError(f"unsupported dtype {dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    return _dtype_code_of(t.dtype)


def _check_qkv(q, k, v):
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4):
            raise ValueError("q, k, v must be contiguous CUDA tensors [B, H, L_pad, d]")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share shape and dtype")


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def dense_mass(q, k, v, L, block, scale=None, out_dtype=torch.float32, o=None, lse=None,
               mass=None, stream=None):
    """Construction step: (o, lse, mass) with mass [B, H, n, n], n = L_pad/block.
    Outside autograd."""
    _check_qkv(q, k, v)
    B, H, Lp, d = q.shape
    n = Lp // block
    scale = default_scale(d) if scale is None else scale
    dev = q.device
    if o is None:
        o = torch.empty(B, H, Lp, d, device=dev, dtype=out_dtype)
    if lse is None:
        lse = torch.empty(B, H, Lp, device=dev, dtype=torch.float32)
    if mass is None:
        mass = torch.empty(B, H, n, n, device=dev, dtype=torch.float32)
    st = _lib.losa_dense_mass(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), B, H,
                              int(L), Lp, d, int(block), float(scale), o.data_ptr(),
                              _dtype_code(o), lse.data_ptr(), mass.data_ptr(), _stream(stream))
    _check("losa_dense_mass", st)
    return o, lse, mass


class Pattern:
    """A frozen block pattern owned by the library (freed on close / GC)."""

    def __init__(self, handle, device):
        self._h = handle
        self.device = device
        v = PatternView()
        _check("losa_pattern_info", _lib.losa_pattern_info(handle, ctypes.byref(v)))
        self.B, self.H, self.n_blocks, self.block = v.B, v.H, v.n_blocks, v.block
        self.nnz, self.n_tiles, self.tile_entries = v.nnz, v.n_tiles, v.tile_entries
        self._view = v

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("pattern was freed")
        return self._h

    def close(self):
        if self._h is not None:
            _lib.losa_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prepare_backward(self, stream=None):
        """Builds the lists by key that sparse_attn_bwd walks: once, before
        the first backward step and outside any capture."""
        with torch.cuda.device(self.device):
            _check("losa_pattern_prepare_bwd",
                   _lib.losa_pattern_prepare_bwd(self.handle, _stream(stream)))
        return self

    def export_backward(self, stream=None):
        """Host copies of the lists by key: key_ptr, key_entry, key_order."""
        n = ctypes.c_int64()
        with torch.cuda.device(self.device):
            st = _lib.losa_pattern_export_bwd(self.handle, ctypes.byref(n), None, None, None,
                                              _stream(stream))
            _check("losa_pattern_export_bwd", st)
            out = {k: torch.empty(m, dtype=torch.int32) for k, m in
                   (("key_ptr", self.n_tiles + 1), ("key_entry", n.value),
                    ("key_order", self.n_tiles))}
            ptr = lambda t: t.data_ptr() if t.numel() else None
            st = _lib.losa_pattern_export_bwd(self.handle, None, *(ptr(t) for t in out.values()),
                                              _stream(stream))
            _check("losa_pattern_export_bwd", st)
        return out

    @property
    def rows(self):
        return self.B * self.H * self.n_blocks

    def density(self):
        return self.nnz / float(self.rows * self.n_blocks)

    def export(self, device=None, stream=None):
        """Copies of the pattern arrays as torch tensors (on `device`,
        default the pattern's device; 'cpu' gives host copies)."""
        device = self.device if device is None else torch.device(device)
        pin = device.type == "cpu"
        sizes = dict(row_ptr=(self.rows + 1, torch.int32), col_idx=(self.nnz, torch.int32),
                     retained_fx=(self.rows, torch.int64), total_fx=(self.rows, torch.int64),
                     tile_ptr=(self.n_tiles + 1, torch.int32),
                     tile_entry=(self.tile_entries, torch.int32),
                     tile_order=(self.n_tiles, torch.int32))
        out = {k: torch.empty(int(n), dtype=dt, device=device, pin_memory=pin)
               for k, (n, dt) in sizes.items()}
        ptr = lambda t: t.data_ptr() if t.numel() else None
        st = _lib.losa_pattern_export(self.handle, *(ptr(out[k]) for k in sizes),
                                      _stream(stream))
        _check("losa_pattern_export", st)
        return out


def select(mass, block, tau=0.99, stream=None):
    """Selection step: a Pattern from a [B, H, n, n] fp32 mass map."""
    if not (mass.is_cuda and mass.is_contiguous() and mass.dtype == torch.float32
            and mass.dim() == 4 and mass.shape[2] == mass.shape[3]):
        raise ValueError("mass must be a contiguous fp32 CUDA tensor [B, H, n, n]")
    B, H, n, _ = mass.shape
    h = ctypes.c_void_p()
    st = _lib.losa_select(mass.data_ptr(), B, H, n, int(block), float(tau), ctypes.byref(h),
                          _stream(stream))
    _check("losa_select", st)
    return Pattern(h, mass.device)


def dense_mass_select(q, k, v, L, block, tau=0.99, scale=None, out_dtype=torch.float32,
                      o=None, lse=None, mass=None, stream=None):
    """Construction and selection in one call, the per-row cut fused into
    the construction kernel: (o, lse, mass, Pattern), each as dense_mass and
    select would give them."""
    _check_qkv(q, k, v)
    B, H, Lp, d = q.shape
    n = Lp // block
    scale = default_scale(d) if scale is None else scale
    dev = q.device
    if o is None:
        o = torch.empty(B, H, Lp, d, device=dev, dtype=out_dtype)
    if lse is None:
        lse = torch.empty(B, H, Lp, device=dev, dtype=torch.float32)
    if mass is None:
        mass = torch.empty(B, H, n, n, device=dev, dtype=torch.float32)
    h = ctypes.c_void_p()
    st = _lib.losa_dense_mass_select(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q),
                                     B, H, int(L), Lp, d, int(block), float(scale), float(tau),
                                     o.data_ptr(), _dtype_code(o), lse.data_ptr(),
                                     mass.data_ptr(), ctypes.byref(h), _stream(stream))
    _check("losa_dense_mass_select", st)
    return o, lse, mass, Pattern(h, dev)


def import_pattern(row_ptr, col_idx, B, H, n_blocks, block, retained_fx=None, total_fx=None,
                   device=None, stream=None):
    """A Pattern from a stored host CSR (e.g. Pattern.export('cpu') of an
    earlier selection). Arrays are converted to contiguous host int32/int64."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("a pattern lives on a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    host = lambda t, dt: None if t is None else \
        torch.as_tensor(t).to("cpu", dtype=dt).contiguous()
    rp, ci = host(row_ptr, torch.int32), host(col_idx, torch.int32)
    rf, tf = host(retained_fx, torch.int64), host(total_fx, torch.int64)
    R = int(B) * int(H) * int(n_blocks)
    if rp.numel() != R + 1 or ci.numel() != int(rp[-1]) or \
            any(t is not None and t.numel() != R for t in (rf, tf)):
        raise ValueError("CSR array sizes do not match B * H * n_blocks")
    ptr = lambda t: None if t is None or t.numel() == 0 else t.data_ptr()
    h = ctypes.c_void_p()
    with torch.cuda.device(device):
        st = _lib.losa_pattern_import(ptr(rp), ptr(ci), ptr(rf), ptr(tf), int(B), int(H),
                                      int(n_blocks), int(block), ctypes.byref(h),
                                      _stream(stream))
    _check("losa_pattern_import", st)
    return Pattern(h, device)


def sparse_attn(q, k, v, L, pattern: Pattern, scale=None, out_dtype=torch.float32, o=None,
                lse=None, want_lse=True, stream=None):
    """Sparse step over a frozen pattern: (o, lse or None). Where autograd
    records it (and o and lse are not given), the backward pass is
    sparse_attn_bwd, without o and lse for fp32 q, k, v; the pattern must be
    prepared for it by then. lse carries no gradient."""
    if o is None and lse is None and _tracked(q, k, v):
        with _on(stream, q.device):
            o, lse = _SparseAttn.apply(q, k, v, L, pattern, scale, out_dtype)
        return o, lse if want_lse else None
    _check_qkv(q, k, v)
    B, H, Lp, d = q.shape
    if (B, H, Lp) != (pattern.B, pattern.H, pattern.n_blocks * pattern.block):
        raise ValueError("q/k/v shape does not match the pattern")
    scale = default_scale(d) if scale is None else scale
    if o is None:
        o = torch.empty(B, H, Lp, d, device=q.device, dtype=out_dtype)
    if lse is None and want_lse:
        lse = torch.empty(B, H, Lp, device=q.device, dtype=torch.float32)
    st = _lib.losa_sparse_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), d,
                               int(L), float(scale), pattern.handle, o.data_ptr(),
                               _dtype_code(o), lse.data_ptr() if lse is not None else None,
                               _stream(stream))
    _check("losa_sparse_attn", st)
    return o, lse


def _tracked(q, k, v):
    """Whether autograd records a call on these tensors (or None)."""
    return torch.is_grad_enabled() and (q is not None and q.requires_grad or
                                        k is not None and k.requires_grad or
                                        v is not None and v.requires_grad)


def _adjacent(t):
    """t, or a copy of it whose features are adjacent in memory."""
    return t if t is None or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _wanted(ctx, grads):
    """The gradients of the first inputs, those that autograd asked for."""
    return [g if n else None for g, n in zip(grads, ctx.needs_input_grad)]


class _SparseAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, L, pattern, scale, out_dtype):
        o, lse = sparse_attn(q, k, v, L, pattern, scale=scale, out_dtype=out_dtype)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.call = L, pattern, scale
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, do, _):
        q, k, v, o, lse = ctx.saved_tensors
        if q.dtype == torch.float32:
            o = lse = None
        L, pattern, scale = ctx.call
        grads = sparse_attn_bwd(q, k, v, o, lse, do.contiguous(), L, pattern, scale=scale)
        return (*_wanted(ctx, grads), None, None, None, None)


def _on(stream, device):
    """The context of a call's own allocations and launch: `device`, and
    `stream` if one is given, so that a workspace freed on return is reused in
    that stream's order. Nothing to enter in the usual case."""
    if device.index is None:
        raise ValueError("tensors must be on a CUDA device")
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    if stream is None and device.index == torch._C._cuda_getDevice():
        return _HERE_AND_NOW
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


_HERE_AND_NOW = contextlib.nullcontext()


def _raw_stream(stream, device):
    """The cudaStream_t of `stream`, by default the device's current one."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def sparse_attn_bwd(q, k, v, o, lse, do, L, pattern: Pattern, scale=None, out_dtype=None,
                    dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of sparse_attn over the same pattern, which
    pattern.prepare_backward() has been called on: o and lse are what the
    forward call returned for q, k, v, do is the gradient of o. The results
    have q's dtype unless out_dtype or the outputs say otherwise. Rows >= L of
    the inputs are not used; those of the results are 0. For fp32 q, k, v both
    o and lse may be None: what is needed of them is then formed in fp32,
    without the forward call's tf32 roundings (see losa.h)."""
    _check_qkv(q, k, v)
    shape, device = q.shape, q.device
    B, H, Lp, d = shape
    if (B, H, Lp) != (pattern.B, pattern.H, pattern.n_blocks * pattern.block):
        raise ValueError("q/k/v shape does not match the pattern")
    if (o is None) != (lse is None) or (o is None and q.dtype != torch.float32):
        raise ValueError("o and lse must be given, or, for fp32 q, k, v, both left out")
    for name, t in (("o", o), ("do", do)):
        if t is not None and not (t.shape == shape and t.device == device and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor of q's shape and device")
    if lse is not None and not (lse.shape == shape[:3] and lse.dtype == torch.float32
                                and lse.device == device and lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor [B, H, L_pad] on q's device")
    if not device == k.device == v.device == pattern.device:
        raise ValueError("q, k, v and the pattern must be on one device")
    scale = default_scale(d) if scale is None else scale
    given = [t for t in (dq, dk, dv) if t is not None]
    if out_dtype is None:
        out_dtype = given[0].dtype if given else q.dtype
    for t in given:
        if not (t.shape == shape and t.dtype == out_dtype and t.device == device
                and t.is_contiguous()):
            raise ValueError("dq, dk, dv must be contiguous tensors of q's shape and device "
                             "and of one dtype")
    in_code, do_code = _dtype_code(q), _dtype_code(do)
    need = _lib.losa_sparse_attn_bwd_workspace(pattern.handle, in_code, do_code, d)
    if need < 0:
        _check("losa_sparse_attn_bwd_workspace", need)
    with _on(stream, device):
        if len(given) < 3:
            dq, dk, dv = (torch.empty_like(q, dtype=out_dtype) if t is None else t
                          for t in (dq, dk, dv))
        if workspace is None:
            workspace = torch.empty(need, device=device, dtype=torch.uint8)
        elif not (workspace.device == device and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous tensor on q's device")
        st = _lib.losa_sparse_attn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), in_code, _ptr(o),
            LOSA_FP32 if o is None else _dtype_code(o), _ptr(lse), do.data_ptr(), do_code, d, int(L), float(scale), pattern.handle,
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _dtype_code(dq), workspace.data_ptr(),
            workspace.nbytes, _raw_stream(stream, device))
    _check("losa_sparse_attn_bwd", st)
    return dq, dk, dv


class Rope:
    """Rotary positions over the axes of a token grid.

    grid    tokens along each axis, outermost first ((T, H, W) for video).
    dims    features that each axis turns, from feature 0 on; those past
            their sum are not turned.
    theta   pair i of an axis with n features turns by position *
            theta^(-2i/n).
    start   position of each axis's first token (a later chunk's offset).
    scale   factor on each axis's positions.
    n_text  leading tokens that are not turned. Text after the video's tokens:
            list positions per token (positions=), zeros for the text, which
            turn nothing.
    pairing "interleaved": features (2i, 2i + 1) of an axis turn together;
            "halves": (i, i + n/2).
    """

    def __init__(self, grid, dims, theta=10000.0, start=None, scale=None, n_text=0,
                 pairing="interleaved"):
        n = len(dims)
        start = (0,) * n if start is None else start
        scale = (1.0,) * n if scale is None else scale
        if not (1 <= n <= 3 and len(grid) == len(start) == len(scale) == n):
            raise ValueError("grid, dims, start and scale must have 1 to 3 axes each")
        if pairing not in ("interleaved", "halves"):
            raise ValueError("pairing must be 'interleaved' or 'halves'")
        if any(not -2**31 <= int(x) < 2**31 for x in (*grid, *dims, *start, n_text)):
            raise ValueError("grid, dims, start and n_text must fit into 32 bits")
        pad = lambda xs, fill: tuple(xs) + (fill,) * (3 - n)
        self.n_axes = n
        self.spec = RopeSpec(n, (ctypes.c_int * 3)(*map(int, pad(grid, 1))),
                             (ctypes.c_int * 3)(*map(int, pad(dims, 0))),
                             (ctypes.c_int * 3)(*map(int, pad(start, 0))),
                             (ctypes.c_double * 3)(*map(float, pad(scale, 1.0))), float(theta),
                             int(n_text), ("interleaved", "halves").index(pairing))
        self.ref = ctypes.byref(self.spec)


def _check_positions(positions, B, L, rope, device):
    if positions is None:
        return None
    if not (positions.device == device and positions.dtype == torch.int32
            and positions.is_contiguous() and positions.shape == (B, L, rope.n_axes)):
        raise ValueError("positions must be a contiguous int32 tensor [B, L, axes] on the "
                         "inputs' device")
    return positions.data_ptr()


def _same(name, tensors):
    """The first of a call's 4-dimensional tensors (None left out), after a
    check that all have its device, shape and dtype."""
    first = None
    for t in tensors:
        if t is None:
            continue
        if first is None:
            first = t
            if not (t.is_cuda and t.dim() == 4):
                raise ValueError(f"{name} must be CUDA tensors of 4 dimensions")
            shape, dtype, device = t.shape, t.dtype, t.device
        elif not (t.shape == shape and t.dtype == dtype and t.device == device):
            raise ValueError(f"{name} must be of one shape, dtype and device")
    if first is None:
        raise ValueError(f"one of {name} must be given")
    return first


_Strides = ctypes.c_int64 * 9


def _token_strides(tensors):
    """The (batch, token, head) strides of a call's three tensors."""
    flat = []
    for t in tensors:
        if t is None:
            flat += (0, 0, 0)
            continue
        b, l, h, f = t.stride()
        if f != 1 and t.shape[3] > 1:
            raise ValueError("features must be adjacent in memory (stride 1)")
        flat += (b, l, h)
    return _Strides(*flat)


_ptr = lambda t: None if t is None else t.data_ptr()


def _empty_each(tensors, shape, dtype, device):
    """A new tensor for each one given."""
    out, first = [], None
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        first = torch.empty(shape, dtype=dtype, device=device) if first is None \
            else torch.empty_like(first)
        out.append(first)
    return out


def rope_pack(q, k, v, block, rope: Rope, positions=None, out_dtype=None, out=None, stream=None):
    """Turns q and k [B, L, H, d] (any strides, features adjacent) by their
    tokens' positions and lays q, k, v out as the attention calls take them:
    [B, H, L_pad, d], L_pad the next multiple of `block`, padded rows 0. Any
    of the three may be None. positions: int32 [B, L, axes] instead of the
    rope's grid and start. out: the three tensors to write."""
    x = _same("q, k, v", (q, k, v))
    if block not in (32, 64, 128):
        raise ValueError("block must be 32, 64 or 128")
    Lp = -(-x.shape[1] // block) * block
    if out is None and _tracked(q, k, v):
        with _on(stream, x.device):
            return _RopePack.apply(q, k, v, Lp, rope, positions, out_dtype)
    return _pack(x, q, k, v, Lp, rope, positions, out_dtype, out, stream)


def _pack(x, q, k, v, Lp, rope, positions, out_dtype, out=None, stream=None):
    """rope_pack into tensors of Lp rows; x is the first of q, k, v given."""
    B, L, H, d = x.shape
    device, dtype = x.device, out_dtype or x.dtype
    strides = _token_strides((q, k, v))
    pos = _check_positions(positions, B, L, rope, device)
    with _on(stream, device):
        if out is None:
            out = _empty_each((q, k, v), (B, H, Lp, d), dtype, device)
        else:
            y = _same("out", out)
            if [t is None for t in (q, k, v)] != [t is None for t in out]:
                raise ValueError("out must have a tensor for each of q, k, v that is given")
            if y.device != device or y.shape != (B, H, Lp, d) or \
                    any(t is not None and not t.is_contiguous() for t in out) or \
                    (out_dtype is not None and y.dtype != out_dtype):
                raise ValueError("out must be contiguous [B, H, L_pad, d] tensors on the "
                                 "inputs' device")
            dtype = y.dtype
        st = _lib.losa_rope_pack(_ptr(q), _ptr(k), _ptr(v), _dtype_code(x), strides, B, H, L, Lp,
                                 d, rope.ref, pos, *[t if t is None else t.data_ptr() for t in out],
                                 _dtype_code_of(dtype), _raw_stream(stream, device))
    if st:
        _check("losa_rope_pack", st)
    return tuple(out)


def rope_unpack(q, k, v, L, rope: Rope, positions=None, out_dtype=None, out=None, stream=None):
    """The way back, and rope_pack's gradient: q, k, v [B, H, L_pad, d] to
    [B, L, H, d], q and k turned by the negative angle. Any of the three may
    be None (an attention output goes back as v alone). out: the tensors to
    write, of any strides with adjacent features."""
    x = _same("q, k, v", (q, k, v))
    if out is None and _tracked(q, k, v):
        with _on(stream, x.device):
            return _RopeUnpack.apply(q, k, v, int(L), rope, positions, out_dtype)
    B, H, Lp, d = x.shape
    L = int(L)
    if any(t is not None and not t.is_contiguous() for t in (q, k, v)):
        raise ValueError("q, k, v must be contiguous [B, H, L_pad, d]")
    device, dtype = x.device, out_dtype or x.dtype
    pos = _check_positions(positions, B, L, rope, device)
    with _on(stream, device):
        if out is None:
            out = _empty_each((q, k, v), (B, L, H, d), dtype, device)
        else:
            y = _same("out", out)
            if [t is None for t in (q, k, v)] != [t is None for t in out]:
                raise ValueError("out must have a tensor for each of q, k, v that is given")
            if y.device != device or y.shape != (B, L, H, d) or \
                    (out_dtype is not None and y.dtype != out_dtype):
                raise ValueError("out must be [B, L, H, d] tensors on the inputs' device")
            dtype = y.dtype
        st = _lib.losa_rope_unpack(_ptr(q), _ptr(k), _ptr(v), _dtype_code(x), B, H, L, Lp, d,
                                   rope.ref, pos, *map(_ptr, out), _dtype_code_of(dtype),
                                   _token_strides(out), _raw_stream(stream, device))
    _check("losa_rope_unpack", st)
    return tuple(out)


class _RopePack(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, Lp, rope, positions, out_dtype):
        x = _same("q, k, v", (q, k, v))
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.call = x.shape[1], rope, x.dtype
        return _pack(x, q, k, v, Lp, rope, positions, out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        L, rope, dtype = ctx.call
        grads = [None if g is None else g.contiguous() for g in _wanted(ctx, grads)]
        if any(g is not None for g in grads):
            grads = rope_unpack(*grads, L, rope, positions=ctx.saved_tensors[0], out_dtype=dtype)
        return (*grads, None, None, None, None)


class _RopeUnpack(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, L, rope, positions, out_dtype):
        x = _same("q, k, v", (q, k, v))
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.call = x.shape[2], rope, x.dtype
        return rope_unpack(q, k, v, L, rope, positions=positions, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        Lp, rope, dtype = ctx.call
        grads = [_adjacent(g) for g in _wanted(ctx, grads)]
        if any(g is not None for g in grads):
            grads = _pack(_same("gradients", grads), *grads, Lp, rope, ctx.saved_tensors[0], dtype)
        return (*grads, None, None, None, None)


class LayerState(NamedTuple):
    """What layer_attn keeps for layer_attn_bwd: packed Q, K, V and O, the row
    log-sum-exp and the call's settings."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    o: torch.Tensor
    lse: torch.Tensor
    L: int
    rope: Rope
    pattern: Pattern
    positions: torch.Tensor
    scale: float


def layer_attn(q, k, v, rope: Rope, pattern: Pattern, positions=None, scale=None, stream=None):
    """A later step's attention from a layer's projections to its output
    projection's input: q, k, v [B, L, H, d] (rope_pack's) are turned and
    packed, attend over the frozen pattern, and O returns to [B, L, H, d] in
    q's dtype. Returns (out, state); state is layer_attn_bwd's, which is also
    out's backward pass where autograd records the call."""
    if _tracked(q, k, v):
        keep = []
        with _on(stream, q.device):
            out = _LayerAttn.apply(q, k, v, rope, pattern, positions, scale, keep)
        return out, keep[0]
    L = q.shape[1]
    with _on(stream, q.device):
        qp, kp, vp = rope_pack(q, k, v, pattern.block, rope, positions=positions, stream=stream)
        # O stays fp32 for the backward pass, whose D = dO . O cancels against
        # dP; the layer's output is rounded once.
        o, lse = sparse_attn(qp, kp, vp, L, pattern, scale=scale, stream=stream)
        out = rope_unpack(None, None, o, L, rope, positions=positions, out_dtype=q.dtype,
                          stream=stream)[2]
    return out, LayerState(qp, kp, vp, o, lse, L, rope, pattern, positions, scale)


def layer_attn_bwd(dout, state: LayerState, out=None, stream=None):
    """Gradients of layer_attn's q, k, v [B, L, H, d] from dout, the gradient
    of its output (any strides, features adjacent). out: the three tensors to
    write, for instance views of one fused gradient."""
    s = state
    with _on(stream, dout.device):
        do = rope_pack(None, None, dout, s.pattern.block, s.rope, positions=s.positions,
                       stream=stream)[2]
        # fp32: the forward call's O and lse carry its tf32 roundings.
        o, lse = (None, None) if s.q.dtype == torch.float32 else (s.o, s.lse)
        grads = sparse_attn_bwd(s.q, s.k, s.v, o, lse, do, s.L, s.pattern, scale=s.scale,
                                stream=stream)
        return rope_unpack(*grads, s.L, s.rope, positions=s.positions, out=out, stream=stream)


class _LayerAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, rope, pattern, positions, scale, keep):
        out, state = layer_attn(q, k, v, rope, pattern, positions=positions, scale=scale)
        keep.append(state)
        ctx.save_for_backward(*state[:5], positions)
        ctx.call = state.L, rope, pattern, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        *packed, positions = ctx.saved_tensors
        L, rope, pattern, scale = ctx.call
        grads = layer_attn_bwd(_adjacent(dout),
                               LayerState(*packed, L, rope, pattern, positions, scale))
        return (*_wanted(ctx, grads), None, None, None, None, None)


def exp2_eval(x, stream=None):
    """2^x with the kernels' FMA-pipe exponential (diagnostic)."""
    if not (x.is_cuda and x.is_contiguous() and x.dtype == torch.float32):
        raise ValueError("x must be a contiguous fp32 CUDA tensor")
    y = torch.empty_like(x)
    _check("losa_exp2_eval", _lib.losa_exp2_eval(x.data_ptr(), y.data_ptr(), x.numel(),
                                                 _stream(stream)))
    return y


def check_status(stream=None):
    """Synchronises the stream and raises if a kernel reported a timeout."""
    _check("losa_check_status", _lib.losa_check_status(_stream(stream)))


def set_wait_limit(cycles: int = 0):
    """Wait limit of later attention launches in SM cycles (0 = default,
    about 2 s); a diagnostic of the kernels' failure path."""
    _check("losa_set_wait_limit", _lib.losa_set_wait_limit(int(cycles)))


def version() -> str:
    return _lib.losa_version().decode()
