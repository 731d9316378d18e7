"""Python binding of the C ABI (include/gbe_elementwise.h).

Argument marshalling only: each ``gbe_*`` function takes torch tensors that
live on the current CUDA device (or in pinned host memory, which the kernels
then read and write in place over the host link), checks that their shapes and dtypes
agree with one another, and passes their pointers, sizes and the current
stream to the C entry point of the same name.  Every step of every op runs
in the CUDA library; there is no other code path.  If the library is not
built, the first call raises :class:`LibraryMissing`.

The functions without the ``gbe_`` prefix (``rmsnorm``, ``rope``, ...) are
conveniences that allocate the outputs with torch and call the ``gbe_``
function.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libgbe_elementwise.so")

GBE_F32, GBE_BF16 = 0, 1
_DTYPES = {torch.float32: GBE_F32, torch.bfloat16: GBE_BF16}

_lib = None
_lock = threading.Lock()


class LibraryMissing(RuntimeError):
    pass


class GbeError(RuntimeError):
    def __init__(self, op: str, status: int, message: str, cuda_error: int = 0):
        super().__init__(f"{op}: status {status} ({message})"
                         + (f", cudaError {cuda_error}" if cuda_error else ""))
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (raises LibraryMissing when it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise LibraryMissing(
                    f"{LIB_PATH} is not built; run elementwise_row_rmsnorm_gb300.build() "
                    "(nvcc, sm_103a) first")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, f32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
            u64 = ctypes.c_uint64
            sigs = {
                "gbe_rmsnorm": [vp, vp, vp, i64, i64, f32, i32, vp],
                "gbe_add_rmsnorm": [vp, vp, vp, vp, vp, i64, i64, f32, i32, vp],
                "gbe_layernorm": [vp, vp, vp, vp, i64, i64, f32, i32, vp],
                "gbe_rope": [vp, vp, vp, i64, i64, i64, i64, vp, f32, i32, i32, vp],
                "gbe_rope_qk": [vp, vp, i64, i64, vp, vp, i64, i64, vp, i64, i64, i64, vp, vp, i64, f32, i32,
                                i32, vp],
                "gbe_rope_cos_sin": [vp, i64, i64, vp, vp],
                "gbe_rope_pair": [vp, vp, vp, i64, i64, i32, vp],
                "gbe_rope_multi": [vp, vp, vp, i64, i64, i64, i64, vp, vp, f32, i32, i32, vp],
                "gbe_qk_norm_rope": [vp, vp, i64, i64, vp, vp, vp, i64, i64, vp, f32, vp, i64, i64, i64, vp, vp,
                                     i64, f32, i32, i32, vp],
                "gbe_silu_mul": [vp, vp, vp, i64, i32, vp],
                "gbe_add": [vp, vp, vp, i64, i32, vp],
                "gbe_embedding": [vp, vp, vp, i64, i64, i64, vp, i32, vp],
                "gbe_argmax": [vp, vp, i64, i64, i32, vp],
                "gbe_sample": [vp, vp, vp, i64, i64, i32, f32, i64, f32, i32, vp],
                "gbe_sample_seeded": [vp, vp, i64, i64, i32, f32, i64, f32, u64, u64, i32, vp],
                "gbe_pcg64_uniforms": [vp, i64, u64, u64, vp],
                "gbe_kv_write": [vp, i64, vp, i64, vp, i64, vp, vp, i32, vp],
                "gbe_kv_read": [vp, i64, vp, i64, vp, i64, vp, vp, i32, vp],
                "gbe_attn_decode": [vp, i64, vp, i64, i64, i64, vp, vp, i64, vp, f32, vp, i64, i32, vp],
                "gbe_attn_decode_workspace": [i64, i64, i64, i64, i64, i64],
                "gbe_attn_prompt": [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, f32, i32, vp],
                "gbe_rope_kv_write": [vp, vp, i64, i64, vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i64, f32, i32, vp, vp,
                                      i32, vp],
                "gbe_attn_decode_window": [vp, i64, vp, i64, i64, i64, vp, vp, i64, vp, i64, i64, f32, vp, i64, i32, vp],
                "gbe_attn_decode_window_workspace": [i64, i64, i64, i64, i64, i64, i64, i64],
                "gbe_attn_prompt_window": [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, i64, i64, f32,
                                           i32, vp],
                "gbe_attn_chunk": [vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, i64, vp, i64, i64, f32, vp, i64, i32, vp],
                "gbe_attn_chunk_workspace": [i64, i64, i64, i64, i64, i64, i64, i64, i64],
                "gbe_version": [],
                "gbe_last_cuda_error": [],
                "gbe_status_string": [i32],
            }
            for name, args in sigs.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = (ctypes.c_char_p if name == "gbe_status_string" else
                              i64 if name.endswith("_workspace") else ctypes.c_int)
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gbe_status_string(status).decode()


def _check(op: str, st: int):
    if st != 0:
        L = lib()
        raise GbeError(op, st, status_string(st), L.gbe_last_cuda_error() if st == 11 else 0)


# The current stream's handle without building a torch Stream object per
# call (the private accessors torch's own extensions use; the public path
# where they are absent).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _cur_device is not None:
            return _raw_stream(_cur_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dt(*ts) -> int:
    dt = ts[0].dtype
    for t in ts:
        if t.dtype != dt:
            raise TypeError(f"all float tensors of one call share a dtype ({dt} vs {t.dtype})")
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")
    return _DTYPES[dt]


def _on_device(t) -> bool:
    """CUDA tensors, and pinned host tensors (mapped at the same address on the
    device, so kernels read and write them in place: zero-copy)."""
    return t.is_cuda or t.is_pinned()


def _dev(*ts):
    for t in ts:
        if not _on_device(t):
            raise ValueError("tensors must be on the CUDA device or in pinned host memory")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


# ---- the C entry points, one to one -----------------------------------------------

def gbe_rmsnorm(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, eps: float, stream=None) -> None:
    _dev(x, w, y)
    d = x.shape[-1]
    if y.shape != x.shape or w.numel() != d:
        raise ValueError("rmsnorm: y must match x and w must have x.shape[-1] entries")
    _check("gbe_rmsnorm", lib().gbe_rmsnorm(_ptr(x), _ptr(w), _ptr(y), x.numel() // d if d else 0, d,
                                            eps, _dt(x, w, y), _stream(stream)))


def gbe_layernorm(x, g, b, y, eps: float, stream=None) -> None:
    """b may be None (no bias)."""
    _dev(*[t for t in (x, g, b, y) if t is not None])
    d = x.shape[-1]
    if y.shape != x.shape or g.numel() != d or (b is not None and b.numel() != d):
        raise ValueError("layernorm: y matches x; g and b have x.shape[-1] entries")
    floats = [t for t in (x, g, b, y) if t is not None]
    _check("gbe_layernorm", lib().gbe_layernorm(_ptr(x), _ptr(g), _ptr(b), _ptr(y), x.numel() // d if d else 0, d,
                                                eps, _dt(*floats), _stream(stream)))


def gbe_add_rmsnorm(x, residual, w, y, h, eps: float, stream=None) -> None:
    _dev(x, residual, w, y, h)
    d = x.shape[-1]
    if not (residual.shape == y.shape == h.shape == x.shape) or w.numel() != d:
        raise ValueError("add_rmsnorm: x, residual, y, h must share a shape; w has x.shape[-1] entries")
    _check("gbe_add_rmsnorm", lib().gbe_add_rmsnorm(
        _ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(h), x.numel() // d if d else 0, d, eps,
        _dt(x, residual, w, y, h), _stream(stream)))


def gbe_rope(x, y, pos, inv_freq, r: int, mu: float = 1.0, layout: int = 0, stream=None) -> None:
    _dev(x, y, pos, inv_freq)
    if x.dim() != 3 or y.shape != x.shape:
        raise ValueError("rope: x is [T, H, D] and y matches it")
    T, H, D = x.shape
    if pos.dtype != torch.int32 or pos.numel() != T:
        raise ValueError("rope: pos is int32[T]")
    if inv_freq.dtype != torch.float32 or inv_freq.numel() < r // 2:
        raise ValueError("rope: inv_freq is float32[r/2]")
    _check("gbe_rope", lib().gbe_rope(_ptr(x), _ptr(y), _ptr(pos), T, H, D, r, _ptr(inv_freq), mu, layout,
                                      _dt(x, y), _stream(stream)))


def _rows_view(t: torch.Tensor, D: int, what: str):
    """(T, H, token stride) of a [T, H, D] view whose heads and entries are
    contiguous but whose tokens may be strided (a slice of a QKV buffer);
    `what` is the call that a refusal names."""
    shape, st = t.shape, t.stride()  # one query each (the per-call host cost matters at decode sizes)
    if len(shape) != 3 or shape[2] != D or st[2] != 1 or (shape[1] > 1 and st[1] != D):
        raise ValueError(f"{what}: operands are [T, H, D] views with contiguous heads")
    return shape[0], shape[1], st[0] if shape[0] > 1 else shape[1] * D


def gbe_rope_qk(q, q_out, k, k_out, pos, inv_freq, r: int, mu: float = 1.0, layout: int = 0,
                cos_sin=None, stream=None) -> None:
    """q, k (and their outputs, which may be the same views): [T, H, D] views
    of one storage type whose token stride may exceed H * D."""
    ts = [t for t in (q, q_out, k, k_out, pos, inv_freq) if t is not None]
    for t in ts:
        if not _on_device(t):
            raise ValueError("tensors must be on the CUDA device or in pinned host memory")
    D = (q if q is not None else k).shape[2]
    T = (q if q is not None else k).shape[0]
    sides = []
    for x, y in ((q, q_out), (k, k_out)):
        if x is None:
            sides.append((None, None, 0, 0))
            continue
        Tx, H, sx = _rows_view(x, D, "rope_qk")
        _, _, sy = _rows_view(y, D, "rope_qk")
        if Tx != T or y.shape != x.shape or sx != sy:
            raise ValueError("rope_qk: an output has its input's shape and token stride")
        sides.append((x.data_ptr(), y.data_ptr(), sx, H))
    if pos.dtype != torch.int32 or pos.numel() != T or not pos.is_contiguous():
        raise ValueError("rope_qk: pos is int32[T]")
    if inv_freq.dtype != torch.float32 or inv_freq.numel() < r // 2:
        raise ValueError("rope_qk: inv_freq is float32[r/2]")
    cache_len = 0
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous() or (r and cos_sin.numel() % r):
            raise ValueError("rope_qk: cos_sin is float32[cache_len, r/2, 2]")
        cache_len = cos_sin.numel() // r if r else 0
    floats = [t for t in (q, q_out, k, k_out) if t is not None]
    (qx, qy, qs, hq), (kx, ky, ks, hk) = sides
    _check("gbe_rope_qk", lib().gbe_rope_qk(qx, qy, qs, hq, kx, ky, ks, hk, _ptr(pos), T, D, r, _ptr(inv_freq),
                                            _ptr(cos_sin), cache_len, mu, layout, _dt(*floats), _stream(stream)))


class RopeOperand(ctypes.Structure):
    """gbe_rope_operand of the C header."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("stride", ctypes.c_int64), ("H", ctypes.c_int64),
                ("r", ctypes.c_int64), ("inv_freq", ctypes.c_void_p), ("mu", ctypes.c_float), ("layout", ctypes.c_int)]


def gbe_rope_pair(a, b, pos, stream=None) -> None:
    """RoPE of two operands in one launch.  a and b (b may be None) are
    tuples (x, y, inv_freq, r, mu, layout): x and y [T, H, D] views with
    contiguous heads whose token stride may exceed H * D (y is x: in place),
    inv_freq float32[r/2]; the operands share pos (int32[T]), T, D and dtype."""
    ops, floats = [], []
    T = D = None
    for o in (a, b):
        if o is None:
            ops.append(None)
            continue
        x, y, inv_freq, r, mu, layout = o
        for t in (x, y, inv_freq):
            if not _on_device(t):
                raise ValueError("tensors must be on the CUDA device or in pinned host memory")
        D = x.shape[2] if D is None else D
        Tx, H, sx = _rows_view(x, D, "rope_pair")
        _, _, sy = _rows_view(y, D, "rope_pair")
        T = Tx if T is None else T
        if Tx != T or y.shape != x.shape or sx != sy:
            raise ValueError("rope_pair: the operands share T and D; an output has its input's shape and stride")
        if inv_freq.dtype != torch.float32 or inv_freq.numel() < r // 2 or not inv_freq.is_contiguous():
            raise ValueError("rope_pair: inv_freq is float32[r/2]")
        ops.append(RopeOperand(x.data_ptr(), y.data_ptr(), sx, H, r, inv_freq.data_ptr(), mu, layout))
        floats += [x, y]
    if ops[0] is None:
        raise ValueError("rope_pair: the first operand is required")
    if pos.dtype != torch.int32 or pos.numel() != T or not pos.is_contiguous() or not _on_device(pos):
        raise ValueError("rope_pair: pos is int32[T]")
    pa = ctypes.byref(ops[0])
    pb = ctypes.byref(ops[1]) if ops[1] is not None else None
    _check("gbe_rope_pair", lib().gbe_rope_pair(ctypes.cast(pa, ctypes.c_void_p), ctypes.cast(pb, ctypes.c_void_p)
                                                if pb is not None else None, _ptr(pos), T, D, _dt(*floats),
                                                _stream(stream)))


def gbe_qk_norm_rope(q, q_out, gq, k, k_out, gk, eps: float, pos, inv_freq, r: int, mu: float = 1.0,
                     layout: int = 0, cos_sin=None, stream=None) -> None:
    """QK-norm (per-head RMSNorm with gains gq / gk of head_dim entries), then
    RoPE; q, k and outputs as for gbe_rope_qk."""
    for t in (q, q_out, k, k_out, gq, gk, pos, inv_freq, cos_sin):
        if t is not None and not _on_device(t):
            raise ValueError("tensors must be on the CUDA device or in pinned host memory")
    ref = q if q is not None else k
    T, D = ref.shape[0], ref.shape[2]
    sides = []
    for x, y, g in ((q, q_out, gq), (k, k_out, gk)):
        if x is None:
            sides.append((None, None, None, 0, 0))
            continue
        Tx, H, sx = _rows_view(x, D, "qk_norm_rope")
        _, _, sy = _rows_view(y, D, "qk_norm_rope")
        if Tx != T or y.shape != x.shape or sx != sy:
            raise ValueError("qk_norm_rope: an output has its input's shape and token stride")
        if g is None or g.numel() != D or not g.is_contiguous() or g.dtype != x.dtype:
            raise ValueError("qk_norm_rope: each gain has head_dim entries of the operand's dtype")
        sides.append((x.data_ptr(), y.data_ptr(), g.data_ptr(), sx, H))
    if pos.dtype != torch.int32 or pos.numel() != T or not pos.is_contiguous():
        raise ValueError("qk_norm_rope: pos is int32[T]")
    if inv_freq.dtype != torch.float32 or inv_freq.numel() < r // 2:
        raise ValueError("qk_norm_rope: inv_freq is float32[r/2]")
    cache_len = 0
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous() or (r and cos_sin.numel() % r):
            raise ValueError("qk_norm_rope: cos_sin is float32[cache_len, r/2, 2]")
        cache_len = cos_sin.numel() // r if r else 0
    floats = [t for t in (q, q_out, k, k_out, gq, gk) if t is not None]
    (qx, qy, qg, qs, hq), (kx, ky, kg, ks, hk) = sides
    _check("gbe_qk_norm_rope", lib().gbe_qk_norm_rope(qx, qy, qs, hq, qg, kx, ky, ks, hk, kg, eps, _ptr(pos), T, D,
                                                      r, _ptr(inv_freq), _ptr(cos_sin), cache_len, mu, layout,
                                                      _dt(*floats), _stream(stream)))


def gbe_rope_multi(x, y, pos, dims, inv_freq, mu: float = 1.0, layout: int = 0, stream=None) -> None:
    """x, y: [T, H, D]; pos: int32 [T, A]; dims: A even slice widths (a host
    sequence); inv_freq: float32, the axes' frequencies concatenated."""
    _dev(x, y, pos, inv_freq)
    if x.dim() != 3 or y.shape != x.shape:
        raise ValueError("rope_multi: x is [T, H, D] and y matches it")
    T, H, D = x.shape
    dims_arr = (ctypes.c_int64 * max(1, len(dims)))(*[int(v) for v in dims])
    A = len(dims)
    if pos.dtype != torch.int32 or pos.numel() != T * A:
        raise ValueError("rope_multi: pos is int32[T, A]")
    if inv_freq.dtype != torch.float32 or inv_freq.numel() < sum(int(v) for v in dims) // 2:
        raise ValueError("rope_multi: inv_freq holds sum(dims)/2 float32 entries")
    _check("gbe_rope_multi", lib().gbe_rope_multi(_ptr(x), _ptr(y), _ptr(pos), T, H, D, A,
                                                  ctypes.cast(dims_arr, ctypes.c_void_p), _ptr(inv_freq), mu, layout,
                                                  _dt(x, y), _stream(stream)))


def gbe_rope_cos_sin(cos_sin, inv_freq, r: int, stream=None) -> None:
    _dev(cos_sin, inv_freq)
    if cos_sin.dtype != torch.float32 or (r and cos_sin.numel() % r) or inv_freq.dtype != torch.float32:
        raise ValueError("rope_cos_sin: cos_sin is float32[cache_len, r/2, 2], inv_freq float32[r/2]")
    cache_len = cos_sin.numel() // r if r else 0
    _check("gbe_rope_cos_sin", lib().gbe_rope_cos_sin(_ptr(cos_sin), cache_len, r, _ptr(inv_freq),
                                                      _stream(stream)))


def gbe_silu_mul(gate, up, y, stream=None) -> None:
    _dev(gate, up, y)
    if not (gate.shape == up.shape == y.shape):
        raise ValueError("silu_mul: gate, up, y must share a shape")
    _check("gbe_silu_mul", lib().gbe_silu_mul(_ptr(gate), _ptr(up), _ptr(y), gate.numel(),
                                              _dt(gate, up, y), _stream(stream)))


def gbe_add(a, b, y, stream=None) -> None:
    _dev(a, b, y)
    if not (a.shape == b.shape == y.shape):
        raise ValueError("add: a, b, y must share a shape")
    _check("gbe_add", lib().gbe_add(_ptr(a), _ptr(b), _ptr(y), a.numel(), _dt(a, b, y), _stream(stream)))


def gbe_embedding(table, ids, out, bad_id_count=None, stream=None) -> None:
    _dev(table, ids, out)
    if bad_id_count is not None:
        _dev(bad_id_count)
        if bad_id_count.dtype != torch.int32 or bad_id_count.numel() != 1:
            raise ValueError("embedding: bad_id_count is one int32")
    if table.dim() != 2 or ids.dtype != torch.int32:
        raise ValueError("embedding: table is [V, d], ids int32")
    V, d = table.shape
    if out.shape != (ids.numel(), d):
        raise ValueError("embedding: out is [n, d]")
    _check("gbe_embedding", lib().gbe_embedding(_ptr(table), _ptr(ids), _ptr(out), ids.numel(), d, V,
                                                _ptr(bad_id_count), _dt(table, out), _stream(stream)))


def gbe_argmax(x, out, stream=None) -> None:
    _dev(x, out)
    n = x.shape[-1]
    rows = math.prod(x.shape[:-1])
    if out.dtype != torch.int32 or out.numel() != rows:
        raise ValueError("argmax: out is int32 with one entry per row")
    _check("gbe_argmax", lib().gbe_argmax(_ptr(x), _ptr(out), rows, n, _dt(x), _stream(stream)))


SAMPLE_METHODS = {"greedy": 0, "temperature": 1, "top_k": 2, "top_p": 3, "min_p": 4}


def gbe_sample(x, u, out, method: str, temperature: float = 1.0, top_k: int = 1, p: float = 1.0,
               stream=None) -> None:
    """One draw per row of x [..., n] at the uniforms u (f32, one per row);
    `p` is top-p's mass or min-p's ratio.  u may be None for greedy."""
    if method not in SAMPLE_METHODS:
        raise ValueError(f"sample: method is one of {sorted(SAMPLE_METHODS)}")
    _dev(x, out)
    n = x.shape[-1]
    rows = math.prod(x.shape[:-1])
    if out.dtype != torch.int32 or out.numel() != rows:
        raise ValueError("sample: out is int32 with one entry per row")
    if u is not None:
        _dev(u)
        if u.dtype != torch.float32 or u.numel() != rows:
            raise ValueError("sample: u is float32 with one entry per row")
    _check("gbe_sample", lib().gbe_sample(_ptr(x), None if u is None else _ptr(u), _ptr(out), rows, n,
                                          SAMPLE_METHODS[method], temperature, top_k, p, _dt(x),
                                          _stream(stream)))


def gbe_sample_seeded(x, out, method: str, seed: int, offset: int = 0, temperature: float = 1.0, top_k: int = 1,
                      p: float = 1.0, stream=None) -> None:
    """One draw per row of x [..., n]; row r draws with the uniform of draw
    offset + r of the PCG64 stream seeded with `seed` (0 <= seed, offset < 2^64)."""
    if method not in SAMPLE_METHODS:
        raise ValueError(f"sample: method is one of {sorted(SAMPLE_METHODS)}")
    _dev(x, out)
    n = x.shape[-1]
    rows = math.prod(x.shape[:-1])
    if out.dtype != torch.int32 or out.numel() != rows:
        raise ValueError("sample: out is int32 with one entry per row")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("sample: seed and offset are unsigned 64-bit integers")
    _check("gbe_sample_seeded", lib().gbe_sample_seeded(_ptr(x), _ptr(out), rows, n, SAMPLE_METHODS[method],
                                                        temperature, top_k, p, seed, offset, _dt(x),
                                                        _stream(stream)))


def gbe_pcg64_uniforms(u, seed: int, offset: int = 0, stream=None) -> None:
    """u (float32, any shape) <- the uniforms of draws offset .. offset + u.numel() - 1."""
    _dev(u)
    if u.dtype != torch.float32:
        raise ValueError("pcg64_uniforms: u is float32")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("pcg64_uniforms: seed and offset are unsigned 64-bit integers")
    _check("gbe_pcg64_uniforms", lib().gbe_pcg64_uniforms(_ptr(u), u.numel(), seed, offset, _stream(stream)))


class _KvCacheStruct(ctypes.Structure):
    """gbe_kv_cache of the C header."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("Hkv", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("D", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_pack_cache = struct.Struct("@PPPPqqqqqi4x").pack
_KV_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}


class KvCache:
    """A paged key-value cache of one layer: k and v are [n_pages, Hkv,
    page_size, D] tensors (float32, bfloat16 or float8_e4m3fn) whose pages are
    contiguous and share a stride (the halves k = kv[:, 0], v = kv[:, 1] of one
    [n_pages, 2, Hkv, page_size, D] tensor will do); a float8_e4m3fn cache also
    has k_scale and v_scale, uint8 [n_pages, Hkv, page_size].  Holds the
    tensors and the description of them that the library reads; the tensors
    cannot be exchanged (make another KvCache, it holds no state of its own)."""
    __slots__ = ("_tensors", "shape", "desc")

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        shape, kind = k.shape, _KV_DTYPES.get(k.dtype)
        if len(shape) != 4 or v.shape != shape or kind is None or v.dtype != k.dtype:
            raise ValueError("KvCache: k and v are [n_pages, Hkv, page_size, D], float32, bfloat16 or float8_e4m3fn")
        N, H, P, D = shape
        stride = H * P * D
        if not (k.is_contiguous() and v.is_contiguous()):
            st = k.stride()
            if N <= 1 or v.stride() != st or st[1:] != (P * D, D, 1):
                raise ValueError("KvCache: the pages of k and v are contiguous and share a stride")
            stride = st[0]
        if kind == 2:
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.uint8 or s.shape != (N, H, P) or not s.is_contiguous():
                    raise ValueError("KvCache: a float8_e4m3fn cache has uint8 scales [n_pages, Hkv, page_size]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("KvCache: only a float8_e4m3fn cache has scales")
        if not (k.is_cuda and v.is_cuda and k_scale is None):
            _where(k, v, k_scale, v_scale)
        self._tensors, self.shape = (k, v, k_scale, v_scale), shape
        # the bytes of a gbe_kv_cache, which the library reads during the call
        self.desc = _pack_cache(k.data_ptr(), v.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
                                0 if v_scale is None else v_scale.data_ptr(), N, H, P, D, stride, kind)


def _where(*ts):
    """Every tensor given is one that the device can address."""
    for t in ts:
        if t is not None and not (t.is_cuda or t.is_pinned()):
            raise ValueError("tensors must be on the CUDA device or in pinned host memory")


def _kv_sides(what, k, v, cache, slots, bad):
    T, H, sk = _rows_view(k, cache.shape[3], what)
    if v.shape != k.shape or H != cache.shape[1]:
        raise ValueError(f"{what}: k and v are [T, Hkv, D] with the cache's Hkv and D")
    sv = sk if v.stride() == k.stride() else _rows_view(v, cache.shape[3], what)[2]
    if slots.dtype != torch.int32 or slots.numel() != T or not slots.is_contiguous():
        raise ValueError(f"{what}: slots is int32[T]")
    if bad is not None and (bad.dtype != torch.int32 or bad.numel() != 1):
        raise ValueError(f"{what}: bad_slot_count is one int32")
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and bad is None):
        _where(k, v, slots, bad)
    return (k.data_ptr(), sk, v.data_ptr(), sv, slots.data_ptr(), T, cache.desc, None if bad is None else bad.data_ptr(),
            _dt(k, v))


def gbe_kv_write(k, v, slots, cache: KvCache, bad_slot_count=None, stream=None) -> None:
    """k, v: [T, Hkv, D] views with contiguous heads (slices of a QKV buffer will do); slots: int32[T], page *
    page_size + row, -1 for a token that is not stored."""
    _check("gbe_kv_write", lib().gbe_kv_write(*_kv_sides("kv_write", k, v, cache, slots, bad_slot_count),
                                              _stream(stream)))


def gbe_kv_read(k, v, slots, cache: KvCache, bad_slot_count=None, stream=None) -> None:
    """k, v: [T, Hkv, D] outputs of the model's dtype, views with contiguous heads; slots as for gbe_kv_write."""
    _check("gbe_kv_read", lib().gbe_kv_read(*_kv_sides("kv_read", k, v, cache, slots, bad_slot_count),
                                            _stream(stream)))


def gbe_rope_kv_write(q, q_out, k, v, pos, slots, cache: KvCache, inv_freq, r: int, mu: float = 1.0, layout: int = 0,
                      cos_sin=None, bad_slot_count=None, stream=None) -> None:
    """q (may be None), q_out, pos, inv_freq, r, mu, layout, cos_sin as for gbe_rope_qk, k, v, slots and bad_slot_count
    as for gbe_kv_write: q_out is q rotated, and k rotated and v are stored; k is not changed."""
    kp, sk, vp, sv, slots_p, T, desc, bad, _ = _kv_sides("rope_kv_write", k, v, cache, slots, bad_slot_count)
    qp = op = None
    sq = Hq = 0
    if q is not None:
        Tq, Hq, sq = _rows_view(q, cache.shape[3], "rope_kv_write")
        if Tq != T or q_out.shape != q.shape or _rows_view(q_out, cache.shape[3], "rope_kv_write")[2] != sq:
            raise ValueError("rope_kv_write: q is [T, Hq, D], and q_out has its shape and token stride")
        qp, op = q.data_ptr(), q_out.data_ptr()
    if pos.dtype != torch.int32 or pos.numel() != T or not pos.is_contiguous():
        raise ValueError("rope_kv_write: pos is int32[T]")
    if inv_freq.dtype != torch.float32 or inv_freq.numel() < r // 2 or not inv_freq.is_contiguous():
        raise ValueError("rope_kv_write: inv_freq is float32[r/2]")
    cache_len = 0
    if cos_sin is not None:
        if cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous() or (r and cos_sin.numel() % r):
            raise ValueError("rope_kv_write: cos_sin is float32[cache_len, r/2, 2]")
        cache_len = cos_sin.numel() // r if r else 0
    _where(q, q_out, pos, inv_freq, cos_sin)
    dtype = _dt(k, v) if q is None else _dt(q, q_out, k, v)
    _check("gbe_rope_kv_write", lib().gbe_rope_kv_write(
        qp, op, sq, Hq, kp, sk, vp, sv, pos.data_ptr(), slots_p, T, r, inv_freq.data_ptr(), _ptr(cos_sin), cache_len, mu,
        layout, desc, bad, dtype, _stream(stream)))


def attn_decode_workspace(B: int, Hq: int, cache: KvCache, max_pages: int, window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace of gbe_attn_decode (of gbe_attn_decode_window, given a window) for B sequences of at most
    max_pages pages."""
    _, H, P, D = cache.shape
    n = lib().gbe_attn_decode_window_workspace(B, Hq, H, D, P, max_pages, window, sinks)
    if n < 0:
        raise ValueError("attn_decode: sizes out of range (Hq a multiple of Hkv, D a multiple of 8 up to 256, ...)")
    return n


def _decode_sides(what, q, out, cache, table, lens, workspace):
    B, Hq, sq = _rows_view(q, cache.shape[3], what)
    if out.shape != q.shape:
        raise ValueError(f"{what}: out has q's shape")
    so = sq if out.stride() == q.stride() else _rows_view(out, cache.shape[3], what)[2]
    rows = table.shape
    if table.dtype != torch.int32 or len(rows) != 2 or rows[0] != B or not table.is_contiguous():
        raise ValueError(f"{what}: table is int32[B, max_pages]")
    if lens.dtype != torch.int32 or lens.numel() != B or not lens.is_contiguous():
        raise ValueError(f"{what}: lens is int32[B]")
    if not (q.is_cuda and out.is_cuda and table.is_cuda and lens.is_cuda):
        _where(q, out, table, lens)
    at, room = _room(workspace)
    return (q.data_ptr(), sq, out.data_ptr(), so, B, Hq, cache.desc, table.data_ptr(), rows[1], lens.data_ptr()), at, room


def _room(workspace):
    if workspace is None:
        return None, 0
    _dev(workspace)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gbe_attn_decode(q, out, cache: KvCache, table, lens, scale: float, workspace=None, stream=None) -> None:
    """q, out: [B, Hq, D]; table: int32[B, max_pages]; lens: int32[B], the new token included; workspace: any tensor
    of attn_decode_workspace bytes (None when that is 0)."""
    args, at, room = _decode_sides("attn_decode", q, out, cache, table, lens, workspace)
    _check("gbe_attn_decode", lib().gbe_attn_decode(*args, scale, at, room, _dt(q, out), _stream(stream)))


def gbe_attn_decode_window(q, out, cache: KvCache, table, lens, window: int, sinks: int, scale: float, workspace=None,
                           stream=None) -> None:
    """As gbe_attn_decode, of the last `window` tokens (0: all) and the first `sinks`; workspace: attn_decode_workspace
    bytes for them."""
    args, at, room = _decode_sides("attn_decode_window", q, out, cache, table, lens, workspace)
    _check("gbe_attn_decode_window", lib().gbe_attn_decode_window(*args, window, sinks, scale, at, room, _dt(q, out),
                                                                  _stream(stream)))


def attn_chunk_workspace(n_seqs: int, T: int, Hq: int, cache: KvCache, max_pages: int, window: int = 0,
                         sinks: int = 0) -> int:
    """Bytes of workspace of gbe_attn_chunk for T new tokens of n_seqs sequences of at most max_pages pages: they go by
    max_pages, not by lengths, so a table cut to the longest sequence's pages needs fewer."""
    _, H, P, D = cache.shape
    n = lib().gbe_attn_chunk_workspace(n_seqs, T, Hq, H, D, P, max_pages, window, sinks)
    if n < 0:
        raise ValueError("attn_chunk: sizes out of range (Hq a multiple of Hkv, D a multiple of 8 up to 256, ...)")
    return n


def gbe_attn_chunk(q, out, cache: KvCache, starts, table, lens, scale: float, window: int = 0, sinks: int = 0,
                   workspace=None, stream=None) -> None:
    """q, out: [T, Hq, D] views with contiguous heads, the new tokens packed; starts: int32[n_seqs + 1]; table:
    int32[n_seqs, max_pages]; lens: int32[n_seqs], the new tokens included; window 0: none; workspace: any tensor of
    attn_chunk_workspace bytes (None when that is 0).  Rows outside [starts[0], starts[-1]) of out are left as they
    were."""
    D = cache.shape[3]
    T, Hq, sq = _rows_view(q, D, "attn_chunk")
    if out.shape != q.shape:
        raise ValueError("attn_chunk: out has q's shape")
    so = sq if out.stride() == q.stride() else _rows_view(out, D, "attn_chunk")[2]
    n = lens.numel()
    if starts.dtype != torch.int32 or starts.numel() != n + 1 or not starts.is_contiguous():
        raise ValueError("attn_chunk: starts is int32[n_seqs + 1]")
    if lens.dtype != torch.int32 or not lens.is_contiguous():
        raise ValueError("attn_chunk: lens is int32[n_seqs]")
    rows = table.shape
    if table.dtype != torch.int32 or len(rows) != 2 or rows[0] != n or not table.is_contiguous():
        raise ValueError("attn_chunk: table is int32[n_seqs, max_pages]")
    if not (q.is_cuda and out.is_cuda and starts.is_cuda and table.is_cuda and lens.is_cuda):
        _where(q, out, starts, table, lens)
    at, room = _room(workspace)
    _check("gbe_attn_chunk", lib().gbe_attn_chunk(
        q.data_ptr(), sq, out.data_ptr(), so, starts.data_ptr(), n, T, Hq, cache.desc, table.data_ptr(), rows[1],
        lens.data_ptr(), window, sinks, scale, at, room, _dt(q, out), _stream(stream)))


def _prompt_sides(what, q, k, v, out, starts):
    D = q.shape[-1]
    T, Hq, sq = _rows_view(q, D, what)
    Tk, Hkv, sk = _rows_view(k, D, what)
    Tv, Hv, sv = _rows_view(v, D, what)
    _, _, so = _rows_view(out, D, what)
    if Tk != T or Tv != T or Hv != Hkv or out.shape != q.shape:
        raise ValueError(f"{what}: q and out are [T, Hq, D], k and v [T, Hkv, D]")
    if starts.dtype != torch.int32 or starts.numel() < 1 or not starts.is_contiguous():
        raise ValueError(f"{what}: starts is int32[n_seqs + 1]")
    _where(q, k, v, out, starts)
    return (q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, out.data_ptr(), so, starts.data_ptr(),
            starts.numel() - 1, T, Hq, Hkv, D)


def gbe_attn_prompt(q, k, v, out, starts, scale: float, stream=None) -> None:
    """q, out: [T, Hq, D], k, v: [T, Hkv, D] views with contiguous heads; starts: int32[n_seqs + 1]; rows outside
    [starts[0], starts[-1]) of out are left as they were."""
    _check("gbe_attn_prompt", lib().gbe_attn_prompt(*_prompt_sides("attn_prompt", q, k, v, out, starts), scale,
                                                    _dt(q, k, v, out), _stream(stream)))


def gbe_attn_prompt_window(q, k, v, out, starts, window: int, sinks: int, scale: float, stream=None) -> None:
    """As gbe_attn_prompt, a row seeing the last `window` rows up to itself (0: all) and the first `sinks`."""
    _check("gbe_attn_prompt_window", lib().gbe_attn_prompt_window(
        *_prompt_sides("attn_prompt_window", q, k, v, out, starts), window, sinks, scale, _dt(q, k, v, out),
        _stream(stream)))


# ---- conveniences that allocate the outputs -------------------------------------------

def _scratch(stream, shape, dtype, device):
    """Uninitialised memory that work on `stream` (None: the current one) writes first.  It comes from that stream's own
    pool, so that what held the memory before and what will after are in order with the call."""
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)  # (an ExternalStream of 0 would be a new stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty(stream, shape, dtype, device):
    """Such memory for an output: the stream that is current may use it too, once it waits for `stream`, and it is handed
    out again only when both are done with it."""
    t = _scratch(stream, shape, dtype, device)
    if stream is not None and t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _like(x: torch.Tensor, stream):
    """A contiguous output of x's shape, type and device."""
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _empty(stream, x.shape, x.dtype, x.device)


def kv_cache(n_pages: int, Hkv: int, page_size: int, D: int, dtype=torch.bfloat16, device="cuda") -> KvCache:
    """A zeroed cache; dtype torch.float8_e4m3fn for the 8-bit one."""
    k, v = (torch.zeros((n_pages, Hkv, page_size, D), dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return KvCache(k, v)
    ks, vs = (torch.zeros((n_pages, Hkv, page_size), dtype=torch.uint8, device=device) for _ in range(2))
    return KvCache(k, v, ks, vs)


def kv_read(cache: KvCache, slots, dtype=None, stream=None):
    """(k, v), each [T, Hkv, D], of the slots; dtype: the cache's own unless it is 8-bit (then bfloat16)."""
    if dtype is None:
        dtype = torch.bfloat16 if cache.k.dtype == torch.float8_e4m3fn else cache.k.dtype
    shape = (slots.numel(), cache.shape[1], cache.shape[3])
    k, v = (_empty(stream, shape, dtype, slots.device) for _ in range(2))
    gbe_kv_read(k, v, slots, cache, None, stream)
    return k, v


def attn_decode(q, cache: KvCache, table, lens, scale: float | None = None, workspace=None, stream=None):
    """[B, Hq, D]; allocates the workspace unless one is given."""
    out = _like(q, stream)
    if workspace is None:
        n = attn_decode_workspace(q.shape[0], q.shape[1], cache, table.shape[1])
        if n:
            workspace = _scratch(stream, n, torch.uint8, q.device)
    gbe_attn_decode(q, out, cache, table, lens, 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale, workspace,
                    stream)
    return out


def attn_prompt(q, k, v, starts, scale: float | None = None, stream=None):
    """[T, Hq, D]; rows outside [starts[0], starts[-1]) are not written."""
    out = _like(q, stream)
    gbe_attn_prompt(q, k, v, out, starts, 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale, stream)
    return out


def attn_decode_window(q, cache: KvCache, table, lens, window: int, sinks: int = 0, scale: float | None = None,
                       workspace=None, stream=None):
    """[B, Hq, D], of the last `window` tokens (0: all) and the first `sinks`; allocates the workspace unless one is
    given."""
    out = _like(q, stream)
    if workspace is None:
        n = attn_decode_workspace(q.shape[0], q.shape[1], cache, table.shape[1], window, sinks)
        if n:
            workspace = _scratch(stream, n, torch.uint8, q.device)
    gbe_attn_decode_window(q, out, cache, table, lens, window, sinks,
                           1.0 / math.sqrt(q.shape[-1]) if scale is None else scale, workspace, stream)
    return out


def attn_prompt_window(q, k, v, starts, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """[T, Hq, D], a row seeing the last `window` rows up to itself (0: all) and the first `sinks`; rows outside
    [starts[0], starts[-1]) are not written."""
    out = _like(q, stream)
    gbe_attn_prompt_window(q, k, v, out, starts, window, sinks, 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale,
                           stream)
    return out


def attn_chunk(q, cache: KvCache, starts, table, lens, scale: float | None = None, window: int = 0, sinks: int = 0,
               workspace=None, stream=None):
    """[T, Hq, D] of the new tokens packed in q; rows outside [starts[0], starts[-1]) are not written; allocates the
    workspace (attn_chunk_workspace bytes, many for a wide table) unless one is given.  The scale comes ahead of window
    and sinks here and behind them in attn_decode_window and attn_prompt_window: name them."""
    out = _like(q, stream)
    if workspace is None:
        n = attn_chunk_workspace(lens.numel(), q.shape[0], q.shape[1], cache, table.shape[1], window, sinks)
        if n:
            workspace = _scratch(stream, n, torch.uint8, q.device)
    gbe_attn_chunk(q, out, cache, starts, table, lens, 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale, window,
                   sinks, workspace, stream)
    return out


def rmsnorm(x, w, eps: float = 1e-5, out=None, stream=None):
    y = _like(x, stream) if out is None else out
    gbe_rmsnorm(x, w, y, eps, stream)
    return y


def layernorm(x, g, b=None, eps: float = 1e-5, stream=None):
    y = _like(x, stream)
    gbe_layernorm(x, g, b, y, eps, stream)
    return y


def add_rmsnorm(x, residual, w, eps: float = 1e-5, stream=None):
    y, h = _like(x, stream), _like(x, stream)
    gbe_add_rmsnorm(x, residual, w, y, h, eps, stream)
    return y, h


def rope(x, pos, inv_freq, r: int, mu: float = 1.0, layout: int = 0, in_place: bool = False, stream=None):
    y = x if in_place else _like(x, stream)
    gbe_rope(x, y, pos, inv_freq, r, mu, layout, stream)
    return y


def rope_cos_sin(inv_freq, r: int, cache_len: int, stream=None):
    t = _empty(stream, (cache_len, r // 2, 2), torch.float32, inv_freq.device)
    gbe_rope_cos_sin(t, inv_freq, r, stream)
    return t


def silu_mul(gate, up, stream=None):
    y = _like(gate, stream)
    gbe_silu_mul(gate, up, y, stream)
    return y


def add(a, b, stream=None):
    y = _like(a, stream)
    gbe_add(a, b, y, stream)
    return y


def embedding(table, ids, bad_id_count=None, stream=None):
    out = _empty(stream, (ids.numel(), table.shape[1]), table.dtype, table.device)
    gbe_embedding(table, ids, out, bad_id_count, stream)
    return out


def argmax(x, stream=None):
    out = _empty(stream, x.shape[:-1], torch.int32, x.device)
    gbe_argmax(x, out, stream)
    return out


def sample_seeded(x, method: str, seed: int, offset: int = 0, temperature: float = 1.0, top_k: int = 1,
                  p: float = 1.0, stream=None):
    out = _empty(stream, x.shape[:-1], torch.int32, x.device)
    gbe_sample_seeded(x, out, method, seed, offset, temperature, top_k, p, stream)
    return out


def pcg64_uniforms(n: int, seed: int, offset: int = 0, device="cuda", stream=None):
    u = _empty(stream, n, torch.float32, device)
    gbe_pcg64_uniforms(u, seed, offset, stream)
    return u


def sample(x, u, method: str, temperature: float = 1.0, top_k: int = 1, p: float = 1.0, stream=None):
    out = _empty(stream, x.shape[:-1], torch.int32, x.device)
    gbe_sample(x, u, out, method, temperature, top_k, p, stream)
    return out
