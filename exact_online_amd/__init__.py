"""exact_online_amd -- exact online causal long convolution on AMD MI355X.

Thin ctypes binding over the C ABI of ``include/fi.h`` (``libfi.so``, HIP for
gfx950).  The functions keep the C names and only marshal arguments: device
pointers may be given as integers or as torch CUDA tensors, streams as
integers (hipStream_t) or torch streams.  Every step of the computation runs
in the library's HIP kernels; if ``libfi.so`` is missing this module raises at
import (build it with ``python exact_online_amd/build.py`` or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct
from pathlib import Path

__all__ = [
    "FI_F32", "FI_BF16", "FI_FEEDBACK_NONE", "FI_FEEDBACK_TANH",
    "FI_OK", "FI_ERR_INVALID", "FI_ERR_NOMEM", "FI_ERR_HIP", "FI_ERR_STATE", "FI_ERR_UNSUPPORTED",
    "FiError", "fi_config", "fi_tile", "fi_create", "fi_step", "fi_run_closed_loop", "fi_reset",
    "fi_destroy", "fi_position", "fi_strerror", "fi_tile_at", "fi_run_prompted", "fi_conv_static", "Mixer",
    "fi_stack_config", "fi_stack_create", "fi_stack_run", "fi_stack_destroy", "Stack", "EXPORTS", "lib",
    "LIB_PATH", "FI_ACT_GELU", "FI_ACT_TANH", "FI_ACT_IDENTITY",
    "fi_view", "fi_lattn_config", "fi_lattn_args", "fi_lattn_create", "fi_lattn_prompt", "fi_lattn_step",
    "fi_lattn_destroy", "LinearAttention", "fi_dense_config", "fi_dense_args", "fi_dense_create", "fi_dense_run",
    "fi_dense_destroy", "Dense", "fi_scores_config", "fi_scores_args", "fi_scores_create", "fi_scores_run",
    "fi_scores_destroy", "TokenScores",
]

FI_F32, FI_BF16 = 0, 1
FI_FEEDBACK_NONE, FI_FEEDBACK_TANH = 0, 1
FI_DEFAULT_SMALL_TILE_MAX = 64
FI_MAX_L = 1 << 25
FI_OK, FI_ERR_INVALID, FI_ERR_NOMEM, FI_ERR_HIP, FI_ERR_STATE, FI_ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5

# EXACT_ONLINE_AMD_LIB may name another build of the same library (the
# phase-timing build libfi_prof.so, for bench.py --phases)
LIB_PATH = Path(os.environ.get("EXACT_ONLINE_AMD_LIB") or Path(__file__).resolve().parent / "libfi.so")
if not LIB_PATH.exists():
    raise ImportError(f"{LIB_PATH} is not built: run `python exact_online_amd/build.py` "
                      "(hipcc, gfx950) before using exact_online_amd")

# PyTorch, when installed, carries its own HIP runtime (same soname as the
# system one this library links).  Loaded first, torch's runtime is the one
# the library binds to, so the process has one runtime; the other order
# loads two, and whichever owns the device leaves the other without it.
try:
    import torch  # noqa: F401
except ImportError:
    pass

lib = ctypes.CDLL(str(LIB_PATH))

# every symbol include/fi.h declares
EXPORTS = ("fi_create", "fi_step", "fi_run_closed_loop", "fi_run_prompted", "fi_reset", "fi_destroy",
           "fi_position", "fi_strerror", "fi_tile_at", "fi_conv_static", "fi_stack_create", "fi_stack_run",
           "fi_stack_destroy", "fi_lattn_create", "fi_lattn_prompt", "fi_lattn_step", "fi_lattn_destroy",
           "fi_dense_create", "fi_dense_run", "fi_dense_destroy", "fi_scores_create", "fi_scores_run",
           "fi_scores_destroy")
FI_ACT_GELU, FI_ACT_TANH, FI_ACT_IDENTITY = 0, 1, 2
FI_STATIC_WORKSPACE_BYTES = 64 << 20


class fi_config(ctypes.Structure):
    # io_dtype is the C enum fi_dtype (int-sized)
    _fields_ = [("B", ctypes.c_int64), ("D", ctypes.c_int64), ("L", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("stream", ctypes.c_void_p),
                ("small_tile_max", ctypes.c_int32)]


class fi_stack_config(ctypes.Structure):
    # act is the C enum fi_activation (int-sized)
    _fields_ = [("B", ctypes.c_int64), ("D", ctypes.c_int64), ("L", ctypes.c_int64), ("M", ctypes.c_int64),
                ("act", ctypes.c_int32), ("stream", ctypes.c_void_p), ("small_tile_max", ctypes.c_int32)]


class fi_tile(ctypes.Structure):
    _fields_ = [("U", ctypes.c_int64), ("in_lo", ctypes.c_int64), ("in_hi", ctypes.c_int64),
                ("out_lo", ctypes.c_int64), ("out_hi", ctypes.c_int64)]


class fi_view(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("row", ctypes.c_int64), ("pos", ctypes.c_int64), ("head", ctypes.c_int64)]


class fi_lattn_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("L", ctypes.c_int64), ("H", ctypes.c_int64), ("Hkv", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("scale", ctypes.c_float),
                ("io_dtype", ctypes.c_int32), ("stream", ctypes.c_void_p)]


class fi_lattn_args(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("L", ctypes.c_int64), ("q", fi_view), ("k", fi_view), ("v", fi_view),
                ("o", fi_view), ("lens", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("n_slots", ctypes.c_int64),
                ("state", ctypes.c_void_p), ("fresh", ctypes.c_int32)]


class fi_dense_config(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("stream", ctypes.c_void_p)]


class fi_dense_args(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("bias", ctypes.c_void_p), ("res", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class fi_scores_config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("V", ctypes.c_int64), ("k", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("stream", ctypes.c_void_p)]


class fi_scores_args(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("targets", ctypes.c_void_p), ("logprob", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("top", ctypes.c_void_p), ("top_id", ctypes.c_void_p)]


_H = ctypes.c_void_p
lib.fi_create.argtypes = [ctypes.POINTER(fi_config), ctypes.c_void_p, ctypes.POINTER(_H)]
lib.fi_create.restype = ctypes.c_int
lib.fi_step.argtypes = [_H, ctypes.c_void_p, ctypes.c_void_p]
lib.fi_step.restype = ctypes.c_int
lib.fi_run_closed_loop.argtypes = [_H, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
lib.fi_run_closed_loop.restype = ctypes.c_int
lib.fi_run_prompted.argtypes = [_H, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
lib.fi_run_prompted.restype = ctypes.c_int
lib.fi_reset.argtypes = [_H]
lib.fi_reset.restype = ctypes.c_int
lib.fi_destroy.argtypes = [_H]
lib.fi_destroy.restype = None
lib.fi_position.argtypes = [_H]
lib.fi_position.restype = ctypes.c_int64
lib.fi_strerror.argtypes = [ctypes.c_int]
lib.fi_strerror.restype = ctypes.c_char_p
lib.fi_tile_at.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(fi_tile)]
lib.fi_tile_at.restype = ctypes.c_int
lib.fi_conv_static.argtypes = [ctypes.POINTER(fi_config), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                               ctypes.c_void_p, ctypes.c_void_p]
lib.fi_conv_static.restype = ctypes.c_int
lib.fi_stack_create.argtypes = [ctypes.POINTER(fi_stack_config), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.POINTER(_H)]
lib.fi_stack_create.restype = ctypes.c_int
lib.fi_stack_run.argtypes = [_H, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]
lib.fi_stack_run.restype = ctypes.c_int
lib.fi_stack_destroy.argtypes = [_H]
lib.fi_stack_destroy.restype = None
lib.fi_lattn_create.argtypes = [ctypes.POINTER(fi_lattn_config), ctypes.c_void_p, ctypes.POINTER(_H)]
lib.fi_lattn_create.restype = ctypes.c_int
lib.fi_lattn_prompt.argtypes = lib.fi_lattn_step.argtypes = [_H, ctypes.POINTER(fi_lattn_args)]
lib.fi_lattn_prompt.restype = lib.fi_lattn_step.restype = ctypes.c_int
lib.fi_dense_create.argtypes = [ctypes.POINTER(fi_dense_config), ctypes.POINTER(_H)]
lib.fi_dense_create.restype = ctypes.c_int
lib.fi_dense_run.argtypes = [_H, ctypes.POINTER(fi_dense_args)]
lib.fi_dense_run.restype = ctypes.c_int
lib.fi_scores_create.argtypes = [ctypes.POINTER(fi_scores_config), ctypes.POINTER(_H)]
lib.fi_scores_create.restype = ctypes.c_int
lib.fi_scores_run.argtypes = [_H, ctypes.POINTER(fi_scores_args)]
lib.fi_scores_run.restype = ctypes.c_int
for _f in (lib.fi_lattn_destroy, lib.fi_dense_destroy, lib.fi_scores_destroy):
    _f.argtypes, _f.restype = [_H], None
# only in the phase-timing build (include/fi_profile.h)
HAS_PROFILE = hasattr(lib, "fi_profile_read")
if HAS_PROFILE:
    lib.fi_profile_read.argtypes = [_H, ctypes.POINTER(ctypes.c_uint64), ctypes.c_int64]
    lib.fi_profile_read.restype = ctypes.c_int64


class FiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {fi_strerror(status)} ({status})")


def _check(status: int, where: str) -> int:
    if status < 0:
        raise FiError(status, where)
    return status


def _ptr(x) -> int:
    if x is None:
        return 0
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x)


def _stream(s) -> int:
    if s is None:
        return 0
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    return int(s)


def fi_strerror(status: int) -> str:
    return lib.fi_strerror(int(status)).decode()


def fi_create(cfg: fi_config, h) -> int:
    """Returns the handle (an integer); raises FiError on failure."""
    out = _H()
    _check(lib.fi_create(ctypes.byref(cfg), _ptr(h), ctypes.byref(out)), "fi_create")
    return int(out.value)


def fi_step(s: int, x_t, y_t) -> None:
    _check(lib.fi_step(s, _ptr(x_t), _ptr(y_t)), "fi_step")


def fi_run_closed_loop(s: int, x_in, fb: int, y, x_out=None) -> None:
    _check(lib.fi_run_closed_loop(s, _ptr(x_in), int(fb), _ptr(y), _ptr(x_out)), "fi_run_closed_loop")


def fi_run_prompted(s: int, x_prompt, p: int, y, x_out=None) -> None:
    _check(lib.fi_run_prompted(s, _ptr(x_prompt), int(p), _ptr(y), _ptr(x_out)), "fi_run_prompted")


def fi_reset(s: int) -> None:
    _check(lib.fi_reset(s), "fi_reset")


def fi_destroy(s) -> None:
    lib.fi_destroy(s)


def fi_position(s) -> int:
    return int(lib.fi_position(s))


def fi_tile_at(L: int, i: int) -> fi_tile:
    t = fi_tile()
    _check(lib.fi_tile_at(int(L), int(i), ctypes.byref(t)), "fi_tile_at")
    return t


def fi_conv_static(cfg: fi_config, h, x_in, fb: int, y, x_out=None) -> None:
    """The no-allocation one-shot run (fixed per-device workspace)."""
    _check(lib.fi_conv_static(ctypes.byref(cfg), _ptr(h), _ptr(x_in), int(fb), _ptr(y), _ptr(x_out)),
           "fi_conv_static")


def fi_stack_create(cfg: fi_stack_config, rho, w1, w2) -> int:
    out = _H()
    _check(lib.fi_stack_create(ctypes.byref(cfg), _ptr(rho), _ptr(w1), _ptr(w2), ctypes.byref(out)),
           "fi_stack_create")
    return int(out.value)


def fi_stack_run(s: int, x0, noise, sigma: float, y, x_out=None) -> None:
    _check(lib.fi_stack_run(s, _ptr(x0), _ptr(noise), float(sigma), _ptr(y), _ptr(x_out)), "fi_stack_run")


def fi_stack_destroy(s) -> None:
    lib.fi_stack_destroy(s)


class Stack:
    """Owning wrapper of one layer stack (marshalling only)."""

    def __init__(self, B, D, L, M, rho, w1, w2, act=FI_ACT_GELU, small_tile_max=0, stream=None):
        self.cfg = fi_stack_config(B=int(B), D=int(D), L=int(L), M=int(M), act=int(act), stream=_stream(stream),
                                   small_tile_max=int(small_tile_max))
        self.handle = fi_stack_create(self.cfg, rho, w1, w2)

    def run(self, x0, y, x_out=None, noise=None, sigma=0.0):
        fi_stack_run(self.handle, x0, noise, sigma, y, x_out)

    def close(self):
        if self.handle:
            fi_stack_destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _create(fn, where: str, *args) -> int:
    out = _H()
    _check(fn(*args, ctypes.byref(out)), where)
    return int(out.value)


def fi_lattn_create(cfg: fi_lattn_config, log_decay) -> int:
    return _create(lib.fi_lattn_create, "fi_lattn_create", ctypes.byref(cfg), _ptr(log_decay))


def fi_lattn_prompt(s: int, args: fi_lattn_args) -> None:
    _check(lib.fi_lattn_prompt(s, args), "fi_lattn_prompt")


def fi_lattn_step(s: int, args: fi_lattn_args) -> None:
    _check(lib.fi_lattn_step(s, args), "fi_lattn_step")


def fi_lattn_destroy(s) -> None:
    lib.fi_lattn_destroy(s)


def fi_dense_create(cfg: fi_dense_config) -> int:
    return _create(lib.fi_dense_create, "fi_dense_create", ctypes.byref(cfg))


def fi_dense_run(s: int, args: fi_dense_args) -> None:
    _check(lib.fi_dense_run(s, args), "fi_dense_run")


def fi_dense_destroy(s) -> None:
    lib.fi_dense_destroy(s)


def fi_scores_create(cfg: fi_scores_config) -> int:
    return _create(lib.fi_scores_create, "fi_scores_create", ctypes.byref(cfg))


def fi_scores_run(s: int, args: fi_scores_args) -> None:
    _check(lib.fi_scores_run(s, args), "fi_scores_run")


def fi_scores_destroy(s) -> None:
    lib.fi_scores_destroy(s)


class _Owner:
    """Owns one handle; `_destroy` frees it."""

    handle = 0

    def close(self):
        if self.handle:
            self._destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _refuse(where: str):
    raise FiError(FI_ERR_INVALID, where)


def _torch(name):
    import torch   # the callers' tensors are its, so it is there
    return getattr(torch, name)


def _io_type(dtype):
    """The tensors' type of an FI_* type (the create call refuses others)."""
    return {FI_F32: _torch("float32"), FI_BF16: _torch("bfloat16")}.get(int(dtype))


def _dense(x, dtype, n, where) -> int:
    """The address of an array of at least n elements; a tensor has to be dense, of this type and on the device.
    None and addresses are taken as they are."""
    if x is None:
        return 0
    if not hasattr(x, "data_ptr"):
        return int(x)
    if x.dtype is not dtype or not x.is_cuda or not x.is_contiguous() or x.numel() < n:
        _refuse(where)
    return x.data_ptr()


_LATTN_ARGS = struct.Struct("@2q" + "P3q" * 4 + "2PqPi4x")   # 4x: the trailing padding


class LinearAttention(_Owner):
    """Linear attention with a decay per head, over the caller's states
    (marshalling only).  q, k, v and o are tensors [B, L, heads, size] of the
    io type, of any strides as long as a head's elements are adjacent; state
    is [slots, Hkv, dk, dv], fp32 and contiguous, updated in place; lens and
    slots are int32 tensors [B] on the device, log_decay is fp32 [Hkv].  Other
    shapes, types, strides and tensors on the host are refused."""

    _destroy = staticmethod(fi_lattn_destroy)

    def __init__(self, B, L, H, Hkv, dk, dv, log_decay, scale=1.0, io_dtype=FI_BF16, stream=None):
        self.cfg = fi_lattn_config(B=int(B), L=int(L), H=int(H), Hkv=int(Hkv), dk=int(dk), dv=int(dv),
                                   scale=float(scale), io_dtype=int(io_dtype), stream=_stream(stream))
        self._is = (int(H), int(Hkv), int(dk), int(dv), _io_type(io_dtype), _torch("float32"), _torch("int32"))
        self._args = fi_lattn_args()
        self.handle = fi_lattn_create(self.cfg, _dense(log_decay, _torch("float32"), int(Hkv), "fi_lattn_create"))

    def _call(self, fn, where, q, k, v, o, state, lens, slots, fresh):
        shape = q.shape
        B, L = shape[0], shape[1]
        H, Hkv, dk, dv, io, f32, i32 = self._is
        qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), o.stride()
        if (shape != (B, L, H, dk) or k.shape != (B, L, Hkv, dk) or v.shape != (B, L, Hkv, dv)
                or o.shape != (B, L, H, dv) or (dk > 1 and (qs[3] != 1 or ks[3] != 1))
                or (dv > 1 and (vs[3] != 1 or os_[3] != 1))
                or q.dtype is not io or k.dtype is not io or v.dtype is not io or o.dtype is not io
                or not (q.is_cuda and k.is_cuda and v.is_cuda and o.is_cuda)):
            _refuse(where)
        n_slots = states = 0
        if state is not None:
            shape = state.shape
            n_slots = shape[0] if shape else 0
            if (shape != (n_slots, Hkv, dk, dv) or state.dtype is not f32 or not state.is_cuda
                    or not state.is_contiguous()):
                _refuse(where)
            states = state.data_ptr()
        # the struct's fields in their order (fi_lattn_args, native layout)
        _LATTN_ARGS.pack_into(
            self._args, 0, B, L, q.data_ptr(), qs[0], qs[1], qs[2], k.data_ptr(), ks[0], ks[1], ks[2],
            v.data_ptr(), vs[0], vs[1], vs[2], o.data_ptr(), os_[0], os_[1], os_[2],
            0 if lens is None else _dense(lens, i32, B, where), 0 if slots is None else _dense(slots, i32, B, where),
            n_slots, states, 1 if fresh else 0)
        status = fn(self.handle, self._args)
        if status < 0:
            raise FiError(status, where)

    def prompt(self, q, k, v, o, state=None, lens=None, slots=None, fresh=False):
        self._call(lib.fi_lattn_prompt, "fi_lattn_prompt", q, k, v, o, state, lens, slots, fresh)

    def step(self, q, k, v, o, state, slots=None):
        self._call(lib.fi_lattn_step, "fi_lattn_step", q, k, v, o, state, None, slots, False)


class Dense(_Owner):
    """y = act(x w^T + bias) + res over rows (marshalling only): x [M, K],
    w [N, K] and bias [N] of io_dtype, res and y [M, N] of out_dtype, rows of
    any stride.  Other shapes, types and tensors on the host are refused."""

    _destroy = staticmethod(fi_dense_destroy)

    def __init__(self, M, N, K, io_dtype=FI_BF16, out_dtype=FI_BF16, act=FI_ACT_IDENTITY, stream=None):
        self.cfg = fi_dense_config(M=int(M), N=int(N), K=int(K), io_dtype=int(io_dtype), out_dtype=int(out_dtype),
                                   act=int(act), stream=_stream(stream))
        self.N, self.K = int(N), int(K)
        self._io, self._out = _io_type(io_dtype), _io_type(out_dtype)
        self.handle = fi_dense_create(self.cfg)

    def run(self, x, w, y, bias=None, res=None):
        M, N, K = x.shape[0], self.N, self.K
        where = "fi_dense_run"
        xs, ws, ys = x.stride(), w.stride(), y.stride()
        if (x.shape != (M, K) or w.shape != (N, K) or y.shape != (M, N) or (K > 1 and (xs[1] != 1 or ws[1] != 1))
                or (N > 1 and ys[1] != 1) or x.dtype is not self._io or w.dtype is not self._io
                or y.dtype is not self._out or not (x.is_cuda and w.is_cuda and y.is_cuda)):
            _refuse(where)
        ldr = 0
        if res is not None:
            if res.shape != (M, N) or res.dtype is not self._out or not res.is_cuda:
                _refuse(where)
            ldr, inner = res.stride()
            if N > 1 and inner != 1:
                _refuse(where)
        ldx, ldw, ldy = xs[0], ws[0], ys[0]
        if M == 1:   # the stride of a single row is any number
            ldx, ldr, ldy = K, N, N
        if N == 1:
            ldw = K
        a = fi_dense_args(M, x.data_ptr(), ldx, w.data_ptr(), ldw, _dense(bias, self._io, N, where), _ptr(res), ldr,
                          y.data_ptr(), ldy)
        _check(lib.fi_dense_run(self.handle, a), where)


class TokenScores(_Owner):
    """Log probabilities of given tokens, entropies and the most probable
    tokens (marshalling only): logits [rows, V] with rows of any stride;
    targets int64 [rows]; logprob, entropy, lse fp32 [rows]; top fp32 and
    top_id int64 [rows, k], contiguous (or longer).  Outputs that are None are
    left out; other shapes, types, strides and tensors on the host are refused."""

    _destroy = staticmethod(fi_scores_destroy)

    def __init__(self, rows, V, k=0, io_dtype=FI_BF16, scale=1.0, stream=None):
        self.cfg = fi_scores_config(rows=int(rows), V=int(V), k=int(k), io_dtype=int(io_dtype), scale=float(scale),
                                    stream=_stream(stream))
        self.V, self.k = int(V), int(k)
        self._io, self._f32, self._i64 = _io_type(io_dtype), _torch("float32"), _torch("int64")
        self.handle = fi_scores_create(self.cfg)

    def run(self, logits, targets=None, logprob=None, entropy=None, top=None, top_id=None, lse=None):
        where, f32, i64 = "fi_scores_run", self._f32, self._i64
        rows = logits.shape[0]
        ld = logits.stride(0) if rows > 1 else self.V   # the stride of a single row is any number
        if (logits.shape != (rows, self.V) or (self.V > 1 and logits.stride(1) != 1) or logits.dtype is not self._io
                or not logits.is_cuda):
            _refuse(where)
        a = fi_scores_args(rows, logits.data_ptr(), ld, _dense(targets, i64, rows, where),
                           *(_dense(x, f32, rows, where) for x in (logprob, entropy, lse)),
                           _dense(top, f32, rows * self.k, where), _dense(top_id, i64, rows * self.k, where))
        _check(lib.fi_scores_run(self.handle, a), where)


def fi_profile_read(s: int):
    """Phase-timing build only: the last pass's record (a list of ints)."""
    if not HAS_PROFILE:
        raise RuntimeError(f"{LIB_PATH} is not the phase-timing build (libfi_prof.so)")
    n = _check(int(lib.fi_profile_read(s, (ctypes.c_uint64 * 1)(), 0)), "fi_profile_read")
    buf = (ctypes.c_uint64 * max(n, 1))()
    _check(int(lib.fi_profile_read(s, buf, n)), "fi_profile_read")
    return list(buf[:n])


def make_config(B: int, D: int, L: int, io_dtype: int = FI_F32, small_tile_max: int = 0,
                stream=None) -> fi_config:
    return fi_config(B=int(B), D=int(D), L=int(L), io_dtype=int(io_dtype), stream=_stream(stream),
                     small_tile_max=int(small_tile_max))


class Mixer:
    """Owning wrapper of one handle (marshalling only)."""

    def __init__(self, B, D, L, h, io_dtype=FI_F32, small_tile_max=0, stream=None):
        self.cfg = make_config(B, D, L, io_dtype, small_tile_max, stream)
        self.B, self.D, self.L = int(B), int(D), int(L)
        self.handle = fi_create(self.cfg, h)

    def step(self, x_t, y_t):
        fi_step(self.handle, x_t, y_t)

    def run(self, x_in, fb, y, x_out=None):
        fi_run_closed_loop(self.handle, x_in, fb, y, x_out)

    def run_prompted(self, x_prompt, p, y, x_out=None):
        fi_run_prompted(self.handle, x_prompt, p, y, x_out)

    def reset(self):
        fi_reset(self.handle)

    @property
    def position(self) -> int:
        return fi_position(self.handle)

    def close(self):
        if self.handle:
            fi_destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
