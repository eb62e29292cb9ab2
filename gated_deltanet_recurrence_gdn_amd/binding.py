"""Thin ctypes binding of libgdn.so (include/gdn.h), same names as the C ABI.

Argument marshalling only: every step of the recurrence runs in the library's HIP
kernels.  PyTorch is used for device memory and streams.  If libgdn.so is missing
the import of this module raises: there is no fallback implementation.

Raw functions (``gdn_create``, ``gdn_forward``, ``gdn_forward_bidi``,
``gdn_forward_packed``, ``gdn_forward_bidi_packed``, ``gdn_forward_noalloc``, ``gdn_free``,
``gdn_last_error``, ``gdn_version``; around the recurrence ``gdn_rotary``, ``gdn_glr_create``,
``gdn_glr_forward``, ``gdn_glr_backward``, ``gdn_group_norm_create``, ``gdn_group_norm_forward``,
``gdn_group_norm_backward``, ``gdn_linear_create``, ``gdn_linear_forward``, ``gdn_linear_backward``,
``gdn_rms_norm_create``, ``gdn_rms_norm_forward``, ``gdn_rms_norm_forward_int8``, ``gdn_rms_norm_backward``,
``gdn_quantize_rows``, ``gdn_matmul_int8``) take device pointers as ints or torch tensors and return the C
status.  ``GDN``, ``GLR``, ``GroupNorm``, ``LinearAttention`` and ``RMSNorm`` wrap a handle for torch
callers, ``rotary``, ``quantize_rows`` and ``matmul_int8`` a call.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn.so")

GDN_OK = 0
GDN_ERR_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_ALIGN = -3
GDN_ERR_ALIAS = -4
GDN_ERR_DEVICE = -5
GDN_ERR_OOM = -6
GDN_ERR_LAUNCH = -7
STATUS_NAMES = {0: "GDN_OK", -1: "GDN_ERR_ARG", -2: "GDN_ERR_UNSUPPORTED", -3: "GDN_ERR_ALIGN",
                -4: "GDN_ERR_ALIAS", -5: "GDN_ERR_DEVICE", -6: "GDN_ERR_OOM", -7: "GDN_ERR_LAUNCH"}
GDN_F32 = 0
GDN_BF16 = 1
GDN_FP8 = 2
GDN_FLAG_BIDI = 1
GDN_FLAG_SEGMENTS = 2
GDN_FLAG_REVERSE = 4
GDN_FLAG_HEAD_DECAY = 8
GDN_FLAG_TRAIN = 16
GDN_ROTARY_HALVES = 1
GDN_ROTARY_INVERSE = 2
GDN_ACT_NONE = 0
GDN_ACT_SILU = 1
GDN_GLR_SAVED_TOKENS = 64


class gdn_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int),
                ("d_k", ctypes.c_int), ("d_v", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("max_T", ctypes.c_longlong), ("flags", ctypes.c_uint)]


class gdn_rotary_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("axis_dim", ctypes.c_int * 3), ("theta", ctypes.c_double),
                ("flags", ctypes.c_uint)]


class gdn_glr_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("gate_dim", ctypes.c_int), ("max_T", ctypes.c_longlong),
                ("flags", ctypes.c_uint)]


class gdn_group_norm_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("C", ctypes.c_int), ("G", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("eps", ctypes.c_float), ("max_N", ctypes.c_longlong)]


class gdn_linear_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("d_k", ctypes.c_int),
                ("d_v", ctypes.c_int), ("io_dtype", ctypes.c_int), ("max_T", ctypes.c_longlong),
                ("flags", ctypes.c_uint)]


class gdn_rms_norm_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("C", ctypes.c_int), ("io_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("max_N", ctypes.c_longlong)]


class gdn_matmul_config(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class GDNError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _load():
    # PyTorch ships its own HIP runtime whose soname (libamdhip64.so.7) is the one
    # libgdn.so needs.  Loading torch first makes the dynamic loader reuse that
    # runtime for libgdn.so, so the process holds one HIP runtime, not two.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m gated_deltanet_recurrence_gdn_amd.build` "
            "(there is no non-HIP implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    lib.gdn_create.argtypes = [ctypes.POINTER(gdn_config), ctypes.POINTER(ctypes.c_void_p)]
    lib.gdn_create.restype = I
    lib.gdn_forward.argtypes = [P, P, P, P, P, P, P, P, P, LL, I, P]
    lib.gdn_forward.restype = I
    lib.gdn_forward_bidi.argtypes = [P, P, P, P, P, P, P, LL, I, P]
    lib.gdn_forward_bidi.restype = I
    lib.gdn_forward_packed.argtypes = [P, P, LL, LL, P, P, P, P, P, LL, I, P]
    lib.gdn_forward_packed.restype = I
    lib.gdn_forward_bidi_packed.argtypes = [P, P, LL, LL, P, P, P, LL, I, P]
    lib.gdn_forward_bidi_packed.restype = I
    lib.gdn_forward_noalloc.argtypes = [ctypes.POINTER(gdn_config), P, P, P, P, P, P, P, P, LL, I, P]
    lib.gdn_forward_noalloc.restype = I
    lib.gdn_rotary.argtypes = [ctypes.POINTER(gdn_rotary_config), P, LL, LL, P, LL, LL, P, LL, LL, I, I, LL, P]
    lib.gdn_rotary.restype = I
    lib.gdn_glr_create.argtypes = [ctypes.POINTER(gdn_glr_config), ctypes.POINTER(ctypes.c_void_p)]
    lib.gdn_glr_create.restype = I
    lib.gdn_glr_forward.argtypes = [P, P, P, P, P, P, P, P, LL, P]
    lib.gdn_glr_forward.restype = I
    lib.gdn_glr_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, LL, P]
    lib.gdn_glr_backward.restype = I
    lib.gdn_group_norm_create.argtypes = [ctypes.POINTER(gdn_group_norm_config), ctypes.POINTER(ctypes.c_void_p)]
    lib.gdn_group_norm_create.restype = I
    lib.gdn_group_norm_forward.argtypes = [P, P, P, P, P, P, LL, LL, P]
    lib.gdn_group_norm_forward.restype = I
    lib.gdn_group_norm_backward.argtypes = [P, P, P, P, P, P, P, P, P, LL, LL, P]
    lib.gdn_group_norm_backward.restype = I
    lib.gdn_linear_create.argtypes = [ctypes.POINTER(gdn_linear_config), ctypes.POINTER(ctypes.c_void_p)]
    lib.gdn_linear_create.restype = I
    lib.gdn_linear_forward.argtypes = [P] + [P, LL, LL] * 3 + [P, P, P, P, LL, P]
    lib.gdn_linear_forward.restype = I
    lib.gdn_linear_backward.argtypes = [P] + [P, LL, LL] * 3 + [P] * 9 + [LL, P]
    lib.gdn_linear_backward.restype = I
    lib.gdn_rms_norm_create.argtypes = [ctypes.POINTER(gdn_rms_norm_config), ctypes.POINTER(ctypes.c_void_p)]
    lib.gdn_rms_norm_create.restype = I
    lib.gdn_rms_norm_forward.argtypes = [P, P, P, P, P, P, P, LL, P]
    lib.gdn_rms_norm_forward.restype = I
    lib.gdn_rms_norm_forward_int8.argtypes = [P, P, P, P, P, P, P, LL, P]
    lib.gdn_rms_norm_forward_int8.restype = I
    lib.gdn_rms_norm_backward.argtypes = [P, P, P, P, P, P, P, P, LL, P]
    lib.gdn_rms_norm_backward.restype = I
    lib.gdn_quantize_rows.argtypes = [I, P, I, P, P, LL, I, P]
    lib.gdn_quantize_rows.restype = I
    lib.gdn_matmul_int8.argtypes = [ctypes.POINTER(gdn_matmul_config), P, P, P, P, P, P, LL, LL, P]
    lib.gdn_matmul_int8.restype = I
    lib.gdn_free.argtypes = [P]
    lib.gdn_free.restype = None
    lib.gdn_last_error.argtypes = [P]
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = ctypes.c_char_p
    return lib


_lib = _load()


def library():
    return _lib


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def gdn_version() -> str:
    return _lib.gdn_version().decode()


def gdn_last_error(h) -> str:
    return _lib.gdn_last_error(h).decode()


def gdn_create(device: int, B: int, H: int, d_k: int, d_v: int, io_dtype: int, max_T: int,
               flags: int = 0):
    """Returns (status, handle); handle is None on failure."""
    cfg = gdn_config(device, B, H, d_k, d_v, io_dtype, max_T, flags)
    h = ctypes.c_void_p()
    st = _lib.gdn_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, (h.value if st == GDN_OK else None)


def gdn_free(h) -> None:
    _lib.gdn_free(h)


def gdn_forward(h, q, k, v, beta, decay, state_in, state_out, out, T: int, chunk_len: int,
                stream=None) -> int:
    return _lib.gdn_forward(h, _p(q), _p(k), _p(v), _p(beta), _p(decay), _p(state_in),
                            _p(state_out), _p(out), int(T), int(chunk_len), stream)


def gdn_forward_bidi(h, q, k, v, beta, decay, out, T: int, chunk_len: int, stream=None) -> int:
    return _lib.gdn_forward_bidi(h, _p(q), _p(k), _p(v), _p(beta), _p(decay), _p(out), int(T),
                                 int(chunk_len), stream)


def gdn_forward_packed(h, qkv, token_stride: int, batch_stride: int, beta_logit, decay_logit, state_in,
                       state_out, out, T: int, chunk_len: int, stream=None) -> int:
    return _lib.gdn_forward_packed(h, _p(qkv), int(token_stride), int(batch_stride), _p(beta_logit),
                                   _p(decay_logit), _p(state_in), _p(state_out), _p(out), int(T),
                                   int(chunk_len), stream)


def gdn_forward_bidi_packed(h, qkv, token_stride: int, batch_stride: int, beta_logit, decay_logit, out,
                            T: int, chunk_len: int, stream=None) -> int:
    return _lib.gdn_forward_bidi_packed(h, _p(qkv), int(token_stride), int(batch_stride), _p(beta_logit),
                                        _p(decay_logit), _p(out), int(T), int(chunk_len), stream)


def gdn_forward_noalloc(cfg: gdn_config, q, k, v, beta, decay, state_in, state_out, out, T: int,
                        chunk_len: int, stream=None) -> int:
    """No handle, no allocation: cfg (a gdn_config) comes with every call; errors are
    read with gdn_last_error(None)."""
    return _lib.gdn_forward_noalloc(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(beta), _p(decay), _p(state_in),
                                    _p(state_out), _p(out), int(T), int(chunk_len), stream)


def gdn_rotary(cfg: gdn_rotary_config, x, x_token_stride: int, x_batch_stride: int, out, out_token_stride: int,
               out_batch_stride: int, positions, positions_batch_stride: int, first_token: int, height: int,
               width: int, T: int, stream=None) -> int:
    """No handle: errors are read with gdn_last_error(None)."""
    return _lib.gdn_rotary(ctypes.byref(cfg), _p(x), int(x_token_stride), int(x_batch_stride), _p(out),
                           int(out_token_stride), int(out_batch_stride), _p(positions), int(positions_batch_stride),
                           int(first_token), int(height), int(width), int(T), stream)


def gdn_glr_create(device: int, B: int, H: int, d: int, io_dtype: int, gate_dim: int, max_T: int, flags: int = 0):
    """Returns (status, handle); handle is None on failure."""
    cfg = gdn_glr_config(device, B, H, d, io_dtype, gate_dim, max_T, flags)
    h = ctypes.c_void_p()
    st = _lib.gdn_glr_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, (h.value if st == GDN_OK else None)


def gdn_glr_forward(h, v, beta, decay, state_in, state_out, saved, out, T: int, stream=None) -> int:
    return _lib.gdn_glr_forward(h, _p(v), _p(beta), _p(decay), _p(state_in), _p(state_out), _p(saved), _p(out),
                                int(T), stream)


def gdn_glr_backward(h, v, beta, decay, saved, dout, dstate_out, dv, dbeta, ddecay, dstate_in, T: int,
                     stream=None) -> int:
    return _lib.gdn_glr_backward(h, _p(v), _p(beta), _p(decay), _p(saved), _p(dout), _p(dstate_out), _p(dv),
                                 _p(dbeta), _p(ddecay), _p(dstate_in), int(T), stream)


def gdn_group_norm_create(device: int, C: int, G: int, io_dtype: int, act: int, eps: float, max_N: int):
    """Returns (status, handle); handle is None on failure."""
    cfg = gdn_group_norm_config(device, C, G, io_dtype, act, eps, max_N)
    h = ctypes.c_void_p()
    st = _lib.gdn_group_norm_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, (h.value if st == GDN_OK else None)


def gdn_group_norm_forward(h, x, weight, bias, out, stats, N: int, S: int, stream=None) -> int:
    return _lib.gdn_group_norm_forward(h, _p(x), _p(weight), _p(bias), _p(out), _p(stats), int(N), int(S), stream)


def gdn_group_norm_backward(h, x, weight, bias, stats, dout, dx, dweight, dbias, N: int, S: int, stream=None) -> int:
    return _lib.gdn_group_norm_backward(h, _p(x), _p(weight), _p(bias), _p(stats), _p(dout), _p(dx), _p(dweight),
                                        _p(dbias), int(N), int(S), stream)


def gdn_linear_create(device: int, B: int, H: int, d_k: int, d_v: int, io_dtype: int, max_T: int, flags: int = 0):
    """Returns (status, handle); handle is None on failure."""
    cfg = gdn_linear_config(device, B, H, d_k, d_v, io_dtype, max_T, flags)
    h = ctypes.c_void_p()
    st = _lib.gdn_linear_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, (h.value if st == GDN_OK else None)


def gdn_linear_forward(h, q, q_ts: int, q_bs: int, k, k_ts: int, k_bs: int, v, v_ts: int, v_bs: int, decay, state_in,
                       state_out, out, T: int, stream=None) -> int:
    return _lib.gdn_linear_forward(h, _p(q), int(q_ts), int(q_bs), _p(k), int(k_ts), int(k_bs), _p(v), int(v_ts),
                                   int(v_bs), _p(decay), _p(state_in), _p(state_out), _p(out), int(T), stream)


def gdn_linear_backward(h, q, q_ts: int, q_bs: int, k, k_ts: int, k_bs: int, v, v_ts: int, v_bs: int, decay, state_in,
                        dout, dstate_out, dq, dk, dv, dlog_decay, dstate_in, T: int, stream=None) -> int:
    return _lib.gdn_linear_backward(h, _p(q), int(q_ts), int(q_bs), _p(k), int(k_ts), int(k_bs), _p(v), int(v_ts),
                                    int(v_bs), _p(decay), _p(state_in), _p(dout), _p(dstate_out), _p(dq), _p(dk),
                                    _p(dv), _p(dlog_decay), _p(dstate_in), int(T), stream)


def gdn_rms_norm_create(device: int, C: int, io_dtype: int, eps: float, max_N: int):
    """Returns (status, handle); handle is None on failure."""
    cfg = gdn_rms_norm_config(device, C, io_dtype, eps, max_N)
    h = ctypes.c_void_p()
    st = _lib.gdn_rms_norm_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, (h.value if st == GDN_OK else None)


def gdn_rms_norm_forward(h, x, residual, weight, sum_out, out, rstd, N: int, stream=None) -> int:
    return _lib.gdn_rms_norm_forward(h, _p(x), _p(residual), _p(weight), _p(sum_out), _p(out), _p(rstd), int(N), stream)


def gdn_rms_norm_forward_int8(h, x, residual, weight, sum_out, out8, scale, N: int, stream=None) -> int:
    return _lib.gdn_rms_norm_forward_int8(h, _p(x), _p(residual), _p(weight), _p(sum_out), _p(out8), _p(scale), int(N),
                                          stream)


def gdn_rms_norm_backward(h, sum_in, weight, rstd, dout, dsum, dx, dweight, N: int, stream=None) -> int:
    return _lib.gdn_rms_norm_backward(h, _p(sum_in), _p(weight), _p(rstd), _p(dout), _p(dsum), _p(dx), _p(dweight),
                                      int(N), stream)


def gdn_quantize_rows(device: int, x, io_dtype: int, out8, scale, N: int, C: int, stream=None) -> int:
    """No handle: errors are read with gdn_last_error(None)."""
    return _lib.gdn_quantize_rows(device, _p(x), io_dtype, _p(out8), _p(scale), int(N), C, stream)


def gdn_matmul_int8(cfg: gdn_matmul_config, a, a_scale, w, w_scale, bias, out, out_stride: int, M: int,
                    stream=None) -> int:
    """No handle: errors are read with gdn_last_error(None)."""
    return _lib.gdn_matmul_int8(ctypes.byref(cfg), _p(a), _p(a_scale), _p(w), _p(w_scale), _p(bias), _p(out),
                                int(out_stride), int(M), stream)


def current_stream():
    """The raw hipStream_t of torch's current stream on the current device."""
    import torch
    return torch.cuda.current_stream().cuda_stream


class GDN:
    """A handle bound to one (device, B, H, d_k, d_v, dtype, max_T) shape, for torch callers.

    ``forward`` / ``forward_bidi`` check shapes and dtypes on the host, allocate the
    outputs that were not passed in (torch.empty on the same device) and call the C ABI
    on torch's current stream.  Errors raise ``GDNError`` with the library's message.
    """

    def __init__(self, B, H, d_k, d_v, dtype="bf16", max_T=0, device=0, bidi=False, segments=False):
        self.B, self.H, self.d_k, self.d_v = B, H, d_k, d_v
        self.dtype = dtype
        self.io = {"bf16": GDN_BF16, "fp32": GDN_F32, "fp8": GDN_FP8}[dtype]
        self.max_T = max_T
        self.device = device
        self.h = None
        self._free = _lib.gdn_free  # kept on the object: usable while the interpreter shuts down
        flags = (GDN_FLAG_BIDI if bidi else 0) | (GDN_FLAG_SEGMENTS if segments else 0)
        st, h = gdn_create(device, B, H, d_k, d_v, self.io, max_T, flags)
        if st != GDN_OK:
            raise GDNError(st, gdn_last_error(None))
        self.h = h

    def close(self):
        if getattr(self, "h", None) is not None:
            self._free(self.h)
            self.h = None

    __del__ = close

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check(self, st):
        if st != GDN_OK:
            raise GDNError(st, gdn_last_error(self.h))

    def _torch_dtype(self):
        """dtype of q, k, v (and qkv)."""
        import torch
        return {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}[self.dtype]

    def _out_dtype(self):
        """dtype of out: fp32 for fp32 inputs, bf16 otherwise."""
        import torch
        return torch.float32 if self.dtype == "fp32" else torch.bfloat16

    def _check_inputs(self, q, k, v, beta, decay):
        import torch
        B, H, dk, dv = self.B, self.H, self.d_k, self.d_v
        T = q.shape[1]
        dt = self._torch_dtype()
        for name, x, shape, want in (("q", q, (B, T, H, dk), dt), ("k", k, (B, T, H, dk), dt),
                                     ("v", v, (B, T, H, dv), dt),
                                     ("beta", beta, (B, T, H), torch.float32),
                                     ("decay", decay, (B, T, H), torch.float32)):
            if tuple(x.shape) != shape or x.dtype != want or not x.is_contiguous():
                raise ValueError(f"{name}: expected contiguous {want} {shape}, got {x.dtype} {tuple(x.shape)}")
        return T

    def _check_given(self, T, out=None, state_in=None, state_out=None):
        """Shape, dtype and layout of the caller's out and states.  The C ABI takes raw
        pointers and cannot know their extents, so a wrong shape is refused here."""
        import torch
        st = (self.B, self.H, self.d_v, self.d_k)
        for name, x, shape, want in (("out", out, (self.B, T, self.H, self.d_v), self._out_dtype()),
                                     ("state_in", state_in, st, torch.float32),
                                     ("state_out", state_out, st, torch.float32)):
            if x is not None and (tuple(x.shape) != shape or x.dtype != want or not x.is_contiguous()):
                raise ValueError(f"{name}: expected contiguous {want} {shape}, got {x.dtype} {tuple(x.shape)}")

    def forward(self, q, k, v, beta, decay, state_in=None, state_out=None, out=None,
                chunk_len=64, return_state=True):
        """Causal recurrence.  Returns (out, state_out)."""
        import torch
        T = self._check_inputs(q, k, v, beta, decay)
        self._check_given(T, out, state_in, state_out)
        if out is None:
            out = torch.empty((self.B, T, self.H, self.d_v), dtype=self._out_dtype(), device=q.device)
        if state_out is None and return_state:
            state_out = torch.empty((self.B, self.H, self.d_v, self.d_k), dtype=torch.float32,
                                    device=q.device)
        self._check(gdn_forward(self.h, q, k, v, beta, decay, state_in, state_out, out, T, chunk_len,
                                current_stream()))
        return out, state_out

    def forward_bidi(self, q, k, v, beta, decay, out=None, chunk_len=64):
        """Bidirectional form.  Returns out."""
        import torch
        T = self._check_inputs(q, k, v, beta, decay)
        self._check_given(T, out)
        if out is None:
            out = torch.empty((self.B, T, self.H, self.d_v), dtype=self._out_dtype(), device=q.device)
        self._check(gdn_forward_bidi(self.h, q, k, v, beta, decay, out, T, chunk_len, current_stream()))
        return out

    def _check_packed(self, qkv, beta_logit, decay_logit):
        """qkv: a [B, T, W] tensor (any strides whose last one is 1, W >= 2 H d_k + H d_v)."""
        import torch
        B, H = self.B, self.H
        if qkv.dim() != 3 or qkv.shape[0] != B or qkv.dtype != self._torch_dtype() or qkv.stride(2) != 1:
            raise ValueError(f"qkv: expected a [B={B}, T, W] {self._torch_dtype()} view with unit last stride, "
                             f"got {qkv.dtype} {tuple(qkv.shape)} strides {qkv.stride()}")
        if qkv.shape[2] < 2 * H * self.d_k + H * self.d_v:
            raise ValueError(f"qkv: last dim {qkv.shape[2]} < 2 H d_k + H d_v")
        T = qkv.shape[1]
        for name, x in (("beta_logit", beta_logit), ("decay_logit", decay_logit)):
            if tuple(x.shape) != (B, T, H) or x.dtype != torch.float32 or not x.is_contiguous():
                raise ValueError(f"{name}: expected contiguous float32 {(B, T, H)}, got {x.dtype} {tuple(x.shape)}")
        return T, qkv.stride(1), qkv.stride(0)

    def forward_packed(self, qkv, beta_logit, decay_logit, state_in=None, state_out=None, out=None,
                       chunk_len=64, return_state=True):
        """Causal recurrence with the fused prologue from a packed [B, T, W] qkv view
        (q, k, v of every head side by side in W; L2-normalised q, k and
        sigmoid / exp(-softplus) gates applied in the kernels).  Returns (out, state_out)."""
        import torch
        T, ts, bs = self._check_packed(qkv, beta_logit, decay_logit)
        self._check_given(T, out, state_in, state_out)
        if out is None:
            out = torch.empty((self.B, T, self.H, self.d_v), dtype=self._out_dtype(), device=qkv.device)
        if state_out is None and return_state:
            state_out = torch.empty((self.B, self.H, self.d_v, self.d_k), dtype=torch.float32,
                                    device=qkv.device)
        self._check(gdn_forward_packed(self.h, qkv, ts, bs, beta_logit, decay_logit, state_in, state_out, out, T,
                                       chunk_len, current_stream()))
        return out, state_out

    def forward_bidi_packed(self, qkv, beta_logit, decay_logit, out=None, chunk_len=64):
        """Bidirectional form with the fused prologue.  Returns out."""
        import torch
        T, ts, bs = self._check_packed(qkv, beta_logit, decay_logit)
        self._check_given(T, out)
        if out is None:
            out = torch.empty((self.B, T, self.H, self.d_v), dtype=self._out_dtype(), device=qkv.device)
        self._check(gdn_forward_bidi_packed(self.h, qkv, ts, bs, beta_logit, decay_logit, out, T, chunk_len,
                                            current_stream()))
        return out


# ---- the operators around the recurrence ------------------------------------------

_IO = {"bf16": GDN_BF16, "fp32": GDN_F32, "fp8": GDN_FP8}


def _io_of(dtype):
    """gdn_dtype of a torch dtype that q, k, v, x may have."""
    import torch
    if dtype is torch.bfloat16:
        return GDN_BF16
    if dtype is torch.float32:
        return GDN_F32
    if dtype is torch.float8_e4m3fn:
        return GDN_FP8
    raise ValueError(f"expected bfloat16, float32 or float8_e4m3fn, got {dtype}")


def _expect(device, name, x, shape, want):
    """Shape, dtype, layout and device of a tensor (None passes): the C ABI takes raw pointers and
    cannot know extents, so a wrong one is refused here."""
    if x is None:
        return
    if x.shape != shape or x.dtype is not want or not x.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {want} {tuple(shape)}, got {x.dtype} {tuple(x.shape)}")
    if x.get_device() != device or device < 0:  # host tensors say -1, as a dry-run handle does
        raise ValueError(f"{name}: expected a tensor on cuda:{device}, got {x.device}")


def _stream_of(device: int):
    """The raw hipStream_t of torch's current stream on that device (not of the current device's).
    torch's own accessor for launchers; torch.cuda.current_stream wraps the same value in an object,
    a microsecond that a call on one token feels."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


@functools.lru_cache(maxsize=256)
def _rotary_config(*values):
    device, B, H, d, io, dims, theta, flags = values
    return gdn_rotary_config(device, B, H, d, io, (ctypes.c_int * 3)(*dims), theta, flags)


def rotary(x, axis_dims, theta=10000.0, positions=None, grid=None, first_token=0, halves=False, inverse=False,
           out=None):
    """Rotary positions over (time, height, width) for x [B, T, H, d] (any strides with the heads of a
    token side by side; q and k of a packed projection are one x of twice the heads).

    axis_dims: elements of a head turned by each axis; positions: int32 [B, T, 3] or [T, 3] (the same for
    every batch element), or None for a raster grid=(height, width) whose first token is first_token (neither
    is read where positions are given).
    halves: pairs (i, i + dim/2) instead of (2i, 2i+1).  inverse: the negative angles, which is the
    gradient with respect to x.  out may be x (in place).  Returns out (fp32 for fp32 x, else bf16).
    Not an autograd function: out carries no gradient, also where x requires one.
    """
    import torch
    if len(axis_dims) != 3:
        raise ValueError(f"axis_dims: expected three sizes (time, height, width), got {axis_dims}")
    io = _io_of(x.dtype)
    odt = torch.float32 if io == GDN_F32 else torch.bfloat16
    device = x.get_device()
    if x.dim() != 4 or device < 0:
        raise ValueError(f"x: expected a [B, T, H, d] tensor on a GPU, got {tuple(x.shape)} on {x.device}")
    B, T, H, d = x.shape
    if out is None:
        out = torch.empty((B, T, H, d), dtype=odt, device=x.device)
    elif out.shape != x.shape or out.dtype is not odt or out.get_device() != device:
        raise ValueError(f"out: expected {odt} {(B, T, H, d)} on {x.device}, got {out.dtype} {tuple(out.shape)}")
    none = 0 in (B, T, H)
    if none:  # nothing to read or write: what remains is checked by a call on no tokens
        B, H = max(B, 1), max(H, 1)
        xbs = obs = 0
        xts = ots = H * d
    else:
        xbs, xts, xhs, xes = x.stride()
        obs, ots, ohs, oes = out.stride()
        for name, hs, es in (("x", xhs, xes), ("out", ohs, oes)):
            if (d > 1 and es != 1) or (H > 1 and hs != d):
                raise ValueError(f"{name}: the heads of a token must lie side by side, got strides "
                                 f"{(x if name == 'x' else out).stride()}")
        if T == 1:  # a dimension of one has no stride of its own
            xts = ots = H * d
        if B == 1:
            xbs = obs = 0
    pbs = 0
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.get_device() != device or not positions.is_contiguous() or \
                tuple(positions.shape) not in ((T, 3), (x.shape[0], T, 3)):
            raise ValueError(f"positions: expected contiguous int32 {(T, 3)} or {(x.shape[0], T, 3)} on {x.device}, "
                             f"got {positions.dtype} {tuple(positions.shape)} on {positions.device}")
        pbs = 3 * T if positions.dim() == 3 else 0
        height = width = 1
        first_token = 0
    elif grid is None:
        raise ValueError("positions or grid must be given")
    else:
        height, width = grid
    flags = (GDN_ROTARY_HALVES if halves else 0) | (GDN_ROTARY_INVERSE if inverse else 0)
    cfg = _rotary_config(device, B, H, d, io, tuple(axis_dims), float(theta), flags)
    st = gdn_rotary(cfg, x, xts, xbs, out, ots, obs, positions, pbs, first_token, height, width,
                    0 if none else T, _stream_of(device))
    if st != GDN_OK:
        raise GDNError(st, gdn_last_error(None))
    return out


class _Handle:
    """A handle of the library: freed on close, as a context manager and with the object."""

    h = None

    def _open(self, made):
        self._free = _lib.gdn_free  # kept on the object: usable while the interpreter shuts down
        st, h = made
        if st != GDN_OK:
            raise GDNError(st, gdn_last_error(None))
        self.h = h

    def close(self):
        if self.h is not None:
            self._free(self.h)
            self.h = None

    __del__ = close

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check(self, st):
        if st != GDN_OK:
            raise GDNError(st, gdn_last_error(self.h))

    def _set_types(self, dtype):
        """The dtype of the input, and of the outputs: fp32 for fp32 inputs, bf16 otherwise."""
        import torch
        self._f32 = torch.float32
        self._in, self._out = {"bf16": (torch.bfloat16, torch.bfloat16), "fp32": (torch.float32, torch.float32),
                               "fp8": (torch.float8_e4m3fn, torch.bfloat16)}[dtype]


class GLR(_Handle):
    """The diagonal gated linear recurrence h_t = a_t h_{t-1} + b_t v_t, for torch callers: a handle bound
    to one (device, B, H, d, dtype, gate, max_T).  gate "head": beta and decay [B, T, H]; "channel":
    [B, T, H, d].  reverse walks the tokens from the last to the first.  Not an autograd function: call
    ``backward``.  Calls on one handle must not overlap on the device (two streams, two graphs): they can
    hang it."""

    def __init__(self, B, H, d, dtype="bf16", max_T=0, device=0, gate="head", reverse=False):
        self.B, self.H, self.d, self.dtype, self.device = B, H, d, dtype, device
        self.gate_dim = {"head": 1, "channel": d}[gate]
        self._set_types(dtype)
        self._state = (B, H, d)
        self._open(gdn_glr_create(device, B, H, d, _IO[dtype], self.gate_dim, max_T,
                                  GDN_FLAG_REVERSE if reverse else 0))

    def _inputs(self, v, beta, decay):
        """(T, shape of v, shape of the gates)"""
        if v.dim() != 4:
            raise ValueError(f"v: expected [B, T, H, d], got {tuple(v.shape)}")
        T = v.shape[1]
        tok = (self.B, T, self.H, self.d)
        gate = tok[:3] if self.gate_dim == 1 else tok
        _expect(self.device, "v", v, tok, self._in)
        _expect(self.device, "beta", beta, gate, self._f32)
        _expect(self.device, "decay", decay, gate, self._f32)
        return T, tok, gate

    def _saved(self, T):
        return (self.B, -(-T // GDN_GLR_SAVED_TOKENS), self.H, self.d)

    def _forward(self, v, beta, decay, state_in, state_out, out, return_state, save):
        import torch
        T, tok, _ = self._inputs(v, beta, decay)
        _expect(self.device, "state_in", state_in, self._state, self._f32)
        _expect(self.device, "state_out", state_out, self._state, self._f32)
        _expect(self.device, "out", out, tok, self._out)
        if out is None:
            out = torch.empty(tok, dtype=self._out, device=v.device)
        if state_out is None and return_state:
            state_out = torch.empty(self._state, dtype=self._f32, device=v.device)
        saved = torch.empty(self._saved(T), dtype=self._f32, device=v.device) if save else None
        self._check(gdn_glr_forward(self.h, v, beta, decay, state_in, state_out, saved, out, T,
                                    _stream_of(self.device)))
        return out, state_out, saved

    def forward(self, v, beta, decay, state_in=None, state_out=None, out=None, return_state=True):
        """Returns (out, state_out).  beta None = 1.  state_out may be state_in (in place)."""
        return self._forward(v, beta, decay, state_in, state_out, out, return_state, False)[:2]

    def forward_train(self, v, beta, decay, state_in=None, state_out=None, out=None, return_state=True):
        """Returns (out, state_out, saved); saved goes to ``backward``."""
        return self._forward(v, beta, decay, state_in, state_out, out, return_state, True)

    def backward(self, v, beta, decay, saved, dout, dstate_out=None):
        """The gradient of ``forward_train`` at the same v, beta, decay and its saved.  Returns
        (dv, dbeta, ddecay, dstate_in); dbeta is None without beta."""
        import torch
        T, tok, gate = self._inputs(v, beta, decay)
        _expect(self.device, "saved", saved, self._saved(T), self._f32)
        _expect(self.device, "dout", dout, tok, self._out)
        _expect(self.device, "dstate_out", dstate_out, self._state, self._f32)
        dv = torch.empty(tok, dtype=self._out, device=v.device)
        dbeta = None if beta is None else torch.empty(gate, dtype=self._f32, device=v.device)
        ddecay = torch.empty(gate, dtype=self._f32, device=v.device)
        dstate_in = torch.empty(self._state, dtype=self._f32, device=v.device)
        self._check(gdn_glr_backward(self.h, v, beta, decay, saved, dout, dstate_out, dv, dbeta, ddecay, dstate_in, T,
                                     _stream_of(self.device)))
        return dv, dbeta, ddecay, dstate_in


class GroupNorm(_Handle):
    """Group norm with an activation ("silu" or "none"), channels last, for torch callers: a handle bound
    to one (device, C, G, dtype, act, eps) and samples up to max_N.  x is [N, ..., C]: every dimension
    between is part of the sample; [N, C] normalises each row (N = B T tokens, a group per head).  Not an
    autograd function: call ``backward``."""

    def __init__(self, C, G, dtype="bf16", act="silu", eps=1e-5, max_N=1, device=0):
        self.C, self.G, self.dtype, self.device = C, G, dtype, device
        self._set_types(dtype)
        self._open(gdn_group_norm_create(device, C, G, _IO[dtype], {"none": GDN_ACT_NONE, "silu": GDN_ACT_SILU}[act],
                                         eps, max_N))

    def _inputs(self, x, weight, bias):
        if x.dim() < 2:
            raise ValueError(f"x: expected [N, ..., C], got {tuple(x.shape)}")
        shape = x.shape
        N, S = shape[0], 1
        for n in shape[1:-1]:
            S *= n
        _expect(self.device, "x", x, (*shape[:-1], self.C), self._in)
        _expect(self.device, "weight", weight, (self.C,), self._f32)
        _expect(self.device, "bias", bias, (self.C,), self._f32)
        return N, S

    def forward(self, x, weight=None, bias=None, out=None, return_stats=True):
        """Returns (out, stats); stats [N, G, 2] (mean, 1 / sqrt(var + eps)) goes to ``backward``."""
        import torch
        N, S = self._inputs(x, weight, bias)
        _expect(self.device, "out", out, x.shape, self._out)
        if out is None:
            out = torch.empty(x.shape, dtype=self._out, device=x.device)
        stats = torch.empty((N, self.G, 2), dtype=self._f32, device=x.device) if return_stats else None
        self._check(gdn_group_norm_forward(self.h, x, weight, bias, out, stats, N, S, _stream_of(self.device)))
        return out, stats

    def backward(self, x, weight, bias, stats, dout):
        """The gradient of ``forward`` at the same x, weight, bias and its stats.  Returns (dx, dweight,
        dbias); dweight and dbias are None without weight and bias."""
        import torch
        N, S = self._inputs(x, weight, bias)
        _expect(self.device, "stats", stats, (N, self.G, 2), self._f32)
        _expect(self.device, "dout", dout, x.shape, self._out)
        dx = torch.empty(x.shape, dtype=self._out, device=x.device)
        dweight = None if weight is None else torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        self._check(gdn_group_norm_backward(self.h, x, weight, bias, stats, dout, dx, dweight, dbias, N, S,
                                            _stream_of(self.device)))
        return dx, dweight, dbias


# ---- an 8-bit layer around a linear attention ---------------------------------------


class LinearAttention(_Handle):
    """Linear attention with a decay, S_t = a_t S_{t-1} + v_t k_t^T and o_t = S_t q_t / sqrt(d_k), for torch
    callers: a handle bound to one (device, B, H, d_k, d_v, dtype, decay, max_T).  decay "token": decay
    [B, T, H]; "head": [H], the same at every token.  reverse walks the tokens from the last to the first.
    q, k [B, T, H, d_k] and v [B, T, H, d_v] may have any strides with the heads of a token side by side (views
    into a packed projection).  train makes room for ``backward``.  Not an autograd function: call
    ``backward``."""

    def __init__(self, B, H, d_k, d_v, dtype="bf16", max_T=0, device=0, decay="token", reverse=False, train=False):
        self.B, self.H, self.d_k, self.d_v, self.dtype, self.device = B, H, d_k, d_v, dtype, device
        self.per_head = {"token": False, "head": True}[decay]
        self._set_types(dtype)
        self._state = (B, H, d_v, d_k)
        flags = (GDN_FLAG_REVERSE if reverse else 0) | (GDN_FLAG_HEAD_DECAY if self.per_head else 0) | \
            (GDN_FLAG_TRAIN if train else 0)
        self._open(gdn_linear_create(device, B, H, d_k, d_v, _IO[dtype], max_T, flags))

    def _rows(self, name, x, T, d):
        """(x, token stride, batch stride) of q, k or v."""
        if x.shape != (self.B, T, self.H, d) or x.dtype is not self._in or x.get_device() != self.device:
            raise ValueError(f"{name}: expected {self._in} {(self.B, T, self.H, d)} on cuda:{self.device}, got "
                             f"{x.dtype} {tuple(x.shape)} on {x.device}")
        bs, ts, hs, es = x.stride()
        if T and (es != 1 or (self.H > 1 and hs != d)):
            raise ValueError(f"{name}: the heads of a token must lie side by side, got strides {x.stride()}")
        # a dimension of one has no stride of its own
        return x, self.H * d if T <= 1 else ts, 0 if self.B == 1 else bs

    def _inputs(self, q, k, v, decay, state_in):
        if q.dim() != 4:
            raise ValueError(f"q: expected [B, T, H, d_k], got {tuple(q.shape)}")
        T = q.shape[1]
        rows = (*self._rows("q", q, T, self.d_k), *self._rows("k", k, T, self.d_k), *self._rows("v", v, T, self.d_v))
        gate = (self.H,) if self.per_head else (self.B, T, self.H)
        _expect(self.device, "decay", decay, gate, self._f32)
        _expect(self.device, "state_in", state_in, self._state, self._f32)
        return T, rows, gate

    def forward(self, q, k, v, decay, state_in=None, state_out=None, out=None, return_state=True):
        """Returns (out, state_out).  state_out may be state_in (in place)."""
        import torch
        T, rows, _ = self._inputs(q, k, v, decay, state_in)
        tok = (self.B, T, self.H, self.d_v)
        _expect(self.device, "state_out", state_out, self._state, self._f32)
        _expect(self.device, "out", out, tok, self._out)
        if out is None:
            out = torch.empty(tok, dtype=self._out, device=q.device)
        if state_out is None and return_state:
            state_out = torch.empty(self._state, dtype=self._f32, device=q.device)
        self._check(gdn_linear_forward(self.h, *rows, decay, state_in, state_out, out, T, _stream_of(self.device)))
        return out, state_out

    def backward(self, q, k, v, decay, dout, state_in=None, dstate_out=None):
        """The gradient of ``forward`` at the same q, k, v, decay and state_in.  Returns (dq, dk, dv, dlog_decay,
        dstate_in); dlog_decay, of decay's shape, is with respect to the logarithm of the decay."""
        import torch
        T, rows, gate = self._inputs(q, k, v, decay, state_in)
        kt, vt = (self.B, T, self.H, self.d_k), (self.B, T, self.H, self.d_v)
        _expect(self.device, "dout", dout, vt, self._out)
        _expect(self.device, "dstate_out", dstate_out, self._state, self._f32)
        dq, dk = (torch.empty(kt, dtype=self._out, device=q.device) for _ in range(2))
        dv = torch.empty(vt, dtype=self._out, device=q.device)
        dlog = torch.empty(gate, dtype=self._f32, device=q.device)
        dstate = torch.empty(self._state, dtype=self._f32, device=q.device)
        self._check(gdn_linear_backward(self.h, *rows, decay, state_in, dout, dstate_out, dq, dk, dv, dlog, dstate, T,
                                        _stream_of(self.device)))
        return dq, dk, dv, dlog, dstate


class RMSNorm(_Handle):
    """Root-mean-square norm with the residual's addition, for torch callers: a handle bound to one (device, C,
    dtype, eps) and up to max_N rows.  x is [..., C], its other dimensions the rows; the sum h = x + residual
    is rounded to x's dtype, and the norm is of h.  Not an autograd function: call ``backward``."""

    def __init__(self, C, dtype="bf16", eps=1e-5, max_N=1, device=0):
        self.C, self.dtype, self.device = C, dtype, device
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f"dtype: expected bf16 or fp32, got {dtype}")
        self._set_types(dtype)
        self._open(gdn_rms_norm_create(device, C, _IO[dtype], eps, max_N))

    def _inputs(self, x, weight, residual, sum_out):
        if x.dim() < 1:
            raise ValueError("x: expected [..., C]")
        shape = (*x.shape[:-1], self.C)
        _expect(self.device, "x", x, shape, self._in)
        _expect(self.device, "weight", weight, (self.C,), self._f32)
        _expect(self.device, "residual", residual, shape, self._in)
        _expect(self.device, "sum_out", sum_out, shape, self._in)
        if residual is None and sum_out is not None:
            raise ValueError("sum_out: there is no sum without residual")
        return x.numel() // self.C

    def _forward(self, x, weight, residual, sum_out, out, train):
        import torch
        N = self._inputs(x, weight, residual, sum_out)
        _expect(self.device, "out", out, x.shape, self._out)
        if out is None:
            out = torch.empty(x.shape, dtype=self._out, device=x.device)
        if residual is not None and sum_out is None:
            sum_out = torch.empty(x.shape, dtype=self._in, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=self._f32, device=x.device) if train else None
        self._check(gdn_rms_norm_forward(self.h, x, residual, weight, sum_out, out, rstd, N, _stream_of(self.device)))
        return out, x if residual is None else sum_out, rstd

    def forward(self, x, weight=None, residual=None, sum_out=None, out=None):
        """Returns (out, h); h is x itself without residual.  sum_out may be x or residual (in place)."""
        return self._forward(x, weight, residual, sum_out, out, False)[:2]

    def forward_train(self, x, weight=None, residual=None, sum_out=None, out=None):
        """Returns (out, h, rstd); h and rstd go to ``backward``."""
        return self._forward(x, weight, residual, sum_out, out, True)

    def forward_int8(self, x, weight=None, residual=None, sum_out=None, out=None, scale=None):
        """Returns (out, scale, h): rows of 8-bit whole numbers with a scale each, for ``matmul_int8``."""
        import torch
        N = self._inputs(x, weight, residual, sum_out)
        _expect(self.device, "out", out, x.shape, torch.int8)
        _expect(self.device, "scale", scale, x.shape[:-1], self._f32)
        if out is None:
            out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        if scale is None:
            scale = torch.empty(x.shape[:-1], dtype=self._f32, device=x.device)
        if residual is not None and sum_out is None:
            sum_out = torch.empty(x.shape, dtype=self._in, device=x.device)
        self._check(gdn_rms_norm_forward_int8(self.h, x, residual, weight, sum_out, out, scale, N,
                                              _stream_of(self.device)))
        return out, scale, x if residual is None else sum_out

    def backward(self, h, weight, rstd, dout, dsum=None, dx=None):
        """The gradient of ``forward_train`` at the same weight and its h and rstd; dsum is what else arrives at
        h.  Returns (dx, dweight): dx is the gradient of x and of residual, and may be dsum (in place); dweight
        is None without weight."""
        import torch
        N = self._inputs(h, weight, None, None)
        _expect(self.device, "rstd", rstd, h.shape[:-1], self._f32)
        for name, y in (("dout", dout), ("dsum", dsum), ("dx", dx)):
            _expect(self.device, name, y, h.shape, self._out)
        if dx is None:
            dx = torch.empty(h.shape, dtype=self._out, device=h.device)
        dweight = None if weight is None else torch.empty_like(weight)
        self._check(gdn_rms_norm_backward(self.h, h, weight, rstd, dout, dsum, dx, dweight, N,
                                          _stream_of(self.device)))
        return dx, dweight


def quantize_rows(x, out=None, scale=None):
    """Rows [..., C] of x (bf16 or fp32, C a multiple of 8 up to 8192) in 8 bits with a scale each: (out int8,
    scale), x about out * scale with scale = max|row| / 127.  For the weights of ``matmul_int8`` [N, K], or
    activations before it."""
    import torch
    device = x.get_device()
    if x.dim() < 1 or device < 0 or x.dtype not in (torch.bfloat16, torch.float32) or not x.is_contiguous():
        raise ValueError(f"x: expected contiguous bfloat16 or float32 rows on a GPU, got {x.dtype} {tuple(x.shape)} "
                         f"on {x.device}")
    _expect(device, "out", out, x.shape, torch.int8)
    _expect(device, "scale", scale, x.shape[:-1], torch.float32)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    C = x.shape[-1]
    st = gdn_quantize_rows(device, x, _io_of(x.dtype), out, scale, x.numel() // C if C else 0, C, _stream_of(device))
    if st != GDN_OK:
        raise GDNError(st, gdn_last_error(None))
    return out, scale


@functools.lru_cache(maxsize=256)
def _matmul_config(*values):
    return gdn_matmul_config(*values)


def matmul_int8(a, a_scale, w, w_scale, bias=None, out=None, dtype="bf16"):
    """out[m, n] = (sum_k a[m, k] w[n, k]) a_scale[m] w_scale[n] + bias[n]: a [..., K] and w [N, K] int8 rows with
    a scale each (K a multiple of 16 up to 65536, N of 8), bias [N] or None.  out [..., N] (fp32 or bf16; dtype where it is not given) may be the first
    columns of wider rows.  Returns out."""
    import torch
    device = a.get_device()
    if a.dim() < 1 or w.dim() != 2 or device < 0:
        raise ValueError(f"expected a [..., K] and w [N, K] on a GPU, got {tuple(a.shape)} on {a.device} and {tuple(w.shape)}")
    N, K = w.shape
    lead = a.shape[:-1]
    _expect(device, "a", a, (*lead, K), torch.int8)
    _expect(device, "a_scale", a_scale, lead, torch.float32)
    _expect(device, "w", w, (N, K), torch.int8)
    _expect(device, "w_scale", w_scale, (N,), torch.float32)
    _expect(device, "bias", bias, (N,), torch.float32)
    M = a_scale.numel()
    if out is None:
        out = torch.empty((*lead, N), dtype={"bf16": torch.bfloat16, "fp32": torch.float32}[dtype], device=a.device)
    elif out.shape != (*lead, N) or out.dtype not in (torch.bfloat16, torch.float32) or out.get_device() != device:
        raise ValueError(f"out: expected bfloat16 or float32 {(*lead, N)} on {a.device}, got {out.dtype} "
                         f"{tuple(out.shape)} on {out.device}")
    stride = N
    if M > 1 and not out.is_contiguous():  # rows one distance apart, all dimensions of a taken together
        rows = out.view(-1, N) if len(lead) == 1 else out.flatten(0, -2)
        if rows.data_ptr() != out.data_ptr() or rows.stride(1) != 1:
            raise ValueError(f"out: rows must be contiguous and evenly apart, got strides {out.stride()}")
        stride = rows.stride(0)
    elif M == 1 and N > 1 and out.stride(-1) != 1:
        raise ValueError(f"out: rows must be contiguous, got strides {out.stride()}")
    io = GDN_F32 if out.dtype is torch.float32 else GDN_BF16
    st = gdn_matmul_int8(_matmul_config(device, N, K, io), a, a_scale, w, w_scale, bias, out, stride, M,
                         _stream_of(device))
    if st != GDN_OK:
        raise GDNError(st, gdn_last_error(None))
    return out
