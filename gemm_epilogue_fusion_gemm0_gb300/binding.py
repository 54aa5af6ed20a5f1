"""ctypes binding of libcoda.so (include/coda.h), same names as the C ABI.

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity and passed as raw device pointers together with the current CUDA
stream.  Every step of the computation runs in the library's kernels; if the
library is missing this module raises at import time.  A process started with
CODA_CHECKED_BUILD=1 loads the checked build (libcoda_checked.so) instead.

With stream= (a torch stream or a raw cudaStream_t handle) a call is enqueued there
and its outputs and workspace, where they are not given, are that stream's memory.
As with any work on another stream, the caller orders it behind whatever wrote the
inputs, keeps them until it is done, and waits for it before reading the outputs.
"""

from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH, LIB_PATH_CHECKED

LIB = LIB_PATH_CHECKED if os.environ.get("CODA_CHECKED_BUILD") == "1" else LIB_PATH

if not os.path.exists(LIB):
    raise ImportError(
        f"{os.path.basename(LIB)} not found at {LIB}: build it first "
        "(python -c 'import __graft_entry__ as g; g.build()')"
    )

_lib = ctypes.CDLL(LIB)

CODA_OK = 0
CODA_ERR_INVALID_ARG = 1
CODA_ERR_UNSUPPORTED_SHAPE = 2
CODA_ERR_MISALIGNED = 3
CODA_ERR_WORKSPACE_TOO_SMALL = 4
CODA_ERR_LAUNCH = 5
CODA_ERR_DEVICE_TIMEOUT = 6
CODA_ERR_NO_DEVICE = 7
CODA_ERR_UNSUPPORTED_DEVICE = 8
CODA_ERR_DEVICE_BOUNDS = 9
STATUS_NAMES = {
    0: "CODA_OK",
    1: "CODA_ERR_INVALID_ARG",
    2: "CODA_ERR_UNSUPPORTED_SHAPE",
    3: "CODA_ERR_MISALIGNED",
    4: "CODA_ERR_WORKSPACE_TOO_SMALL",
    5: "CODA_ERR_LAUNCH",
    6: "CODA_ERR_DEVICE_TIMEOUT",
    7: "CODA_ERR_NO_DEVICE",
    8: "CODA_ERR_UNSUPPORTED_DEVICE",
    9: "CODA_ERR_DEVICE_BOUNDS",
}

_vp, _i64, _sz, _f32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint64
_st, _int = ctypes.c_int, ctypes.c_int

EXPORTS = {
    # name: (restype, argtypes)
    "coda_fwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_bwd_dgrad_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_fwd_unfused_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_fwd": (_st, [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "coda_fwd_unfused": (_st, [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "coda_bwd_dgrad": (_st, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "coda_get_device_status": (_st, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "coda_set_wait_timeout_ns": (None, [_u64]),
    "coda_status_string": (ctypes.c_char_p, [_st]),
    "coda_watchdog_selftest": (_st, [_u64, _vp]),
    "coda_set_launch_events": (None, [_vp, ctypes.c_int]),
    "coda_bwd_dgrad_noalloc": (_st, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "coda_set_mma_mode": (_st, [ctypes.c_int]),
    "coda_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_bwd": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                       _vp, _sz, _vp]),
    "coda_bwd_swiglu_dgrad_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "coda_bwd_swiglu_dgrad": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp,
                                    _vp, _vp, _vp, _sz, _vp]),
    "coda_fwd_swiglu": (_st, [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                              _sz, _vp]),
    "coda_get_mma_mode": (ctypes.c_int, []),
    "coda_set_fold_rowreduce": (_st, [ctypes.c_int]),
    "coda_set_split_tail": (_st, [ctypes.c_int]),
    "coda_set_col_plan": (_st, [ctypes.c_int]),
    "coda_set_serpentine_k": (_st, [ctypes.c_int]),
    "coda_get_serpentine_k": (ctypes.c_int, []),
    "coda_set_dgrad_pieces": (_st, [ctypes.c_int]),
    "coda_get_dgrad_pieces": (ctypes.c_int, []),
    "coda_dgrad_piece_plan": (ctypes.c_int, [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_int32)]),
    "coda_fwd_fp8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_fwd_fp8": (_st, [_vp, _f32, _vp, _f32, _vp, _vp, _vp, _f32, _f32, _f32, _i64, _i64, _i64, _vp,
                           _vp, _vp, _vp, _sz, _vp]),
    "coda_quant_q8": (_st, [_vp, _i64, _i64, _int, _vp, _vp, _vp]),
    "coda_dequant_q8": (_st, [_vp, _vp, _i64, _i64, _int, _vp, _vp]),
    "coda_add_rmsnorm_q8": (_st, [_vp, _vp, _vp, _f32, _i64, _i64, _vp, _vp, _vp, _vp]),
    "coda_matmul_q8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "coda_matmul_q8": (_st, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "coda_matmul_q8_plan": (_int, [_i64, _i64, _i64, _int, _int, _vp, _vp]),
    "coda_bwd_swiglu_dgrad_q8": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                       _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}

for _name, (_res, _args) in EXPORTS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class CodaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def status_string(status: int) -> str:
    return _lib.coda_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != CODA_OK:
        raise CodaError(status, where)


def _stream_ptr(stream, device=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)  # a raw cudaStream_t handle
    if device is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on {device}")
    return int(stream.cuda_stream)


def _dev(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# The current stream's raw handle without building a torch.cuda.Stream object (2 us of a call's
# host time on Grace); the public route where this torch does not have it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Call:
    """Marshalling for one call: every tensor must be a contiguous CUDA tensor
    of the stated dtype and shape on the device of the call's first tensor,
    and the C function runs with that device current (the C ABI works on the
    current device, so a tensor on another one would hand the kernels a
    pointer they cannot use)."""

    __slots__ = ("where", "device", "index", "stream", "user")

    def __init__(self, where: str, device: torch.device, stream=None):
        self.where, self.device = where, device
        self.index = device.index if device.type == "cuda" else None
        # the stream asked for, if any, and (once something is allocated) what to allocate it on
        self.stream, self.user = stream, None

    def empty(self, shape, dtype) -> torch.Tensor:
        """Memory for this call.  For a call on another stream than the current one it comes from
        that stream's memory: a block just freed on the current stream may still be in use there,
        and nothing orders the other stream behind that.  What is done with it on the
        current stream, before it is freed, is waited for before it is handed out again."""
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        handle = _stream_ptr(self.stream, self.device)
        if handle == _raw_stream(self.index):
            return torch.empty(shape, dtype=dtype, device=self.device)
        if self.user is None:
            # 1 is CUDA's handle of the legacy default stream, which torch knows as 0
            self.user = (self.stream if isinstance(self.stream, torch.cuda.Stream)
                         else torch.cuda.ExternalStream(0 if handle == 1 else handle,
                                                        device=self.device))
        with torch.cuda.stream(self.user):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def t(self, t, dtype, shape, name) -> int:
        # the common case in few steps; anything else is told apart (and raised) below
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                and t.is_contiguous() and t.get_device() == self.index):
            return t.data_ptr()
        p = _dev(t, dtype, shape, name)
        if t.device != self.device:
            raise ValueError(f"{self.where}: {name} is on {t.device}, the call's first tensor on "
                             f"{self.device}")
        return p

    def opt(self, t, dtype, shape, name):
        return None if t is None else self.t(t, dtype, shape, name)

    def out(self, t, dtype, shape, name) -> tuple:
        """An output and its address: `t` checked, or allocated (and then in need of no check)."""
        if t is None:
            t = self.empty(shape, dtype)
            return t, t.data_ptr()
        return t, self.t(t, dtype, shape, name)

    def scratch(self, ws, need: int) -> tuple:
        """The workspace, its address and its size: `ws` checked, or `need` bytes allocated (to be
        kept until the call is enqueued: freed memory is reused in stream order)."""
        if ws is None:
            need = max(need, 16)
            ws = self.empty(need, torch.uint8)
            return ws, ws.data_ptr(), need
        return (ws, *self.ws(ws))

    def ws(self, ws) -> tuple:
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
            raise TypeError(f"{self.where}: the workspace must be a contiguous CUDA tensor")
        if ws.get_device() != self.index:
            raise ValueError(f"{self.where}: the workspace is on {ws.device}, the call's first "
                             f"tensor on {self.device}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def run(self, fn, *args, stream=None) -> None:
        if self.index == torch.cuda.current_device():
            st = fn(*args, _raw_stream(self.index) if stream is None
                    else _stream_ptr(stream, self.device))
        else:
            with torch.cuda.device(self.device):
                st = fn(*args, _stream_ptr(stream, self.device))
        if st != CODA_OK:
            raise CodaError(st, self.where)


# --------------------------------------------------------------------------- sizes
def coda_fwd_workspace_bytes(M: int, d: int, N1: int) -> int:
    return int(_lib.coda_fwd_workspace_bytes(M, d, N1))


def coda_fwd_unfused_workspace_bytes(M: int, d: int, N1: int) -> int:
    return int(_lib.coda_fwd_unfused_workspace_bytes(M, d, N1))


def coda_bwd_dgrad_workspace_bytes(M: int, d: int, N1: int) -> int:
    return int(_lib.coda_bwd_dgrad_workspace_bytes(M, d, N1))


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device byte buffer of at least `nbytes` (torch allocates it)."""
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------- calls
def _fwd_common(fn, wsfn, x, W0, z, gamma, W1, eps, h, r, y, ws, stream):
    M, d = x.shape
    N1 = W1.shape[1]
    bf = torch.bfloat16
    c = _Call(fn.__name__, x.device, stream)
    ins = (c.t(x, bf, (M, d), "x"), c.t(W0, bf, (d, d), "W0"), c.t(z, bf, (M, d), "z"),
           c.t(gamma, bf, (d,), "gamma"), c.t(W1, bf, (d, N1), "W1"))
    h, hp = c.out(h, bf, (M, d), "h")
    r, rp = c.out(r, torch.float32, (M,), "r")
    y, yp = c.out(y, bf, (M, N1), "y")
    ws, wk, wkb = c.scratch(ws, wsfn(M, d, N1))
    c.run(fn, *ins, float(eps), M, d, N1, hp, rp, yp, wk, wkb, stream=stream)
    return h, r, y


def coda_fwd(x, W0, z, gamma, W1, eps, h=None, r=None, y=None, ws=None, stream=None):
    """Fused forward; returns (h, r, y).  Outputs are allocated if not given."""
    return _fwd_common(_lib.coda_fwd, coda_fwd_workspace_bytes, x, W0, z, gamma, W1, eps,
                       h, r, y, ws, stream)


def coda_fwd_unfused(x, W0, z, gamma, W1, eps, h=None, r=None, y=None, ws=None, stream=None):
    """Unfused reference sequence (measurement only); returns (h, r, y)."""
    return _fwd_common(_lib.coda_fwd_unfused, coda_fwd_unfused_workspace_bytes, x, W0, z, gamma,
                       W1, eps, h, r, y, ws, stream)


def coda_fwd_swiglu(x, W0, z, gamma, W1, eps, h=None, r=None, a=None, y=None, want_y=False,
                    ws=None, stream=None):
    """Fused forward with the SwiGLU gated activation; W1 = [W_gate | W_up].
    Returns (h, r, a) or (h, r, a, y) with want_y=True (pre-activation)."""
    M, d = x.shape
    N1 = W1.shape[1]
    bf = torch.bfloat16
    c = _Call("coda_fwd_swiglu", x.device, stream)
    ins = (c.t(x, bf, (M, d), "x"), c.t(W0, bf, (d, d), "W0"), c.t(z, bf, (M, d), "z"),
           c.t(gamma, bf, (d,), "gamma"), c.t(W1, bf, (d, N1), "W1"))
    h, hp = c.out(h, bf, (M, d), "h")
    r, rp = c.out(r, torch.float32, (M,), "r")
    a, ap = c.out(a, bf, (M, N1 // 2), "a")
    yp = None
    if want_y or y is not None:
        y, yp = c.out(y, bf, (M, N1), "y")
    ws, wk, wkb = c.scratch(ws, coda_fwd_workspace_bytes(M, d, N1))
    c.run(_lib.coda_fwd_swiglu, *ins, float(eps), M, d, N1, hp, rp, yp, ap, wk, wkb, stream=stream)
    return (h, r, a, y) if y is not None else (h, r, a)


def coda_fwd_fp8_workspace_bytes(M: int, d: int, N1: int) -> int:
    return int(_lib.coda_fwd_fp8_workspace_bytes(M, d, N1))


def coda_fwd_fp8(x_q, sx, W0_q, sW0, z, gamma, W1_q, sW1, s_hg, eps, h=None, r=None, y=None,
                 ws=None, stream=None):
    """FP8 forward: x_q, W0_q, W1_q are float8_e4m3fn (or uint8) code tensors with
    per-tensor scales; returns (h, r, y)."""
    M, d = x_q.shape
    N1 = W1_q.shape[1]
    bf = torch.bfloat16
    c = _Call("coda_fwd_fp8", x_q.device, stream)

    def code(t, shape, name):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"{name} must hold E4M3 codes (float8_e4m3fn or uint8)")
        return c.t(t, t.dtype, shape, name)

    ins = (code(x_q, (M, d), "x_q"), float(sx), code(W0_q, (d, d), "W0_q"), float(sW0),
           c.t(z, bf, (M, d), "z"), c.t(gamma, bf, (d,), "gamma"), code(W1_q, (d, N1), "W1_q"),
           float(sW1), float(s_hg), float(eps))
    h, hp = c.out(h, bf, (M, d), "h")
    r, rp = c.out(r, torch.float32, (M,), "r")
    y, yp = c.out(y, bf, (M, N1), "y")
    ws, wk, wkb = c.scratch(ws, coda_fwd_fp8_workspace_bytes(M, d, N1))
    c.run(_lib.coda_fwd_fp8, *ins, M, d, N1, hp, rp, yp, wk, wkb, stream=stream)
    return h, r, y


def coda_bwd_dgrad(dy, W1, h, r, gamma, dh=None, ws=None, stream=None):
    """Fused RMSNorm-branch data gradient; returns dh."""
    M, N1 = dy.shape
    d = W1.shape[0]
    bf = torch.bfloat16
    c = _Call("coda_bwd_dgrad", dy.device, stream)
    ins = (c.t(dy, bf, (M, N1), "dy"), c.t(W1, bf, (d, N1), "W1"), c.t(h, bf, (M, d), "h"),
           c.t(r, torch.float32, (M,), "r"), c.t(gamma, bf, (d,), "gamma"))
    dh, dhp = c.out(dh, bf, (M, d), "dh")
    ws, wk, wkb = c.scratch(ws, coda_bwd_dgrad_workspace_bytes(M, d, N1))
    c.run(_lib.coda_bwd_dgrad, *ins, M, d, N1, dhp, wk, wkb, stream=stream)
    return dh


def coda_bwd_swiglu_dgrad_workspace_bytes(M: int, d: int, N1: int, Dout: int) -> int:
    return int(_lib.coda_bwd_swiglu_dgrad_workspace_bytes(M, d, N1, Dout))


def coda_bwd_swiglu_dgrad(dout, W2, y, W1, h, r, gamma, dy=None, s=None, dh=None, ws=None,
                          stream=None):
    """SwiGLU backward (statistic formed upstream) + tile-local RMSNorm-branch
    data gradient; returns (dy, s, dh)."""
    M, Dout = dout.shape
    half = W2.shape[0]
    N1 = 2 * half
    d = W1.shape[0]
    bf = torch.bfloat16
    c = _Call("coda_bwd_swiglu_dgrad", dout.device, stream)
    ins = (c.t(dout, bf, (M, Dout), "dout"), c.t(W2, bf, (half, Dout), "W2"),
           c.t(y, bf, (M, N1), "y"), c.t(W1, bf, (d, N1), "W1"), c.t(h, bf, (M, d), "h"),
           c.t(r, torch.float32, (M,), "r"), c.t(gamma, bf, (d,), "gamma"))
    dy, dyp = c.out(dy, bf, (M, N1), "dy")
    s, sp = c.out(s, torch.float32, (M,), "s")
    dh, dhp = c.out(dh, bf, (M, d), "dh")
    ws, wk, wkb = c.scratch(ws, coda_bwd_swiglu_dgrad_workspace_bytes(M, d, N1, Dout))
    c.run(_lib.coda_bwd_swiglu_dgrad, *ins, M, d, N1, Dout, dyp, sp, dhp, wk, wkb, stream=stream)
    return dy, s, dh


# --------------------------------------------------------------------------- 8-bit operators
def _q8_scales(M: int, n: int, block: int) -> tuple:
    """Shape of the scales of [M, n] codes: one per row (block 0) or per row and `block` columns."""
    return (M, -(-n // block)) if block else (M,)


def coda_quant_q8(x, block=0, q=None, s=None, stream=None):
    """INT8 codes and scales of x [M, n]; a scale per row (block=0) or per row and 128
    columns (block=128, a checkpoint).  Returns (q, s)."""
    shape = M, n = x.shape
    if block not in (0, 128):
        raise ValueError(f"block must be 0 (a scale per row) or 128, got {block}")
    c = _Call("coda_quant_q8", x.device, stream)
    xp = c.t(x, torch.bfloat16, shape, "x")
    q, qp = c.out(q, torch.int8, shape, "q")
    s, sp = c.out(s, torch.float32, _q8_scales(M, n, block), "s")
    c.run(_lib.coda_quant_q8, xp, M, n, block, qp, sp, stream=stream)
    return q, s


def coda_dequant_q8(q, s, block=0, x=None, stream=None):
    """The values of codes q with scales s (as coda_quant_q8 gives them) in bf16; returns x."""
    shape = M, n = q.shape
    c = _Call("coda_dequant_q8", q.device, stream)
    if block not in (0, 128):
        raise ValueError(f"block must be 0 (a scale per row) or 128, got {block}")
    qp = c.t(q, torch.int8, shape, "q")
    sp = c.t(s, torch.float32, _q8_scales(M, n, block), "s")
    x, xp = c.out(x, torch.bfloat16, shape, "x")
    c.run(_lib.coda_dequant_q8, qp, sp, M, n, block, xp, stream=stream)
    return x


def coda_add_rmsnorm_q8(x, gamma, eps, z=None, h=None, q=None, s=None, stream=None):
    """Residual addition h = x + z and RMS norm with INT8 codes and a scale per token; returns
    (h, q, s).  Without z no h is written and x itself is returned in its place."""
    shape = M, d = x.shape
    if z is None and h is not None:
        raise ValueError("h is an output of the residual's addition: it needs z")
    c = _Call("coda_add_rmsnorm_q8", x.device, stream)
    bf = torch.bfloat16
    xp, gp = c.t(x, bf, shape, "x"), c.t(gamma, bf, (d,), "gamma")
    if z is None:
        h, hp, zp = x, None, None
    else:
        zp = c.t(z, bf, shape, "z")
        h, hp = c.out(h, bf, shape, "h")
    q, qp = c.out(q, torch.int8, shape, "q")
    s, sp = c.out(s, torch.float32, (M,), "s")
    c.run(_lib.coda_add_rmsnorm_q8, xp, zp, gp, float(eps), M, d, hp, qp, sp, stream=stream)
    return h, q, s


def coda_matmul_q8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(_lib.coda_matmul_q8_workspace_bytes(M, K, N))


def coda_matmul_q8_plan(M: int, K: int, N: int, sms: int, pairs: int, clusters) -> tuple:
    """The form that coda_matmul_q8 would take on such a device as (form, parts along K, tokens
    per CTA pair, two blocks per SM); form 0 refused, 1 few tokens, 2 mid-size, 3 whole GEMM."""
    fit, out = (ctypes.c_int32 * 3)(*clusters), (ctypes.c_int32 * 3)()
    form = int(_lib.coda_matmul_q8_plan(M, K, N, int(sms), int(pairs), fit, out))
    if form < 0:
        raise ValueError("coda_matmul_q8_plan: invalid arguments")
    return (form, int(out[0]), int(out[1]), bool(out[2]))


def coda_matmul_q8(a_q, a_s, W_q, w_s, z=None, y=None, ws=None, stream=None):
    """INT8 product y = a_s * w_s * (a_q @ W_q) (+ z), a scale per token (a_s [M]) and per channel
    (w_s [N]); W_q [K, N]; returns y (bf16).  No workspace is needed (or looked at) where
    coda_matmul_q8_workspace_bytes is 0."""
    M, K = a_q.shape
    N = W_q.shape[1]
    c = _Call("coda_matmul_q8", a_q.device, stream)
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    ap, asp = c.t(a_q, i8, (M, K), "a_q"), c.t(a_s, f32, (M,), "a_s")
    wp, wsp = c.t(W_q, i8, (K, N), "W_q"), c.t(w_s, f32, (N,), "w_s")
    zp = None if z is None else c.t(z, bf, (M, N), "z")
    y, yp = c.out(y, bf, (M, N), "y")
    need = _lib.coda_matmul_q8_workspace_bytes(M, K, N)
    ws, wk, wkb = c.scratch(ws, need) if need else (None, None, 0)
    c.run(_lib.coda_matmul_q8, ap, asp, wp, wsp, zp, M, K, N, yp, wk, wkb, stream=stream)
    return y


def coda_bwd_swiglu_dgrad_q8(dout, W2, y_q, y_s, W1, h, r, gamma, dy=None, s=None, dh=None, a=None,
                             want_a=False, ws=None, stream=None):
    """coda_bwd_swiglu_dgrad from an 8-bit checkpoint of the pre-activation (y_q, y_s as
    coda_quant_q8 with block=128 gives them); returns (dy, s, dh), or (dy, s, dh, a) with
    want_a=True (the gated activation recomputed from the checkpoint)."""
    M, Dout = dout.shape
    half = W2.shape[0]
    N1 = 2 * half
    d = W1.shape[0]
    c = _Call("coda_bwd_swiglu_dgrad_q8", dout.device, stream)
    bf, f32 = torch.bfloat16, torch.float32
    ins = (c.t(dout, bf, (M, Dout), "dout"), c.t(W2, bf, (half, Dout), "W2"),
           c.t(y_q, torch.int8, (M, N1), "y_q"), c.t(y_s, f32, _q8_scales(M, N1, 128), "y_s"),
           c.t(W1, bf, (d, N1), "W1"), c.t(h, bf, (M, d), "h"), c.t(r, f32, (M,), "r"),
           c.t(gamma, bf, (d,), "gamma"))
    dy, dyp = c.out(dy, bf, (M, N1), "dy")
    s, sp = c.out(s, f32, (M,), "s")
    dh, dhp = c.out(dh, bf, (M, d), "dh")
    ap = None
    if want_a or a is not None:
        a, ap = c.out(a, bf, (M, half), "a")
    ws, wk, wkb = c.scratch(ws, _lib.coda_bwd_swiglu_dgrad_workspace_bytes(M, d, N1, Dout))
    c.run(_lib.coda_bwd_swiglu_dgrad_q8, *ins, M, d, N1, Dout, dyp, sp, dhp, ap, wk, wkb,
          stream=stream)
    return (dy, s, dh, a) if a is not None else (dy, s, dh)


def coda_bwd_workspace_bytes(M: int, d: int, N1: int) -> int:
    return int(_lib.coda_bwd_workspace_bytes(M, d, N1))


def coda_bwd(dy, x, W0, W1, h, r, gamma, dh_res=None, out=None, ws=None, stream=None):
    """All gradients of the chain; returns dict dh (= dz), dx, dgamma, dW0, dW1."""
    M, N1 = dy.shape
    d = W1.shape[0]
    bf, f32 = torch.bfloat16, torch.float32
    o = dict(out or {})
    c = _Call("coda_bwd", dy.device, stream)
    ins = (c.t(dy, bf, (M, N1), "dy"), c.t(x, bf, (M, d), "x"), c.t(W0, bf, (d, d), "W0"),
           c.t(W1, bf, (d, N1), "W1"), c.t(h, bf, (M, d), "h"), c.t(r, f32, (M,), "r"),
           c.t(gamma, bf, (d,), "gamma"), c.opt(dh_res, bf, (M, d), "dh_res"))
    outs = []
    for name, dtype, shape in (("dh", bf, (M, d)), ("dx", bf, (M, d)), ("dgamma", f32, (d,)),
                               ("dW0", f32, (d, d)), ("dW1", f32, (d, N1))):
        if name in o:
            outs.append(c.t(o[name], dtype, shape, name))
        else:
            o[name], p = c.out(None, dtype, shape, name)
            outs.append(p)
    ws, wk, wkb = c.scratch(ws, coda_bwd_workspace_bytes(M, d, N1))
    c.run(_lib.coda_bwd, *ins, M, d, N1, *outs, wk, wkb, stream=stream)
    return o


def coda_get_device_status(stream=None) -> tuple[int, int]:
    """(status, detail) after synchronising the stream; clears the status."""
    detail = ctypes.c_uint32(0)
    st = _lib.coda_get_device_status(_stream_ptr(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def coda_set_mma_mode(mode: int) -> None:
    """0: single-CTA 128x256 tiles; 1: CTA-pair 256x256 tiles (tcgen05 cta_group::2)."""
    _check(_lib.coda_set_mma_mode(int(mode)), "coda_set_mma_mode")


def coda_set_fold_rowreduce(enable: int) -> None:
    """1: r is formed in GEMM1's epilogue (2 launches); 0: separate reduction (default)."""
    _check(_lib.coda_set_fold_rowreduce(int(enable)), "coda_set_fold_rowreduce")


def coda_set_split_tail(enable: int) -> None:
    """1: the forward's CTA-pair GEMMs split their last tiles along K (default); 0: whole tiles."""
    _check(_lib.coda_set_split_tail(int(enable)), "coda_set_split_tail")


def coda_set_col_plan(enable: int) -> None:
    """1 (2): the CTA-pair data gradients may use narrower column tiles, widths in steps of
    16 (64), that spread evenly over the pairs; 0: 256-column tiles (default)."""
    _check(_lib.coda_set_col_plan(int(enable)), "coda_set_col_plan")


def coda_set_serpentine_k(enable: int) -> None:
    """1: the CTA-pair data gradients load every other wave's K blocks backwards; 0: forwards
    (default)."""
    _check(_lib.coda_set_serpentine_k(int(enable)), "coda_set_serpentine_k")


def coda_get_serpentine_k() -> int:
    return int(_lib.coda_get_serpentine_k())


def coda_set_dgrad_pieces(enable: int) -> None:
    """1 (default): the CTA-pair data gradients may cut their last row blocks' tiles into K
    pieces when whole tiles would leave the last wave partly idle; 0: whole tiles."""
    _check(_lib.coda_set_dgrad_pieces(int(enable)), "coda_set_dgrad_pieces")


def coda_get_dgrad_pieces() -> int:
    return int(_lib.coda_get_dgrad_pieces())


def coda_dgrad_piece_plan(M: int, d: int, N1: int, npairs: int, tile_local: bool = False):
    """The data gradient's piece plan on `npairs` CTA pairs as (tiles whole, pieces,
    first levelled pair, levelling pieces per such pair), or None for whole tiles."""
    out = (ctypes.c_int32 * 4)()
    rc = int(_lib.coda_dgrad_piece_plan(M, d, N1, int(npairs), int(bool(tile_local)), out))
    if rc < 0:
        raise ValueError("coda_dgrad_piece_plan: invalid arguments")
    return tuple(int(v) for v in out) if rc == 1 else None


def coda_get_mma_mode() -> int:
    return int(_lib.coda_get_mma_mode())


def coda_set_wait_timeout_ns(ns: int) -> None:
    _lib.coda_set_wait_timeout_ns(int(ns))


def coda_watchdog_selftest(timeout_ns: int, stream=None) -> int:
    return int(_lib.coda_watchdog_selftest(int(timeout_ns), _stream_ptr(stream)))


_events_keepalive = None


def coda_set_launch_events(events) -> None:
    """Measurement hook: record events[k] after the k-th kernel launch of each
    following coda_* call (events: list of torch.cuda.Event, or None)."""
    global _events_keepalive
    if not events:
        _lib.coda_set_launch_events(None, 0)
        _events_keepalive = None
        return
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event lazily, on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
    _events_keepalive = (arr, events)
    _lib.coda_set_launch_events(ctypes.cast(arr, ctypes.c_void_p), len(events))


def raw() -> ctypes.CDLL:
    """The loaded library (for direct C-ABI calls, e.g. with bad arguments)."""
    return _lib
