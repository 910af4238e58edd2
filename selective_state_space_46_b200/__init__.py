"""B200-native (sm_100a) Mamba-1 selective scan: Python binding of libmssm.so.

This module only marshals arguments: it turns torch tensors into the C ABI's
``mssm_tensor`` descriptors (pointer, dtype, shape, strides) and calls the
entry points declared in ``include/mssm.h`` with the same names.  Every step of
the computation runs in the library's CUDA kernels; there is no CPU or PyTorch
fallback, and importing fails loudly when the library has not been built.

Build the library with ``python selective_state_space_46_b200/build.py``.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Tuple

import torch

__all__ = [
    "MssmError", "mssm_selective_scan_fwd", "mssm_selective_scan_fwd_noalloc", "mssm_state_update",
    "mssm_state_update_ex",
    "mssm_get_error", "mssm_set_option", "mssm_shutdown", "mssm_version", "mssm_status_string",
    "mssm_last_error", "selective_scan_fwd", "state_update", "lib_path",
    "MSSM_OPT_FORCE_GENERAL_A", "MSSM_OPT_CHUNK_LEN", "MSSM_OPT_KERNEL_TIMING", "MSSM_OPT_SCHEDULE", "SCHEDULES",
    "MSSM_OPT_DECODE_PATH", "DECODE_PATHS", "MSSM_OPT_TEST_HOOKS", "MSSM_OPT_ROWS_PER_CTA", "MSSM_OPT_ROWS_PER_THREAD", "MSSM_ERR_TIMEOUT", "mssm_kernel_stats", "mssm_scan_plan",
    "mssm_selective_scan_fwd_ex", "MSSM_DISC_EULER", "MSSM_DISC_ZOH",
    "mssm_causal_conv1d_fwd", "mssm_causal_conv1d_update", "causal_conv1d", "causal_conv1d_update",
    "mssm_selective_scan_bwd", "selective_scan_bwd",
    "MSSM_OPT_GATED_WARPS", "MSSM_OPT_GATED_SPLIT", "MSSM_OPT_W4_PLAN", "MSSM_OPT_GATED_STEP_ROWS", "mssm_gated_scan_fwd", "mssm_gated_scan_bwd", "mssm_gated_state_update",
    "gated_scan_fwd", "gated_scan_bwd", "gated_state_update",
    "mssm_w4_pack", "mssm_w4_linear", "W4Weight", "w4_pack", "w4_linear",
    "KERNEL_KINDS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libmssm.so")
if not os.path.exists(lib_path):
    raise ImportError(f"{lib_path} is missing: build it with `python selective_state_space_46_b200/build.py` "
                      "(nvcc, sm_100a); there is no fallback implementation")
_lib = ctypes.CDLL(lib_path)


class _Missing:
    """Stands for the descriptor writer where it cannot be loaded: the operators that use it say so when they are called."""

    def __init__(self, cause):
        self._cause = cause

    def __getattr__(self, name):
        raise ImportError("the binding's descriptor writer (_marshal.so), which the gated recurrence and the 4-bit linear map "
                          "use, is missing or was built for another torch: build it with "
                          "`python selective_state_space_46_b200/build.py`") from self._cause


try:
    from . import _marshal
except ImportError as e:
    _marshal = _Missing(e)

MSSM_F32, MSSM_BF16 = 0, 1
MSSM_OK, MSSM_ERR_INVALID_ARG, MSSM_ERR_UNSUPPORTED, MSSM_ERR_CUDA, MSSM_ERR_TIMEOUT = 0, 1, 2, 3, 4
MSSM_OPT_FORCE_GENERAL_A, MSSM_OPT_CHUNK_LEN, MSSM_OPT_KERNEL_TIMING, MSSM_OPT_SCHEDULE = 1, 2, 3, 4
MSSM_OPT_DECODE_PATH = 5
MSSM_OPT_TEST_HOOKS = 6
MSSM_OPT_ROWS_PER_CTA = 7
MSSM_OPT_ROWS_PER_THREAD = 8
MSSM_OPT_GATED_WARPS, MSSM_OPT_GATED_SPLIT, MSSM_OPT_W4_PLAN, MSSM_OPT_GATED_STEP_ROWS = 9, 10, 11, 12
MSSM_DISC_EULER, MSSM_DISC_ZOH = 0, 1
SCHEDULES = {"forward": 1, "summaries+forward": 2, "chained": 3, "fused": 4, "split": 5}
DECODE_PATHS = {"stream": 1, "bulk_tile": 2, "per_row": 3}
KERNEL_KINDS = ("scan_chunk_state", "scan_out", "state_update", "conv", "scan_bwd", "gated_scan", "gated_bwd",
                "gated_step", "w4_linear")


class mssm_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class mssm_scan_ext(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("discretization", ctypes.c_int32),
                ("h0", ctypes.POINTER(mssm_tensor)), ("cu_seqlens", ctypes.POINTER(mssm_tensor)),
                ("max_seqlen", ctypes.c_int64)]


_P = ctypes.POINTER(mssm_tensor)
_V = ctypes.c_void_p
_lib.mssm_selective_scan_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _P, _V]
_lib.mssm_selective_scan_fwd.restype = ctypes.c_int
_lib.mssm_selective_scan_fwd_ex.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int,
                                            ctypes.POINTER(mssm_scan_ext), _P, _P, _V]
_lib.mssm_selective_scan_fwd_ex.restype = ctypes.c_int
_lib.mssm_selective_scan_fwd_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _P, _V]
_lib.mssm_selective_scan_fwd_noalloc.restype = ctypes.c_int
_lib.mssm_state_update.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _V]
_lib.mssm_state_update.restype = ctypes.c_int
_lib.mssm_state_update_ex.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _V]
_lib.mssm_state_update_ex.restype = ctypes.c_int
_lib.mssm_selective_scan_bwd.argtypes = [_P] * 8 + [ctypes.c_int] + [_P] * 9 + [_V]
_lib.mssm_selective_scan_bwd.restype = ctypes.c_int
_lib.mssm_causal_conv1d_fwd.argtypes = [_P, _P, _P, _P, ctypes.c_int64, ctypes.c_int, _P, _V]
_lib.mssm_causal_conv1d_fwd.restype = ctypes.c_int
_lib.mssm_causal_conv1d_update.argtypes = [_P, _P, _P, _P, ctypes.c_int, _P, _V]
_lib.mssm_causal_conv1d_update.restype = ctypes.c_int
_lib.mssm_status_string.argtypes = [ctypes.c_int]
_lib.mssm_status_string.restype = ctypes.c_char_p
_lib.mssm_last_error.restype = ctypes.c_char_p
_lib.mssm_get_error.argtypes = [_V]
_lib.mssm_get_error.restype = ctypes.c_int
_lib.mssm_set_option.argtypes = [ctypes.c_int, ctypes.c_int64]
_lib.mssm_set_option.restype = ctypes.c_int
_lib.mssm_shutdown.restype = ctypes.c_int
_lib.mssm_version.restype = ctypes.c_char_p
_lib.mssm_kernel_stats_all.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_double), ctypes.c_int]
_lib.mssm_kernel_stats_all.restype = ctypes.c_int
# the entry points below take descriptor addresses from _Descs
_lib.mssm_gated_scan_fwd.argtypes = [_V] * 11
_lib.mssm_gated_scan_fwd.restype = ctypes.c_int
_lib.mssm_gated_scan_bwd.argtypes = [_V] * 20
_lib.mssm_gated_scan_bwd.restype = ctypes.c_int
_lib.mssm_gated_state_update.argtypes = [_V] * 8 + [ctypes.c_float, _V, _V]
_lib.mssm_gated_state_update.restype = ctypes.c_int
_lib.mssm_w4_packed_sizes.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)] * 2
_lib.mssm_w4_packed_sizes.restype = ctypes.c_int
_lib.mssm_w4_pack.argtypes = [_V] * 3 + [ctypes.c_int64] * 2 + [_V] * 4
_lib.mssm_w4_pack.restype = ctypes.c_int
_lib.mssm_w4_linear.argtypes = [_V] * 4 + [ctypes.c_int64] + [_V] * 3
_lib.mssm_w4_linear.restype = ctypes.c_int
_lib.mssm_scan_plan.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int64),
                                ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int)]
_lib.mssm_scan_plan.restype = ctypes.c_int
_lib.mssm_scan_plan_packed.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int)]
_lib.mssm_scan_plan_packed.restype = ctypes.c_int


class mssm_scan_plan_info(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("schedule", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32),
                ("rows_per_thread", ctypes.c_int32), ("chunk_len", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("grid", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib.mssm_scan_plan_query.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                      ctypes.c_int, ctypes.POINTER(mssm_scan_plan_info)]
_lib.mssm_scan_plan_query.restype = ctypes.c_int


class MssmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{mssm_status_string(status)}: {message}")
        self.status = status


MSSM_I32, MSSM_U8 = 2, 3
_DT = {torch.float32: MSSM_F32, torch.bfloat16: MSSM_BF16, torch.int32: MSSM_I32, torch.uint8: MSSM_U8}


def _desc(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.dim() > 4:
        raise ValueError("tensors have at most 4 dims")
    d = mssm_tensor()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _DT.get(t.dtype, -1)
    d.ndim = t.dim()
    for i, (s, st) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = s
        d.stride[i] = st
    return ctypes.byref(d), d


def _ref(x):
    return None if x is None else x[0]


def _stream(stream, ref: torch.Tensor):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(ref.device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int):
    if status != MSSM_OK:
        raise MssmError(status, mssm_last_error())


def mssm_status_string(status: int) -> str:
    return _lib.mssm_status_string(status).decode()


def mssm_last_error() -> str:
    return _lib.mssm_last_error().decode()


def mssm_version() -> str:
    return _lib.mssm_version().decode()


def mssm_set_option(option: int, value: int) -> None:
    _check(_lib.mssm_set_option(option, value))


def mssm_shutdown() -> None:
    _check(_lib.mssm_shutdown())


def mssm_kernel_stats(reset: bool = False) -> dict:
    """Launch counts and (when MSSM_OPT_KERNEL_TIMING is on) timed launches and summed ms, per kernel kind."""
    n = len(KERNEL_KINDS)
    launches = (ctypes.c_int64 * n)()
    timed = (ctypes.c_int64 * n)()
    ms = (ctypes.c_double * n)()
    _check(_lib.mssm_kernel_stats_all(n, launches, timed, ms, int(reset)))
    return {k: {"launches": launches[i], "timed": timed[i], "ms": ms[i]} for i, k in enumerate(KERNEL_KINDS)}


def mssm_scan_plan(Bt: int, D: int, L: int, sm_count: int = 0, total_len: int = -1, io_dtype: str = "bf16") -> dict:
    """Launch plan of the scan for a [Bt, D, L] problem, or for Bt packed sequences of at most
    L steps summing to ``total_len``, with ``io_dtype`` ('bf16' or 'f32') I/O (mssm_scan_plan_query;
    host only, launches nothing)."""
    info = mssm_scan_plan_info()
    info.struct_size = ctypes.sizeof(mssm_scan_plan_info)
    dt = {"bf16": MSSM_BF16, "f32": MSSM_F32}[io_dtype]
    _check(_lib.mssm_scan_plan_query(Bt, D, L, total_len, dt, sm_count, ctypes.byref(info)))
    return {"rows_per_cta": info.rows_per_cta, "rows_per_thread": info.rows_per_thread,
            "chunk_len": info.chunk_len, "n_chunks": info.n_chunks, "grid": info.grid,
            "schedule": ("forward", "summaries+forward", "chained", "fused", "split")[info.schedule]}


def mssm_get_error(stream=None) -> None:
    s = ctypes.c_void_p(None) if stream is None else (
        ctypes.c_void_p(stream.cuda_stream) if isinstance(stream, torch.cuda.Stream) else ctypes.c_void_p(int(stream)))
    _check(_lib.mssm_get_error(s))


def mssm_selective_scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus_flag, out, last_state,
                            stream=None) -> None:
    """Marshal torch tensors into ``mssm_selective_scan_fwd`` (see include/mssm.h)."""
    ds = [_desc(t) for t in (u, delta, A, B, C, D, z, delta_bias, out, last_state)]
    _check(_lib.mssm_selective_scan_fwd(*[_ref(x) for x in ds[:8]], int(softplus_flag),
                                        _ref(ds[8]), _ref(ds[9]), _stream(stream, u)))


def mssm_selective_scan_fwd_ex(u, delta, A, B, C, D, z, delta_bias, softplus_flag, out, last_state,
                               h0=None, discretization=MSSM_DISC_EULER, cu_seqlens=None, max_seqlen=0,
                               stream=None) -> None:
    """Marshal torch tensors into ``mssm_selective_scan_fwd_ex``: the scan from an initial
    state ``h0`` (None: zero) with the given discretisation, over packed sequences when
    ``cu_seqlens`` (int32 device offsets) and ``max_seqlen`` are given (see include/mssm.h)."""
    ds = [_desc(t) for t in (u, delta, A, B, C, D, z, delta_bias, out, last_state)]
    dh = _desc(h0)
    dc = _desc(cu_seqlens)
    ext = mssm_scan_ext(ctypes.sizeof(mssm_scan_ext), int(discretization),
                        None if dh is None else ctypes.pointer(dh[1]),
                        None if dc is None else ctypes.pointer(dc[1]), int(max_seqlen))
    _check(_lib.mssm_selective_scan_fwd_ex(*[_ref(x) for x in ds[:8]], int(softplus_flag), ctypes.byref(ext),
                                           _ref(ds[8]), _ref(ds[9]), _stream(stream, u)))


def mssm_selective_scan_fwd_noalloc(u, delta, A, B, C, D, z, delta_bias, softplus_flag, out, last_state,
                                    stream=None) -> None:
    """Marshal torch tensors into ``mssm_selective_scan_fwd_noalloc``: the same scan for
    callers that cannot allocate device memory during the call (see include/mssm.h)."""
    ds = [_desc(t) for t in (u, delta, A, B, C, D, z, delta_bias, out, last_state)]
    _check(_lib.mssm_selective_scan_fwd_noalloc(*[_ref(x) for x in ds[:8]], int(softplus_flag),
                                                _ref(ds[8]), _ref(ds[9]), _stream(stream, u)))


def mssm_state_update(state, x, dt, A, B, C, D, z, out, stream=None) -> None:
    """Marshal torch tensors into ``mssm_state_update`` (state updated in place)."""
    ds = [_desc(t) for t in (state, x, dt, A, B, C, D, z, out)]
    _check(_lib.mssm_state_update(*[_ref(v) for v in ds], _stream(stream, x)))


def mssm_state_update_ex(state, x, dt, A, B, C, D, z, dt_bias, softplus_flag, out,
                         discretization=MSSM_DISC_EULER, stream=None) -> None:
    """Marshal torch tensors into ``mssm_state_update_ex`` (state updated in place)."""
    ds = [_desc(t) for t in (state, x, dt, A, B, C, D, z, dt_bias)]
    do = _desc(out)
    _check(_lib.mssm_state_update_ex(*[_ref(v) for v in ds], int(softplus_flag), int(discretization), _ref(do),
                                     _stream(stream, x)))


def mssm_selective_scan_bwd(u, delta, A, B, C, D, z, delta_bias, softplus_flag, dout, du, ddelta, dA, dB, dC,
                            dD, dz, ddelta_bias, stream=None) -> None:
    """Marshal torch tensors into ``mssm_selective_scan_bwd`` (see include/mssm.h)."""
    ds = [_desc(t) for t in (u, delta, A, B, C, D, z, delta_bias)]
    gs = [_desc(t) for t in (dout, du, ddelta, dA, dB, dC, dD, dz, ddelta_bias)]
    _check(_lib.mssm_selective_scan_bwd(*[_ref(x) for x in ds], int(softplus_flag), *[_ref(x) for x in gs],
                                        _stream(stream, u)))


def selective_scan_bwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, dout=None,
                       stream=None) -> dict:
    """Allocate the gradients with torch and run the backward scan on the GPU."""
    f32 = dict(device=u.device, dtype=torch.float32)
    g = dict(du=torch.empty_like(u), ddelta=torch.empty_like(u), dA=torch.empty(A.shape, **f32),
             dB=torch.empty(B.shape, **f32), dC=torch.empty(C.shape, **f32),
             dD=None if D is None else torch.empty(D.shape, **f32),
             dz=None if z is None else torch.empty_like(z),
             ddelta_bias=None if delta_bias is None else torch.empty(delta_bias.shape, **f32))
    mssm_selective_scan_bwd(u, delta, A, B, C, D, z, delta_bias, softplus, dout, g["du"], g["ddelta"], g["dA"],
                            g["dB"], g["dC"], g["dD"], g["dz"], g["ddelta_bias"], stream)
    return g


def mssm_causal_conv1d_fwd(x, weight, bias, out, cu_seqlens=None, max_seqlen=0, silu_flag=True,
                           stream=None) -> None:
    """Marshal torch tensors into ``mssm_causal_conv1d_fwd`` (see include/mssm.h)."""
    ds = [_desc(t) for t in (x, weight, bias, cu_seqlens)]
    _check(_lib.mssm_causal_conv1d_fwd(*[_ref(v) for v in ds], int(max_seqlen), int(silu_flag), _ref(_desc(out)),
                                       _stream(stream, x)))


def mssm_causal_conv1d_update(conv_state, x, weight, bias, out, silu_flag=True, stream=None) -> None:
    """Marshal torch tensors into ``mssm_causal_conv1d_update`` (conv_state updated in place)."""
    ds = [_desc(t) for t in (conv_state, x, weight, bias)]
    _check(_lib.mssm_causal_conv1d_update(*[_ref(v) for v in ds], int(silu_flag), _ref(_desc(out)),
                                          _stream(stream, x)))


class _Block(threading.local):
    """A thread's block of ``mssm_tensor`` descriptors, written in place by ``_marshal``, and of one
    ``mssm_gated_ext`` behind them."""
    MOST = 20
    EXT = struct.Struct("ifQQ")  # struct_size, decay_scale, h0, cu_seqlens

    def __init__(self):
        end = self.MOST * ctypes.sizeof(mssm_tensor)
        self.buffer = ctypes.create_string_buffer(end + self.EXT.size)
        self.base = ctypes.addressof(self.buffer)
        self.ext_at, self.ext = end, self.base + end

    def gated_ext(self, decay_scale, h0, cu_seqlens):
        self.EXT.pack_into(self.buffer, self.ext_at, self.EXT.size, decay_scale, h0 or 0, cu_seqlens or 0)
        return self.ext


class mssm_gated_ext(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("decay_scale", ctypes.c_float),
                ("h0", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p)]


assert ctypes.sizeof(mssm_tensor) == 80 and ctypes.sizeof(mssm_gated_ext) == _Block.EXT.size
_block = _Block()
_SCAN = ctypes.cast(_lib.mssm_gated_scan_fwd, ctypes.c_void_p).value
_SCAN_BWD = ctypes.cast(_lib.mssm_gated_scan_bwd, ctypes.c_void_p).value
_GRADS = ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dh0")
_STEP = ctypes.cast(_lib.mssm_gated_state_update, ctypes.c_void_p).value
_LINEAR = ctypes.cast(_lib.mssm_w4_linear, ctypes.c_void_p).value


def _call(stream, device, fn, *args):
    """A library call on a stream of the tensors' device, which is made current for it."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != MSSM_OK:
        _check(status)


class _allocating_on:
    """Tensors allocated here belong to the stream that the call runs on."""

    def __init__(self, stream, device):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            # torch takes the address 0 for no address, and then makes a stream of its own
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
        self.guard = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def mssm_gated_scan_fwd(x, r, i, lam, r_bias, i_bias, z, out, last_state, decay_scale=8.0, h0=None, cu_seqlens=None,
                        stream=None) -> None:
    """Marshal torch tensors into ``mssm_gated_scan_fwd`` (see include/mssm.h)."""
    b = _block
    dev, *d = _marshal.describe(b.base, x, r, i, lam, r_bias, i_bias, z, out, last_state, h0, cu_seqlens)
    _call(stream, dev, _lib.mssm_gated_scan_fwd, *d[:7], b.gated_ext(decay_scale, d[9], d[10]), d[7], d[8])


def mssm_gated_scan_bwd(x, r, i, lam, r_bias, i_bias, z, dout, dlast_state, dx, dr, di, dz, dlam, dr_bias, di_bias,
                        dh0, workspace=None, decay_scale=8.0, h0=None, cu_seqlens=None, stream=None) -> None:
    """Marshal torch tensors into ``mssm_gated_scan_bwd`` (see include/mssm.h)."""
    b = _block
    dev, *d = _marshal.describe(b.base, x, r, i, lam, r_bias, i_bias, z, dout, dlast_state, dx, dr, di, dz, dlam,
                                dr_bias, di_bias, dh0, workspace, h0, cu_seqlens)
    _call(stream, dev, _lib.mssm_gated_scan_bwd, *d[:7], b.gated_ext(decay_scale, d[18], d[19]), *d[7:18])


def mssm_gated_state_update(state, x, r, i, lam, r_bias, i_bias, z, out, decay_scale=8.0, stream=None) -> None:
    """Marshal torch tensors into ``mssm_gated_state_update`` (state updated in place)."""
    dev, *d, o = _marshal.describe(_block.base, state, x, r, i, lam, r_bias, i_bias, z, out)
    _call(stream, dev, _lib.mssm_gated_state_update, *d, decay_scale, o)


def mssm_w4_pack(codes, scales, zeros, in_features, group_size, qweight, qscales, qzeros, stream=None) -> None:
    """Marshal torch tensors into ``mssm_w4_pack`` (see include/mssm.h)."""
    dev, *d = _marshal.describe(_block.base, codes, scales, zeros, qweight, qscales, qzeros)
    _call(stream, dev, _lib.mssm_w4_pack, *d[:3], in_features, group_size, *d[3:])


def mssm_w4_linear(x, qweight, qscales, qzeros, group_size, bias, out, stream=None) -> None:
    """Marshal torch tensors into ``mssm_w4_linear`` (see include/mssm.h)."""
    dev, *d, b, o = _marshal.describe(_block.base, x, qweight, qscales, qzeros, bias, out)
    _call(stream, dev, _lib.mssm_w4_linear, *d, group_size, b, o)


# --------------------------------------------------------------------------
# allocation conveniences (torch allocates; the library computes)
# --------------------------------------------------------------------------

def causal_conv1d(x, weight, bias=None, silu=True, cu_seqlens=None, max_seqlen=None, out=None,
                  stream=None) -> torch.Tensor:
    """Causal depthwise conv1d (+ SiLU) of ``x`` [Bt, D, L] on the GPU; returns ``out``."""
    if not x.is_cuda:
        raise ValueError("causal_conv1d runs on CUDA tensors only")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if cu_seqlens.numel() > 1 else 0
    mssm_causal_conv1d_fwd(x, weight, bias, out, cu_seqlens, max_seqlen or 0, silu, stream)
    return out


def causal_conv1d_update(conv_state, x, weight, bias=None, silu=True, out=None, stream=None) -> torch.Tensor:
    """One decode step of the conv on the GPU (``conv_state`` updated in place); returns ``out``."""
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    mssm_causal_conv1d_update(conv_state, x, weight, bias, out, silu, stream)
    return out

def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                       out=None, last_state=None, return_last_state=True, h0=None, zoh=False,
                       cu_seqlens=None, max_seqlen=None,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Allocate ``out`` (and ``last_state``) with torch and run the scan on the GPU
    (from ``h0`` when given; zero-order-hold input term when ``zoh``; packed sequences
    when ``cu_seqlens`` is given, with ``max_seqlen`` read back from it if omitted)."""
    if not u.is_cuda:
        raise ValueError("selective_scan_fwd runs on CUDA tensors only")
    if out is None:
        out = torch.empty_like(u, memory_format=torch.contiguous_format)
    nstate = u.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if last_state is None and return_last_state:
        last_state = torch.empty(nstate, u.shape[1], A.shape[1], device=u.device, dtype=torch.float32)
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if nstate > 0 else 0
    if h0 is None and not zoh and cu_seqlens is None:
        mssm_selective_scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, out, last_state, stream)
    else:
        mssm_selective_scan_fwd_ex(u, delta, A, B, C, D, z, delta_bias, softplus, out, last_state, h0=h0,
                                   discretization=MSSM_DISC_ZOH if zoh else MSSM_DISC_EULER,
                                   cu_seqlens=cu_seqlens, max_seqlen=max_seqlen or 0, stream=stream)
    return out, last_state


def state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None,
                 zoh=False, stream=None) -> torch.Tensor:
    """Run one decode step on the GPU (``state`` updated in place); returns ``out``."""
    if not x.is_cuda:
        raise ValueError("state_update runs on CUDA tensors only")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    mssm_state_update_ex(state, x, dt, A, B, C, D, z, dt_bias, softplus, out,
                         discretization=MSSM_DISC_ZOH if zoh else MSSM_DISC_EULER, stream=stream)
    return out


def gated_scan_fwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, c=8.0, h0=None, cu_seqlens=None, out=None,
                   last_state=None, return_last_state=True,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The real-gated linear recurrence over ``x`` [Bt, D, L] with recurrence gate ``r`` and input gate
    ``i`` (both before bias and sigmoid), decay rate ``c * softplus(lam)`` and optional silu gate ``z``,
    from ``h0`` [S, D] when given, over packed sequences when ``cu_seqlens`` is.  Returns ``(out,
    last_state)``; steps outside every packed sequence are not written."""
    both = _marshal.scan(_SCAN, x, r, i, lam, r_bias, i_bias, z, c, h0, cu_seqlens, out, last_state, return_last_state,
                         stream)
    if type(both) is int:
        _check(both)
    return both


def gated_scan_bwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, dout=None, c=8.0, h0=None, cu_seqlens=None,
                   dlast_state=None, stream=None) -> dict:
    """Allocate the gradients with torch and run the gated recurrence's backward pass: ``dx, dr, di, dz,
    dlam, dr_bias, di_bias, dh0`` (None where the input is; ``dh0`` is given with ``h0``).  Gradients at steps
    outside every packed sequence are not written."""
    g = _marshal.scan_bwd(_SCAN_BWD, x, r, i, lam, r_bias, i_bias, z, c, h0, cu_seqlens, dout, dlast_state, stream)
    if type(g) is int:
        _check(g)
    return dict(zip(_GRADS, g))


def gated_state_update(state, x, r, i, lam, r_bias=None, i_bias=None, z=None, c=8.0, out=None,
                       stream=None) -> torch.Tensor:
    """One decode step of the gated recurrence on ``x`` [Bt, D] (``state`` [Bt, D] updated in place);
    returns ``out``."""
    out = _marshal.step(_STEP, state, x, r, i, lam, r_bias, i_bias, z, c, out, stream)
    if type(out) is int:
        _check(out)
    return out


class W4Weight:
    """A weight of 4-bit codes with group scales, laid out for ``w4_linear`` by ``w4_pack``."""

    __slots__ = ("qweight", "qscales", "qzeros", "in_features", "out_features", "group_size")

    def __init__(self, qweight, qscales, qzeros, in_features, out_features, group_size):
        self.qweight, self.qscales, self.qzeros = qweight, qscales, qzeros
        self.in_features, self.out_features, self.group_size = in_features, out_features, group_size


def w4_pack(codes, scales, zeros=None, in_features=None, group_size=128, stream=None) -> W4Weight:
    """Lay out a weight of 4-bit codes: ``codes`` [N, (K + 1) / 2] uint8 (input 2j in the low nibble of byte j,
    2j + 1 in the high one), ``scales`` [N, G] fp32 or bf16 with G = ceil(K / group_size), ``zeros`` [N, G] uint8
    (None: 8).  ``in_features`` is K, needed when it is odd (default: two per byte)."""
    if codes.dim() != 2:
        raise ValueError("codes: expected 2 dims [N, (K + 1) / 2]")
    n, k = codes.shape[0], int(2 * codes.shape[1] if in_features is None else in_features)
    words, groups = ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.mssm_w4_packed_sizes(n, k, group_size, ctypes.byref(words), ctypes.byref(groups)))
    with _allocating_on(stream, codes.device):
        q = torch.empty(words.value, device=codes.device, dtype=torch.int32)
        qs = torch.empty(groups.value, device=codes.device, dtype=scales.dtype)
        qz = None if zeros is None else torch.empty(groups.value, device=codes.device, dtype=torch.uint8)
    mssm_w4_pack(codes, scales, zeros, k, group_size, q, qs, qz, stream)
    return W4Weight(q, qs, qz, k, n, group_size)


def w4_linear(x, weight: W4Weight, bias=None, out=None, stream=None) -> torch.Tensor:
    """``x`` [M, K] times the packed weight's transpose, plus ``bias`` [N]; returns ``out`` [M, N]."""
    if x.dim() != 2 or x.shape[1] != weight.in_features:
        raise ValueError(f"x: expected [M, {weight.in_features}], got {list(x.shape)}")
    if out is not None and out.shape != (x.shape[0], weight.out_features):
        raise ValueError(f"out: expected [{x.shape[0]}, {weight.out_features}], got {list(out.shape)}")
    out = _marshal.linear(_LINEAR, x, weight.qweight, weight.qscales, weight.qzeros, weight.group_size, bias,
                          weight.out_features, out, stream)
    if type(out) is int:
        _check(out)
    return out
