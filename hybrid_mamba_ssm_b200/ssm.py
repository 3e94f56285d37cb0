"""Python binding of libssm (include/ssm.h): argument marshalling only.

Torch tensors supply device memory and the current CUDA stream; every step of
the scan runs in the library's kernels.  Importing this module loads
``libssm.so`` and raises ImportError if it is missing or cannot be loaded --
there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import warnings
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm.so")

SSM_F32, SSM_BF16, SSM_F16 = 0, 1, 2
STATUS_NAMES = {0: "SSM_OK", 1: "SSM_ERR_INVALID_ARG", 2: "SSM_ERR_UNSUPPORTED",
                3: "SSM_ERR_MISALIGNED", 4: "SSM_ERR_CUDA", 5: "SSM_ERR_TIMEOUT",
                6: "SSM_ERR_DEVICE_INPUT", 7: "SSM_ERR_RANGE", 8: "SSM_ERR_INTERNAL"}
SSM_ERR_TIMEOUT, SSM_ERR_DEVICE_INPUT, SSM_ERR_RANGE = 5, 6, 7
EXPORTS = ("ssd_chunk_scan", "ssd_chunk_scan_workspace_size", "ssm_state_update",
           "ssd_chunk_scan_slots", "ssm_state_update_slots", "causal_conv1d_fwd",
           "causal_conv1d_update", "ssm_state_update_multi", "ssm_state_commit",
           "causal_conv1d_update_multi", "ssm_gated_rmsnorm", "selective_scan_fwd",
           "selective_scan_saved_size", "selective_scan_workspace_size", "selective_scan_bwd",
           "selective_scan_bwd_workspace_size", "selective_state_update", "causal_conv1d_bwd",
           "causal_conv1d_bwd_workspace_size", "ssm_pool_copy", "ssm_pool_zero", "ssm_pool_compact",
           "ssm_pool_compact_workspace_size", "ssm_status_string",
           "ssm_version", "ssm_testing_scan_stalled", "ssm_testing_conv1d_stalled")
ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libssm.so is not built ({LIB_PATH}); run "
                          "`python -m hybrid_mamba_ssm_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.ssd_chunk_scan.restype = i
    lib.ssd_chunk_scan.argtypes = [i, i, vp, i, i, i, i, i, i, vp, vp, vp, vp, vp,
                                   vp, vp, i, vp, vp, vp, sz, vp, vp]
    lib.ssd_chunk_scan_noalloc.restype = i
    lib.ssd_chunk_scan_noalloc.argtypes = [i, i, vp, i, i, i, i, i, i, vp, vp, vp, vp, vp,
                                           vp, vp, i, vp, vp, vp, vp]
    lib.ssd_chunk_scan_workspace_size.restype = sz
    lib.ssd_chunk_scan_workspace_size.argtypes = [i] * 7
    lib.ssm_state_update.restype = i
    lib.ssm_state_update.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, i,
                                     vp, vp]
    lib.ssd_chunk_scan_slots.restype = i
    lib.ssd_chunk_scan_slots.argtypes = [i, i, vp, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp,
                                         vp, i, vp, i, vp, vp, i, vp, vp, vp]
    lib.ssm_state_update_slots.restype = i
    lib.ssm_state_update_slots.argtypes = [i, i, i, i, i, i, vp, i, vp, i, vp, vp, vp, vp, vp,
                                           vp, vp, vp, i, vp, vp, vp]
    lib.causal_conv1d_fwd.restype = i
    lib.causal_conv1d_fwd.argtypes = [i, i, vp, i, i, i, vp, vp, vp, i, vp, i, vp, vp, i, vp,
                                      vp, vp]
    lib.causal_conv1d_update.restype = i
    lib.causal_conv1d_update.argtypes = [i, i, i, i, vp, vp, vp, i, vp, i, vp, i, vp, vp, vp]
    lib.ssm_state_update_multi.restype = i
    lib.ssm_state_update_multi.argtypes = [i, i, i, i, i, i, i, vp, i, vp, vp, vp, vp, vp, vp,
                                           vp, vp, vp, vp, i, vp, vp, vp]
    lib.ssm_state_commit.restype = i
    lib.ssm_state_commit.argtypes = [i, i, i, i, i, vp, vp, vp, i, vp, vp, vp]
    lib.causal_conv1d_update_multi.restype = i
    lib.causal_conv1d_update_multi.argtypes = [i, i, i, i, i, vp, vp, vp, i, vp, i, vp, vp, i,
                                               vp, vp, vp]
    lib.ssm_gated_rmsnorm.restype = i
    lib.ssm_gated_rmsnorm.argtypes = [i, i, i, i, vp, i, vp, vp, ctypes.c_float, i, vp, vp]
    i64, ll = ctypes.c_int64, ctypes.c_longlong
    lib.selective_scan_fwd.restype = i
    lib.selective_scan_fwd.argtypes = [i, i, vp, i, i, i, i, vp, i64, i, vp, i64, vp, vp, i64, vp, i64,
                                       vp, vp, i64, vp, vp, vp, i, vp, vp, i, vp, vp, vp, sz, vp, vp]
    lib.selective_scan_saved_size.restype = sz
    lib.selective_scan_saved_size.argtypes = [i, ll, i, i]
    lib.selective_scan_workspace_size.restype = sz
    lib.selective_scan_workspace_size.argtypes = [i, ll, i, i, i]
    lib.selective_scan_bwd.restype = i
    lib.selective_scan_bwd.argtypes = [i, i, vp, i, i, i, i, vp, i64, vp, i64, i, vp, i64, vp, vp, i64,
                                       vp, i64, vp, vp, i64, vp, vp, vp] + [vp] * 10 + [sz, vp, vp]
    lib.selective_scan_bwd_workspace_size.restype = sz
    lib.selective_scan_bwd_workspace_size.argtypes = [i, ll, i, i, i]
    lib.selective_state_update.restype = i
    lib.selective_state_update.argtypes = [i, i, i, i, vp, i, vp, i, vp, i64, i, vp, i64, vp, vp, i64,
                                           vp, i64, vp, vp, i64, vp, i, vp, vp, vp]
    lib.causal_conv1d_bwd.restype = i
    lib.causal_conv1d_bwd.argtypes = [i, i, vp, i, i, i, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, sz,
                                      vp, vp]
    lib.causal_conv1d_bwd_workspace_size.restype = sz
    lib.causal_conv1d_bwd_workspace_size.argtypes = [ll, i, i]
    lib.ssm_pool_copy.restype = i
    lib.ssm_pool_copy.argtypes = [i, vp, i, i, vp, vp, vp, vp]
    lib.ssm_pool_zero.restype = i
    lib.ssm_pool_zero.argtypes = [i, vp, i, i, vp, vp, vp]
    lib.ssm_pool_compact.restype = i
    lib.ssm_pool_compact.argtypes = [i, vp, i, i, vp, vp, vp, sz, vp, vp]
    lib.ssm_pool_compact_workspace_size.restype = sz
    lib.ssm_pool_compact_workspace_size.argtypes = [i, i]
    lib.ssm_status_string.restype = ctypes.c_char_p
    lib.ssm_status_string.argtypes = [i]
    lib.ssm_version.restype = i
    u64 = ctypes.c_ulonglong
    lib.ssm_testing_scan_stalled.restype = i
    lib.ssm_testing_scan_stalled.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, vp, u64, vp, vp]
    lib.ssm_testing_conv1d_stalled.restype = i
    lib.ssm_testing_conv1d_stalled.argtypes = [i, i, i, i, vp, vp, vp, u64, vp, vp]
    return lib


lib = _load()


class _NoMarshal:
    """In the place of the _marshal module where there is none for this torch: every call takes the Python path."""

    @staticmethod
    def _none(*args):
        return None

    scan_fwd = scan_bwd = state_update = conv1d_bwd = pool_copy = pool_zero = pool_compact = _none


def _load_marshal():
    """The C++ side of the per-channel and pool calls (host code only, built
    against one torch).  Without it they launch the same kernels, with a few
    times the host time a call."""
    try:
        from . import _marshal
        built_for = getattr(_marshal, "torch_version", None)
        if built_for == str(torch.__version__):
            return _marshal
        why = f"it was built for torch {built_for}, this is {torch.__version__}"
    except ImportError as e:
        why = str(e)
    warnings.warn(f"_marshal.so is not used ({why}); calls take more host time.  To build it: "
                  "`python -m hybrid_mamba_ssm_b200.build`", RuntimeWarning, stacklevel=2)
    return _NoMarshal


_marshal = _load_marshal()


class DtParams(ctypes.Structure):
    """ssm_dt_params: dt <- clamp(softplus(dt + dt_bias[h])) inside the kernels."""
    _fields_ = [("dt_bias", ctypes.c_void_p), ("softplus", ctypes.c_int), ("clamp", ctypes.c_int),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


def _dt_params(dt_bias, dt_softplus, dt_limit):
    """A DtParams reference for the keyword arguments, or None when dt is final."""
    if dt_bias is None and not dt_softplus and dt_limit is None:
        return None
    _dev(dt_bias, "dt_bias", torch.float32)
    lo, hi = dt_limit if dt_limit is not None else (0.0, 0.0)
    p = DtParams(None if dt_bias is None else dt_bias.data_ptr(), int(bool(dt_softplus)),
                 int(dt_limit is not None), float(lo), float(hi))
    return ctypes.byref(p)


class Rounding(ctypes.Structure):
    """ssm_rounding: stochastic rounding of an fp16 state pool (Philox-4x32)."""
    _fields_ = [("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("philox_rounds", ctypes.c_int)]


def _state_format(pool, rounding):
    """(state dtype code, ssm_rounding reference or None) of a state pool.
    rounding: None (nearest even) or (seed, offset[, philox_rounds=10])."""
    if pool.dtype == torch.float32:
        return SSM_F32, None
    if pool.dtype != torch.float16:
        raise TypeError(f"state pool must be float32 or float16, got {pool.dtype}")
    if rounding is None:
        return SSM_F16, None
    seed, offset = int(rounding[0]), int(rounding[1])
    rounds = int(rounding[2]) if len(rounding) > 2 else 10
    return SSM_F16, ctypes.byref(Rounding(seed, offset, rounds))


class SSMError(RuntimeError):
    """A libssm entry point returned a nonzero status."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.ssm_status_string(status).decode()}")


def _check(status: int, where: str) -> None:
    if status != 0:
        raise SSMError(status, where)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return SSM_BF16
    if t == torch.float32:
        return SSM_F32
    raise TypeError(f"unsupported dtype {t}; use torch.bfloat16 or torch.float32")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def ssd_chunk_scan(x, dt, A, B, C, D=None, initial_state=None, cu_seqlens=None,
                   chunk_size: int = 128, y=None, final_state=None, y_dtype=None,
                   return_final_state: bool = True, status=None, stream=None, workspace="auto"):
    """Chunked SSD prefill scan.

    x  : [nseq, L, H, P] (fixed length) or [T, H, P] with ``cu_seqlens``
    dt : [nseq, L, H] or [T, H], fp32
    A  : [H] fp32;  D : [H] fp32 or None
    B, C : [nseq, L, G, N] or [T, G, N], same dtype as x
    initial_state : [nseq, H, P, N] fp32 or None (zeros); may be ``final_state``
    cu_seqlens : int32 [nseq+1] CUDA tensor of packed offsets, or None
    y / final_state : optional preallocated outputs
    workspace : CUDA tensor of at least ssd_chunk_scan_workspace_size(...) bytes (a
        fixed-length batch then runs the balanced schedule), None for none, or
        "auto" (the default): one is allocated through torch when these shapes
        can use it
    Returns (y, final_state) -- final_state is None if not requested.
    """
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens", torch.int32)
        T, H, P = x.shape
        nseq = cu_seqlens.shape[0] - 1
        seqlen = T
    else:
        nseq, L, H, P = x.shape
        T, seqlen = nseq * L, L
    G, N = B.shape[-2], B.shape[-1]
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(B, "B", x.dtype)
    _dev(C, "C", x.dtype)
    _dev(D, "D", torch.float32)
    _dev(initial_state, "initial_state", torch.float32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.empty(x.shape, dtype=y_dtype, device=x.device)
    _dev(y, "y", y_dtype)
    if final_state is None and return_final_state:
        final_state = torch.empty((nseq, H, P, N), dtype=torch.float32, device=x.device)
    _dev(final_state, "final_state", torch.float32)
    _dev(status, "status", torch.int32)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be a CUDA tensor, None or "auto"')
        n = 0 if cu_seqlens is not None else ssd_chunk_scan_workspace_size(
            nseq, seqlen, H, P, N, G, chunk_size)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    _dev(workspace, "workspace")
    st = lib.ssd_chunk_scan(nseq, seqlen, _ptr(cu_seqlens), H, P, N, G, int(chunk_size),
                            in_code, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                            _ptr(D), _ptr(initial_state), _dtype_code(y.dtype), _ptr(y),
                            _ptr(final_state), _ptr(workspace),
                            0 if workspace is None else workspace.numel() * workspace.element_size(),
                            _ptr(status), _stream(stream))
    _check(st, "ssd_chunk_scan")
    return y, final_state


def ssd_chunk_scan_noalloc(x, dt, A, B, C, y, final_state=None, D=None, initial_state=None,
                           cu_seqlens=None, chunk_size: int = 128, status=None, stream=None):
    """ssd_chunk_scan with its workspace taken from the library's built-in
    scratch; nothing here allocates, so y (and final_state, if wanted) must be
    given.  Layouts as for ssd_chunk_scan.  For callers that must not allocate
    device memory (a pool owned by another framework, or no allocator at
    hand).  The first call on a device looks up the scratch's address; calls
    whose launches overlap on the GPU race on the one scratch per device."""
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens", torch.int32)
        T, H, P = x.shape
        nseq = cu_seqlens.shape[0] - 1
        seqlen = T
    else:
        nseq, seqlen, H, P = x.shape
    G, N = B.shape[-2], B.shape[-1]
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(B, "B", x.dtype)
    _dev(C, "C", x.dtype)
    _dev(D, "D", torch.float32)
    _dev(initial_state, "initial_state", torch.float32)
    if y is None:
        raise ValueError("ssd_chunk_scan_noalloc: y must be preallocated")
    _dev(y, "y", y.dtype)
    _dev(final_state, "final_state", torch.float32)
    _dev(status, "status", torch.int32)
    st = lib.ssd_chunk_scan_noalloc(nseq, seqlen, _ptr(cu_seqlens), H, P, N, G, int(chunk_size),
                                    in_code, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                    _ptr(D), _ptr(initial_state), _dtype_code(y.dtype), _ptr(y),
                                    _ptr(final_state), _ptr(status), _stream(stream))
    _check(st, "ssd_chunk_scan_noalloc")
    return y, final_state


def ssd_chunk_scan_workspace_size(nseq, seqlen, nheads, head_dim, d_state, ngroups,
                                  chunk_size=128) -> int:
    """Bytes of optional workspace ssd_chunk_scan can use for these shapes on the
    current device (the balanced schedule of fixed-length batches); 0 if none."""
    return int(lib.ssd_chunk_scan_workspace_size(nseq, seqlen, nheads, head_dim, d_state,
                                                 ngroups, chunk_size))


def ssm_state_update(state, x, dt, A, B, C, D=None, y=None, y_dtype=None, stream=None):
    """One-token decode update, in place on ``state`` [batch, H, P, N] fp32.

    x : [batch, H, P];  dt : [batch, H] fp32;  A, D : [H] fp32;
    B, C : [batch, G, N] (same dtype as x).  Returns y [batch, H, P].
    """
    _dev(state, "state", torch.float32)
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    batch, H, P, N = state.shape
    G = B.shape[-2]
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(B, "B", x.dtype)
    _dev(C, "C", x.dtype)
    _dev(D, "D", torch.float32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.empty((batch, H, P), dtype=y_dtype, device=state.device)
    _dev(y, "y", y_dtype)
    st = lib.ssm_state_update(batch, H, P, N, G, in_code, _ptr(state), _ptr(x), _ptr(dt),
                              _ptr(A), _ptr(B), _ptr(C), _ptr(D), _dtype_code(y.dtype),
                              _ptr(y), _stream(stream))
    _check(st, "ssm_state_update")
    return y


def ssd_chunk_scan_slots(x, dt, A, B, C, D, state_pool, slot_idx, has_initial_state=None,
                         cu_seqlens=None, chunk_size: int = 128, y=None, y_dtype=None,
                         status=None, stream=None, dt_bias=None, dt_softplus=False,
                         dt_limit=None, rounding=None):
    """Chunked SSD prefill whose states live in a pool, updated in place.

    state_pool : [max_slots, H, P, N] fp32; sequence s starts from
        state_pool[slot_idx[s]] (or zero where has_initial_state[s] == 0) and
        its final state is written back to the same row.
    slot_idx, has_initial_state : int32 CUDA tensors [nseq] (slot_idx None:
        sequence s uses row s).
    dt_bias [H] fp32, dt_softplus, dt_limit (lo, hi): transform the raw dt
        inside the kernel (dt <- clamp(softplus(dt + dt_bias))).
    state_pool may be float16; rounding = (seed, offset[, philox_rounds])
        then rounds the written states stochastically (None: nearest even).
    Other arguments as for ssd_chunk_scan.  Returns y.
    """
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens", torch.int32)
        T, H, P = x.shape
        nseq = cu_seqlens.shape[0] - 1
        seqlen = T
    else:
        nseq, L, H, P = x.shape
        seqlen = L
    G, N = B.shape[-2], B.shape[-1]
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(B, "B", x.dtype)
    _dev(C, "C", x.dtype)
    _dev(D, "D", torch.float32)
    _dev(state_pool, "state_pool")
    sd, rnd = _state_format(state_pool, rounding)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(has_initial_state, "has_initial_state", torch.int32)
    _dev(status, "status", torch.int32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.empty(x.shape, dtype=y_dtype, device=x.device)
    _dev(y, "y", y_dtype)
    dtp = _dt_params(dt_bias, dt_softplus, dt_limit)
    st = lib.ssd_chunk_scan_slots(nseq, seqlen, _ptr(cu_seqlens), H, P, N, G, int(chunk_size),
                                  in_code, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                  dtp, _ptr(state_pool), sd, rnd, state_pool.shape[0], _ptr(slot_idx),
                                  _ptr(has_initial_state), _dtype_code(y.dtype), _ptr(y),
                                  _ptr(status), _stream(stream))
    _check(st, "ssd_chunk_scan_slots")
    return y


def ssm_state_update_slots(state_pool, slot_idx, x, dt, A, B, C, D=None, y=None, y_dtype=None,
                           status=None, stream=None, dt_bias=None, dt_softplus=False,
                           dt_limit=None, rounding=None):
    """One-token decode update of pool rows: batch row b updates
    state_pool[slot_idx[b]] in place (slot_idx[b] < 0: padding row, skipped;
    slot_idx None: row b).  state_pool may be float16, with rounding =
    (seed, offset[, philox_rounds]) for stochastic rounding (None: nearest).
    Returns y [batch, H, P] (padding rows left as they were)."""
    _dev(state_pool, "state_pool")
    sd, rnd = _state_format(state_pool, rounding)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    batch, H, P = x.shape
    N = state_pool.shape[-1]
    G = B.shape[-2]
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(B, "B", x.dtype)
    _dev(C, "C", x.dtype)
    _dev(D, "D", torch.float32)
    _dev(status, "status", torch.int32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.zeros((batch, H, P), dtype=y_dtype, device=x.device)
    _dev(y, "y", y_dtype)
    dtp = _dt_params(dt_bias, dt_softplus, dt_limit)
    st = lib.ssm_state_update_slots(batch, H, P, N, G, in_code, _ptr(state_pool), sd, rnd,
                                    state_pool.shape[0], _ptr(slot_idx), _ptr(x), _ptr(dt),
                                    _ptr(A), _ptr(B), _ptr(C), _ptr(D), dtp, _dtype_code(y.dtype),
                                    _ptr(y), _ptr(status), _stream(stream))
    _check(st, "ssm_state_update_slots")
    return y


def _activation(activation) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(map(str, ACTIVATIONS))}")
    return ACTIVATIONS[activation]


def causal_conv1d_fwd(x, weight, bias=None, conv_state=None, cu_seqlens=None,
                      activation="silu", slot_idx=None, has_initial_state=None, y=None,
                      y_dtype=None, status=None, stream=None):
    """Causal depthwise conv1d over whole sequences (prefill), channels-last.

    x : [nseq, L, dim] or, with cu_seqlens (int32 [nseq+1]), packed [T, dim];
        bf16 or fp32.
    weight : [dim, width] fp32 (width <= 8); bias : [dim] fp32 or None.
    conv_state : [rows, dim, width-1] in x's dtype, or None; read as the
        history before each sequence and overwritten with its last width-1
        inputs.  rows = nseq, or the pool size when slot_idx is given.
    slot_idx, has_initial_state : int32 [nseq] or None.
    Returns y shaped like x.
    """
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens", torch.int32)
        T, dim = x.shape
        nseq, seqlen = cu_seqlens.shape[0] - 1, T
    else:
        nseq, seqlen, dim = x.shape
    _dev(weight, "weight", torch.float32)
    width = weight.shape[-1]
    _dev(bias, "bias", torch.float32)
    _dev(conv_state, "conv_state", x.dtype)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(has_initial_state, "has_initial_state", torch.int32)
    _dev(status, "status", torch.int32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.empty(x.shape, dtype=y_dtype, device=x.device)
    _dev(y, "y", y_dtype)
    max_slots = conv_state.shape[0] if (conv_state is not None and slot_idx is not None) else 0
    st = lib.causal_conv1d_fwd(nseq, seqlen, _ptr(cu_seqlens), dim, width, in_code, _ptr(x),
                               _ptr(weight), _ptr(bias), _activation(activation),
                               _ptr(conv_state), max_slots, _ptr(slot_idx),
                               _ptr(has_initial_state), _dtype_code(y.dtype), _ptr(y),
                               _ptr(status), _stream(stream))
    _check(st, "causal_conv1d_fwd")
    return y


def causal_conv1d_update(x, weight, bias, conv_state, activation="silu", slot_idx=None,
                         y=None, y_dtype=None, status=None, stream=None):
    """One decode token per batch row; conv_state [rows, dim, width-1] rolls in
    place (rows = batch, or the pool size when slot_idx is given; a negative
    slot marks a padding row).  x : [batch, dim].  Returns y [batch, dim]."""
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    batch, dim = x.shape
    _dev(weight, "weight", torch.float32)
    width = weight.shape[-1]
    _dev(bias, "bias", torch.float32)
    _dev(conv_state, "conv_state", x.dtype)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(status, "status", torch.int32)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if y is None:
        y = torch.zeros((batch, dim), dtype=y_dtype, device=x.device)
    _dev(y, "y", y_dtype)
    max_slots = conv_state.shape[0] if (conv_state is not None and slot_idx is not None) else 0
    st = lib.causal_conv1d_update(batch, dim, width, in_code, _ptr(x), _ptr(weight), _ptr(bias),
                                  _activation(activation), _ptr(conv_state), max_slots,
                                  _ptr(slot_idx), _dtype_code(y.dtype), _ptr(y), _ptr(status),
                                  _stream(stream))
    _check(st, "causal_conv1d_update")
    return y


def ssm_state_update_multi(state, x, dt, A, B, C, D=None, slot_idx=None, accept_len=None,
                           inter_states=None, y=None, y_dtype=None, want_y=True,
                           want_inter=False, status=None, stream=None, dt_bias=None,
                           dt_softplus=False, dt_limit=None):
    """Speculative decode: ntok draft tokens per batch row from the row's state.

    state : [rows, H, P, N] fp32 (rows = batch, or a pool with slot_idx);
    x : [batch, ntok, H, P]; dt : [batch, ntok, H]; B, C : [batch, ntok, G, N].
    accept_len : int32 [batch] or None -- rewrite each row with its state after
    accept_len[b] tokens (None: the state is only read).
    Returns (y or None, inter_states or None); inter_states [batch, ntok, H, P,
    N] fp32 holds the state after each draft token when want_inter is set.
    """
    _dev(state, "state", torch.float32)
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    batch, ntok, H, P = x.shape
    N = state.shape[-1]
    G = B.shape[-2]
    for t, n, d in ((dt, "dt", torch.float32), (A, "A", torch.float32), (B, "B", x.dtype),
                    (C, "C", x.dtype), (D, "D", torch.float32), (slot_idx, "slot_idx", torch.int32),
                    (accept_len, "accept_len", torch.int32), (status, "status", torch.int32)):
        _dev(t, n, d)
    if want_inter and inter_states is None:
        inter_states = torch.empty((batch, ntok, H, P, N), dtype=torch.float32, device=x.device)
    _dev(inter_states, "inter_states", torch.float32)
    if want_y and y is None:
        y = torch.empty((batch, ntok, H, P), dtype=y_dtype or x.dtype, device=x.device)
    if y is not None:
        _dev(y, "y")
    y_code = _dtype_code(y.dtype) if y is not None else in_code
    max_slots = state.shape[0] if slot_idx is not None else 0
    st = lib.ssm_state_update_multi(batch, ntok, H, P, N, G, in_code, _ptr(state), max_slots,
                                    _ptr(slot_idx), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                    _ptr(D), _dt_params(dt_bias, dt_softplus, dt_limit),
                                    _ptr(accept_len), _ptr(inter_states), y_code,
                                    _ptr(y), _ptr(status), _stream(stream))
    _check(st, "ssm_state_update_multi")
    return y, inter_states


def ssm_state_commit(inter_states, accept_len, state, slot_idx=None, status=None, stream=None):
    """state row of b <- inter_states[b, accept_len[b] - 1] (unchanged where 0)."""
    _dev(inter_states, "inter_states", torch.float32)
    _dev(accept_len, "accept_len", torch.int32)
    _dev(state, "state", torch.float32)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(status, "status", torch.int32)
    batch, ntok, H, P, N = inter_states.shape
    max_slots = state.shape[0] if slot_idx is not None else 0
    st = lib.ssm_state_commit(batch, ntok, H, P, N, _ptr(inter_states), _ptr(accept_len),
                              _ptr(state), max_slots, _ptr(slot_idx), _ptr(status),
                              _stream(stream))
    _check(st, "ssm_state_commit")


def causal_conv1d_update_multi(x, weight, bias, conv_state, activation="silu", slot_idx=None,
                               accept_len=None, y=None, y_dtype=None, want_y=True,
                               status=None, stream=None):
    """ntok draft tokens per batch row through the causal conv1d.  x : [batch,
    ntok, dim]; conv_state [rows, dim, width-1] is rewritten with the window
    after accept_len[b] tokens (None: only read).  Returns y or None."""
    _dev(x, "x")
    in_code = _dtype_code(x.dtype)
    batch, ntok, dim = x.shape
    _dev(weight, "weight", torch.float32)
    width = weight.shape[-1]
    _dev(bias, "bias", torch.float32)
    _dev(conv_state, "conv_state", x.dtype)
    _dev(slot_idx, "slot_idx", torch.int32)
    _dev(accept_len, "accept_len", torch.int32)
    _dev(status, "status", torch.int32)
    if want_y and y is None:
        y = torch.empty((batch, ntok, dim), dtype=y_dtype or x.dtype, device=x.device)
    if y is not None:
        _dev(y, "y")
    y_code = _dtype_code(y.dtype) if y is not None else in_code
    max_slots = conv_state.shape[0] if (conv_state is not None and slot_idx is not None) else 0
    st = lib.causal_conv1d_update_multi(batch, ntok, dim, width, in_code, _ptr(x), _ptr(weight),
                                        _ptr(bias), _activation(activation), _ptr(conv_state),
                                        max_slots, _ptr(slot_idx), _ptr(accept_len), y_code,
                                        _ptr(y), _ptr(status), _stream(stream))
    _check(st, "causal_conv1d_update_multi")
    return y


def ssm_gated_rmsnorm(y, z, weight, group_size: int, eps: float = 1e-5, out=None,
                      out_dtype=None, stream=None):
    """out = (y * silu(z)) / rms over groups of group_size channels * weight.
    y, z : [rows, dim] (or any shape whose last axis is dim); weight [dim] fp32.
    out may be y itself.  Returns out."""
    _dev(y, "y")
    _dev(z, "z")
    _dev(weight, "weight", torch.float32)
    dim = y.shape[-1]
    rows = y.numel() // dim if dim else 0
    if out is None:
        out = torch.empty(y.shape, dtype=out_dtype or y.dtype, device=y.device)
    _dev(out, "out")
    st = lib.ssm_gated_rmsnorm(rows, dim, int(group_size), _dtype_code(y.dtype), _ptr(y),
                               _dtype_code(z.dtype), _ptr(z), _ptr(weight), float(eps),
                               _dtype_code(out.dtype), _ptr(out), _stream(stream))
    _check(st, "ssm_gated_rmsnorm")
    return out


# ---------------------------------------------------------------------------
# Per-channel selective scan, its gradient and decode update, the conv1d
# gradient, and the rows of state pools.
#
# Each call first goes to its function of the _marshal module, which does the
# same checks and allocations in C++ for a call that is plainly right (tensors
# of the current device, default stream and workspace).  It answers None for
# anything else (and where it is missing, _NoMarshal); the Python below then
# names what is wrong, or takes the options that _marshal does not.
# ---------------------------------------------------------------------------
def _plain(answer, where):
    """Whether _marshal made the call (its results are `answer`); raises on a library error."""
    if answer.__class__ is int:
        raise SSMError(answer, where)
    return answer is not None


@contextlib.contextmanager
def _enter(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_NO_SCOPE = contextlib.nullcontext()
_F32, _I32 = torch.float32, torch.int32


def _scope(t, stream):
    """The device of t and the given stream made current, so that what a call
    allocates belongs to the stream that uses it."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    if stream is None and dev == torch.cuda.current_device():
        return _NO_SCOPE
    return _enter(t.device, stream)


def _raw_stream(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _dev_like(t, name, dev, dtype=None, shape=None):
    """None, or t's address: a contiguous tensor on device dev, of the given type and shape."""
    if t is None:
        return None
    if t.get_device() == dev and t.is_contiguous() and (dtype is None or t.dtype is dtype) \
            and (shape is None or t.shape == shape):
        return t.data_ptr()
    _dev(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _count(n, name):
    """n as the ABI takes it (ctypes would drop the bits above an int's)."""
    if n > 0x7fffffff:
        raise ValueError(f"{name} is {n}: at most 2^31 - 1 are supported")
    return n


def _token_rows(t, name, lead, row, dev, dtype):
    """Elements between the tokens of an activation of shape lead + row (lead:
    (T,), or (nseq, L)), whose rows are contiguous and equally spaced."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if shape != lead + row:
        raise ValueError(f"{name} must have shape {lead + row}, got {tuple(shape)}")
    k = len(lead)
    width = row[0] if len(row) == 1 else row[0] * row[1]
    if 0 in lead:
        return width
    if (row[-1] > 1 and strides[-1] != 1) or (len(row) == 2 and row[0] > 1 and strides[k] != row[1]):
        raise ValueError(f"the rows of {name} must be contiguous")
    if k == 1:
        return strides[0] if shape[0] > 1 else width
    n, length = lead
    token = strides[1] if length > 1 else (strides[0] if n > 1 else width)
    if n > 1 and length > 1 and strides[0] != length * token:
        raise ValueError(f"the tokens of {name} must be equally spaced")
    return token


def _scan_lead(x, cu_seqlens, dev):
    """(leading axes, nseq, seqlen, tokens, dim) of an x [nseq, L, dim] or packed [T, dim]."""
    if cu_seqlens is not None:
        _dev_like(cu_seqlens, "cu_seqlens", dev, _I32)
        if x.dim() != 2 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("packed x must be [T, dim] with cu_seqlens [nseq+1]")
        T, dim = _count(x.shape[0], "the number of tokens"), _count(x.shape[1], "dim")
        return (T,), _count(cu_seqlens.shape[0] - 1, "the number of sequences"), T, T, dim
    if x.dim() != 3:
        raise ValueError("x must be [nseq, L, dim], or [T, dim] with cu_seqlens")
    n, length, dim = x.shape
    for v, name in ((n, "the number of sequences"), (length, "the sequence length"), (dim, "dim")):
        _count(v, name)
    return (n, length), n, length, n * length, dim


def _scan_operands(lead, dim, dev, x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit):
    """Checks the operands of a per-channel scan.  (d_state, groups, and the
    arguments in_dtype .. dt_params of the call, around dy where it takes one)."""
    dtype = x.dtype
    in_code, dt_code = _dtype_code(dtype), _dtype_code(dt.dtype)
    if A.dim() != 2 or B.dim() != len(lead) + 2:
        raise ValueError("A must be [dim, d_state], B and C the tokens' [ngroups, d_state]")
    N, G = _count(A.shape[1], "d_state"), _count(B.shape[-2], "ngroups")
    row, bc = (dim,), (G, N)
    a = _dev_like(A, "A", dev, _F32, (dim, N))
    d = _dev_like(D, "D", dev, _F32, row)
    params = None
    if dt_bias is not None or dt_softplus or dt_limit is not None:
        bias = _dev_like(dt_bias, "dt_bias", dev, _F32, row)
        lo, hi = (0.0, 0.0) if dt_limit is None else dt_limit
        params = ctypes.byref(DtParams(bias, bool(dt_softplus), dt_limit is not None, lo, hi))
    xs = _token_rows(x, "x", lead, row, dev, dtype)
    dts = _token_rows(dt, "dt", lead, row, dev, dt.dtype)
    Bs = _token_rows(B, "B", lead, bc, dev, dtype)
    Cs = _token_rows(C, "C", lead, bc, dev, dtype)
    zs = 0 if z is None else _token_rows(z, "z", lead, row, dev, dtype)
    return N, G, in_code, (x.data_ptr(), xs, dt_code, dt.data_ptr(), dts, a, B.data_ptr(), Bs, C.data_ptr(), Cs,
                           d, _addr(z), zs, params)


def _workspace(workspace, size, like, dev):
    """(tensor to keep, address, bytes) of a workspace: "auto" allocates `size` bytes."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be a CUDA tensor, None or "auto"')
        if not size:
            return None, None, 0
        workspace = like.new_empty(size, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), size
    if workspace is None:
        return None, None, 0
    return workspace, _dev_like(workspace, "workspace", dev), workspace.numel() * workspace.element_size()


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, initial_state=None, cu_seqlens=None,
                       final_state=None, slot_idx=None, has_initial_state=None, dt_bias=None,
                       dt_softplus=False, dt_limit=None, y=None, y_dtype=None,
                       return_final_state: bool = True, save_states: bool = False, status=None,
                       stream=None, workspace="auto"):
    """Per-channel selective scan over whole sequences.

    x, dt, z : [nseq, L, dim] or, with cu_seqlens (int32 [nseq+1]), packed
        [T, dim]; x and z bf16 or fp32, dt x's type or fp32; z (the gate) may
        be None.  Views whose rows are contiguous are taken as they are.
    A : [dim, d_state] fp32;  D, dt_bias : [dim] fp32 or None
    B, C : [nseq, L, G, d_state] or [T, G, d_state], x's dtype
    dt_bias, dt_softplus, dt_limit (lo, hi): dt <- clamp(softplus(dt + dt_bias))
    initial_state, final_state : [nseq, dim, d_state] fp32, or with slot_idx
        (int32 [nseq]) a pool [max_slots, dim, d_state]; they may be the same
        tensor.  has_initial_state : int32 [nseq], 0 starts from zero.
    save_states : also return what selective_scan_bwd needs of this call.
    workspace : as for ssd_chunk_scan; lets a long sequence on few channels
        run in concurrent ranges.
    Returns (y, final_state), or (y, final_state, saved) with save_states.
    """
    if stream is None and isinstance(workspace, str) and workspace == "auto" and y_dtype is None:
        out = _marshal.scan_fwd(x, cu_seqlens, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit, initial_state,
                                final_state, slot_idx, has_initial_state, y, return_final_state, save_states, status)
        if _plain(out, "selective_scan_fwd"):
            return out if save_states else out[:2]
    with _scope(x, stream):
        dev = x.get_device()
        lead, nseq, seqlen, T, dim = _scan_lead(x, cu_seqlens, dev)
        N, G, in_code, operands = _scan_operands(lead, dim, dev, x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
        rows = nseq
        if slot_idx is not None:
            states = final_state if final_state is not None else initial_state
            if states is None:
                raise ValueError("slot_idx needs a state pool")
            rows = _count(states.shape[0], "max_slots")
        elif final_state is None and return_final_state:
            final_state = x.new_empty((nseq, dim, N), dtype=_F32)
        if y is None:
            y = x.new_empty(x.shape, dtype=y_dtype or x.dtype)
        saved = x.new_empty(lib.selective_scan_saved_size(nseq, T, dim, N) // 4, dtype=_F32) if save_states else None
        size = lib.selective_scan_workspace_size(nseq, T, dim, N, G) if isinstance(workspace, str) else 0
        ws, ws_ptr, ws_bytes = _workspace(workspace, size, x, dev)
        st = lib.selective_scan_fwd(
            nseq, seqlen, _addr(cu_seqlens), dim, N, G, in_code, *operands,
            _dev_like(initial_state, "initial_state", dev, _F32, (rows, dim, N)),
            _dev_like(final_state, "final_state", dev, _F32, (rows, dim, N)), rows,
            _dev_like(slot_idx, "slot_idx", dev, _I32, (nseq,)),
            _dev_like(has_initial_state, "has_initial_state", dev, _I32, (nseq,)),
            _dtype_code(y.dtype), _dev_like(y, "y", dev, y_dtype, x.shape), _addr(saved), ws_ptr, ws_bytes,
            _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "selective_scan_fwd")
    return (y, final_state, saved) if save_states else (y, final_state)


def selective_scan_saved_size(nseq, ntokens, dim, d_state) -> int:
    """Bytes that selective_scan_fwd(save_states=True) keeps for the backward pass."""
    return int(lib.selective_scan_saved_size(nseq, ntokens, dim, d_state))


def selective_scan_workspace_size(nseq, ntokens, dim, d_state, ngroups=1) -> int:
    """Bytes of optional workspace selective_scan_fwd can use for these sizes; 0 if none."""
    return int(lib.selective_scan_workspace_size(nseq, ntokens, dim, d_state, ngroups))


class SelectiveScanGrads(NamedTuple):
    """Gradients of selective_scan_fwd; None where the input was not given (or,
    dinitial_state, not asked for)."""
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: torch.Tensor | None
    dz: torch.Tensor | None
    ddt_bias: torch.Tensor | None
    dinitial_state: torch.Tensor | None


def selective_scan_bwd(dy, x, dt, A, B, C, saved, D=None, z=None, dfinal_state=None, cu_seqlens=None,
                       dt_bias=None, dt_softplus=False, dt_limit=None, want_dinitial: bool = False,
                       status=None, stream=None, workspace="auto") -> SelectiveScanGrads:
    """Gradient of selective_scan_fwd called with the same inputs and
    save_states=True (`saved` is its third result).  dy : like x.
    dfinal_state : [nseq, dim, d_state] fp32 or None.  The gradients have their
    inputs' shapes and types (contiguous).  The workspace grows with the square
    of d_state (2 GiB for 8192 tokens of 8192 channels at 64 states, 8 at 128):
    selective_scan_bwd_workspace_size says how large it is."""
    if stream is None and isinstance(workspace, str) and workspace == "auto":
        out = _marshal.scan_bwd(x, cu_seqlens, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit, dy, saved,
                                dfinal_state, want_dinitial, status)
        if _plain(out, "selective_scan_bwd"):
            return SelectiveScanGrads(*out)
    with _scope(x, stream):
        dev = x.get_device()
        lead, nseq, seqlen, T, dim = _scan_lead(x, cu_seqlens, dev)
        N, G, in_code, operands = _scan_operands(lead, dim, dev, x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
        dys = _token_rows(dy, "dy", lead, (dim,), dev, x.dtype)
        if saved.numel() * 4 != lib.selective_scan_saved_size(nseq, T, dim, N):
            raise ValueError("saved is not that of a forward call of these sizes")

        # a batch of no sequences launches nothing: its sums are zero
        new = x.new_zeros if nseq == 0 else x.new_empty
        g = SelectiveScanGrads(
            new(x.shape), new(dt.shape, dtype=dt.dtype), new((dim, N), dtype=_F32), new(B.shape), new(C.shape),
            None if D is None else new((dim,), dtype=_F32), None if z is None else new(z.shape),
            None if dt_bias is None else new((dim,), dtype=_F32),
            new((nseq, dim, N), dtype=_F32) if want_dinitial else None)
        size = lib.selective_scan_bwd_workspace_size(nseq, T, dim, N, G) if isinstance(workspace, str) else 0
        ws, ws_ptr, ws_bytes = _workspace(workspace, size, x, dev)
        st = lib.selective_scan_bwd(
            nseq, seqlen, _addr(cu_seqlens), dim, N, G, in_code, dy.data_ptr(), dys, *operands,
            _dev_like(saved, "saved", dev, _F32),
            _dev_like(dfinal_state, "dfinal_state", dev, _F32, (nseq, dim, N)),
            *[_addr(t) for t in (g.dx, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias, g.dinitial_state)],
            ws_ptr, ws_bytes, _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "selective_scan_bwd")
    return g


def selective_scan_bwd_workspace_size(nseq, ntokens, dim, d_state, ngroups=1) -> int:
    """Bytes of workspace selective_scan_bwd needs for these sizes."""
    return int(lib.selective_scan_bwd_workspace_size(nseq, ntokens, dim, d_state, ngroups))


def selective_state_update(state, x, dt, A, B, C, D=None, z=None, slot_idx=None, dt_bias=None,
                           dt_softplus=False, dt_limit=None, y=None, y_dtype=None, status=None,
                           stream=None):
    """One token per batch row of the per-channel selective scan, in place on
    ``state`` [batch, dim, d_state] fp32, or on rows slot_idx (int32 [batch],
    negative: padding row) of a pool [max_slots, dim, d_state].

    x, dt, z : [batch, dim];  B, C : [batch, G, d_state];  A, D, dt_bias and the
    dt transform as for selective_scan_fwd.  Returns y [batch, dim] (padding
    rows left as they were)."""
    if stream is None and y_dtype is None:
        out = _marshal.state_update(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit, state, slot_idx, y, status)
        if _plain(out, "selective_state_update"):
            return out[0]
    with _scope(x, stream):
        if x.dim() != 2:
            raise ValueError("x must be [batch, dim]")
        dev = x.get_device()
        batch, dim = _count(x.shape[0], "batch"), _count(x.shape[1], "dim")
        N, G, in_code, operands = _scan_operands((batch,), dim, dev, x, dt, A, B, C, D, z, dt_bias, dt_softplus,
                                                 dt_limit)
        rows = batch if slot_idx is None else _count(state.shape[0], "max_slots")
        if y is None:
            y = x.new_zeros((batch, dim), dtype=y_dtype or x.dtype)
        st = lib.selective_state_update(
            batch, dim, N, G, _dev_like(state, "state", dev, _F32, (rows, dim, N)), rows,
            _dev_like(slot_idx, "slot_idx", dev, _I32, (batch,)), in_code, *operands, _dtype_code(y.dtype),
            _dev_like(y, "y", dev, y_dtype, (batch, dim)), _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "selective_state_update")
    return y


def causal_conv1d_bwd(dy, x, weight, bias=None, initial_state=None, dfinal_state=None, cu_seqlens=None,
                      activation="silu", status=None, stream=None, workspace="auto"):
    """Gradient of causal_conv1d_fwd.  dy, x : [nseq, L, dim] or packed [T, dim]
    (bf16 or fp32); weight [dim, width], bias [dim] fp32.  initial_state : the
    conv states before the forward call [nseq, dim, width-1] (it overwrites
    its conv_state), or None; dfinal_state : gradient of the states it left, or
    None.  Returns (dx, dweight, dbias, dinitial_state); dbias is None without
    bias, dinitial_state None without initial_state."""
    if stream is None and isinstance(workspace, str) and workspace == "auto":
        out = _marshal.conv1d_bwd(x, cu_seqlens, dy, weight, bias, initial_state, dfinal_state,
                                  _activation(activation), status)
        if _plain(out, "causal_conv1d_bwd"):
            return out
    with _scope(x, stream):
        dev = x.get_device()
        in_code = _dtype_code(x.dtype)
        _, nseq, seqlen, T, dim = _scan_lead(x, cu_seqlens, dev)
        if weight.dim() != 2:
            raise ValueError("weight must be [dim, width]")
        width = _count(weight.shape[1], "width")
        dx, dweight = x.new_empty(x.shape), weight.new_empty((dim, width))
        dbias = None if bias is None else weight.new_empty((dim,))
        line = (nseq, dim, width - 1)
        dinitial = None if initial_state is None else x.new_empty(line)
        size = lib.causal_conv1d_bwd_workspace_size(T, dim, width) if isinstance(workspace, str) else 0
        ws, ws_ptr, ws_bytes = _workspace(workspace, size, x, dev)
        st = lib.causal_conv1d_bwd(
            nseq, seqlen, _addr(cu_seqlens), dim, width, in_code,
            _dev_like(dy, "dy", dev, x.dtype, x.shape), _dev_like(x, "x", dev),
            _dev_like(weight, "weight", dev, _F32, (dim, width)), _dev_like(bias, "bias", dev, _F32, (dim,)),
            _activation(activation), _dev_like(initial_state, "initial_state", dev, x.dtype, line),
            _dev_like(dfinal_state, "dfinal_state", dev, x.dtype, line), dx.data_ptr(), dweight.data_ptr(),
            _addr(dbias), _addr(dinitial), ws_ptr, ws_bytes, _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "causal_conv1d_bwd")
    return dx, dweight, dbias, dinitial


def _pools(pools):
    """(ssm_pool array, count, max_slots, a tensor of them) of tensors [max_slots, ...]
    whose rows are contiguous."""
    pools = (pools,) if isinstance(pools, torch.Tensor) else pools
    if not pools:
        raise ValueError("no pools given")
    first = pools[0]
    dev, slots = first.get_device(), _count(first.shape[0], "max_slots") if first.dim() else -1
    fields, shape, strides, size = [], None, None, 0
    for p in pools:
        # the pools of a stack's layers are mostly alike: a layout is looked at once
        if p.shape != shape or p.stride() != strides or p.element_size() != size:
            shape, strides, size = p.shape, p.stride(), p.element_size()
            if p.dim() < 1 or shape[0] != slots:
                raise ValueError("pools must be tensors [max_slots, ...] with the same number of slots")
            step = 1
            for n, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
                if n > 1 and stride != step:
                    raise ValueError("the rows of a pool must be contiguous")
                step *= n
            row, pitch = step * size, (strides[0] if slots > 1 else step) * size
        if p.get_device() != dev:
            raise ValueError("pools must be CUDA tensors on one device")
        fields += p.data_ptr(), row, pitch
    # ssm_pool is three 64-bit fields: base, row_bytes, row_stride
    return (ctypes.c_int64 * len(fields))(*fields), len(pools), slots, first


def ssm_pool_copy(pools, src_idx, dst_idx, status=None, stream=None) -> None:
    """Rows dst_idx[i] <- src_idx[i] of every pool, for i in order (a fork copies
    one row to several).  pools : one tensor or a list of tensors [max_slots,
    ...] with contiguous rows (any types); src_idx, dst_idx : int32 [n], an
    entry with a negative index is skipped."""
    if stream is None and _plain(_marshal.pool_copy(pools, src_idx, dst_idx, status), "ssm_pool_copy"):
        return
    arr, n, slots, like = _pools(pools)
    with _scope(like, stream):
        dev, pairs = like.get_device(), _count(src_idx.shape[0], "the number of pairs")
        st = lib.ssm_pool_copy(n, arr, slots, pairs, _dev_like(src_idx, "src_idx", dev, _I32, (pairs,)),
                               _dev_like(dst_idx, "dst_idx", dev, _I32, (pairs,)),
                               _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "ssm_pool_copy")


def ssm_pool_zero(pools, row_idx, status=None, stream=None) -> None:
    """Rows row_idx (int32 [n]; negative: skipped) of every pool <- 0."""
    if stream is None and _plain(_marshal.pool_zero(pools, row_idx, status), "ssm_pool_zero"):
        return
    arr, n, slots, like = _pools(pools)
    with _scope(like, stream):
        dev, rows = like.get_device(), _count(row_idx.shape[0], "the number of rows")
        st = lib.ssm_pool_zero(n, arr, slots, rows, _dev_like(row_idx, "row_idx", dev, _I32, (rows,)),
                               _dev_like(status, "status", dev, _I32), _raw_stream(dev))
    _check(st, "ssm_pool_zero")


def ssm_pool_compact(pools, slot_idx, status=None, stream=None, workspace="auto"):
    """Moves the live rows (those that slot_idx, int32 [nrows], names) to the
    front of every pool and rewrites slot_idx in place.  Returns their number,
    an int32 scalar tensor."""
    if stream is None and isinstance(workspace, str) and workspace == "auto":
        out = _marshal.pool_compact(pools, slot_idx, status)
        if _plain(out, "ssm_pool_compact"):
            return out[0]
    arr, n, slots, like = _pools(pools)
    with _scope(like, stream):
        dev, rows = like.get_device(), _count(slot_idx.shape[0], "the number of rows")
        live = slot_idx.new_empty(())
        size = lib.ssm_pool_compact_workspace_size(slots, rows) if isinstance(workspace, str) else 0
        ws, ws_ptr, ws_bytes = _workspace(workspace, size, like, dev)
        st = lib.ssm_pool_compact(n, arr, slots, rows, _dev_like(slot_idx, "slot_idx", dev, _I32, (rows,)),
                                  live.data_ptr(), ws_ptr, ws_bytes, _dev_like(status, "status", dev, _I32),
                                  _raw_stream(dev))
    _check(st, "ssm_pool_compact")
    return live


# ---------------------------------------------------------------------------
# Testing hooks (include/ssm_testing.h): the pipelined kernels with a stalled
# producer and a short wait limit, to exercise their timeout path.
# ---------------------------------------------------------------------------
def testing_scan_stalled(x, dt, A, B, C, y, status, wait_ns: int = 1_000_000, stream=None):
    """Tensor-core scan kernel whose producer issues nothing: every CTA's first
    bounded wait expires after ``wait_ns`` and the kernel writes
    SSM_ERR_TIMEOUT to ``status``.  x [nseq, L, H, 64] bf16, dt [nseq, L, H],
    B, C [nseq, L, G, 128] bf16, y like x (meaningless output)."""
    for t, n in ((x, "x"), (y, "y"), (B, "B"), (C, "C")):
        _dev(t, n, torch.bfloat16)
    _dev(dt, "dt", torch.float32)
    _dev(A, "A", torch.float32)
    _dev(status, "status", torch.int32)
    nseq, L, H, _ = x.shape
    G = B.shape[-2]
    st = lib.ssm_testing_scan_stalled(nseq, L, H, G, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                      _ptr(y), int(wait_ns), _ptr(status), _stream(stream))
    _check(st, "ssm_testing_scan_stalled")


def testing_conv1d_stalled(x, weight, y, status, wait_ns: int = 1_000_000, stream=None):
    """Bulk-copy ring conv1d kernel whose producer issues nothing (see
    testing_scan_stalled).  x, y [nseq, L, dim] bf16, weight [dim, width] fp32."""
    _dev(x, "x", torch.bfloat16)
    _dev(y, "y", torch.bfloat16)
    _dev(weight, "weight", torch.float32)
    _dev(status, "status", torch.int32)
    nseq, L, dim = x.shape
    st = lib.ssm_testing_conv1d_stalled(nseq, L, dim, weight.shape[1], _ptr(x), _ptr(weight),
                                        _ptr(y), int(wait_ns), _ptr(status), _stream(stream))
    _check(st, "ssm_testing_conv1d_stalled")
