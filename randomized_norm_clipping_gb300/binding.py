"""ctypes binding of libdprc (include/dprc.h): argument marshalling only.

Every function here takes torch tensors for device memory, passes their data
pointers and the current CUDA stream to the C ABI of the same name, and raises
``DprcError`` on a non-zero status.  All arithmetic runs in the library's
kernels; there is no fallback of any kind: if libdprc.so is missing, loading
raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# DPRC_LIBRARY=debug loads the bounds-checked build (libdprc_debug.so: every
# computed index checked before its access, failures recorded in the device
# error word as DPRC_DEVERR_BOUNDS); anything else, the release build.
LIB_PATH = os.path.join(
    PKG_DIR, "libdprc_debug.so" if os.environ.get("DPRC_LIBRARY") == "debug" else "libdprc.so")

DPRC_F32, DPRC_BF16 = 0, 1
(DPRC_OP_HUTCH, DPRC_OP_HUTCHPP, DPRC_OP_EXACT, DPRC_OP_HUTCH_LAYERS, DPRC_OP_HUTCH_PM1,
 DPRC_OP_HUTCH_HOST) = (1, 2, 3, 4, 5, 6)
(DPRC_EXACT_AUTO, DPRC_EXACT_DIRECT, DPRC_EXACT_GHOST, DPRC_EXACT_GHOST_N128,
 DPRC_EXACT_GHOST_N256) = (0, 1, 2, 3, 4)
STATUS = {0: "ok", 1: "null pointer", 2: "shape", 3: "dtype", 4: "alignment",
          5: "workspace", 6: "cuda", 7: "non-finite", 8: "device", 9: "too large"}

# The C prototypes of include/dprc.h, as (name, restype, argtypes).
_c = ctypes
_PROTOS = [
    ("dprc_abi_version", _c.c_int, []),
    ("dprc_status_string", _c.c_char_p, [_c.c_int]),
    ("dprc_workspace_bytes", _c.c_size_t,
     [_c.c_int, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64]),
    ("dprc_norm_hutch", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_norm_hutchpp", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_exact_norm", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_clip_factors", _c.c_int,
     [_c.c_void_p, _c.c_int64, _c.c_float, _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    ("dprc_add_noise", _c.c_int,
     [_c.c_void_p, _c.c_int64, _c.c_float, _c.c_float, _c.c_uint64, _c.c_uint64, _c.c_void_p]),
    ("dprc_add_noise_at", _c.c_int,
     [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_uint64, _c.c_float, _c.c_float, _c.c_uint64,
      _c.c_uint64, _c.c_void_p]),
    ("dprc_philox_words", _c.c_int,
     [_c.c_void_p, _c.c_int64, _c.c_uint64, _c.c_uint64, _c.c_uint64, _c.c_void_p]),
    ("dprc_device_error", _c.c_int, [_c.c_void_p, _c.c_int]),
    ("dprc_set_phase_events", _c.c_int, [_c.c_void_p, _c.c_int]),
    ("dprc_norm_hutch_pm1", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_uint64, _c.c_uint64, _c.c_int, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_norm_hutch_layers", _c.c_int,
     [_c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int,
      _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_norm_hutch_layers_clip", _c.c_int,
     [_c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int,
      _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_float, _c.c_void_p,
      _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_norm_hutch_launches", _c.c_int,
     [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64]),
    ("dprc_norm_hutchpp_launches", _c.c_int,
     [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64]),
    ("dprc_exact_norm_form", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_int, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_exact_norm_plan", _c.c_int,
     [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int]),
    ("dprc_norm_hutch_clip_host", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_float, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_norm_hutch_clip", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_float, _c.c_void_p, _c.c_void_p,
      _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_norm_hutch_noalloc", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int, _c.c_void_p]),
    ("dprc_test_hutch_fault", _c.c_int,
     [_c.c_int, _c.c_uint64, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
      _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_embed_plan_bytes", _c.c_size_t, [_c.c_int64, _c.c_int64]),
    ("dprc_embed_workspace_bytes", _c.c_size_t, [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64]),
    ("dprc_embed_lookup", _c.c_int,
     [_c.c_void_p, _c.c_int, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_float, _c.c_void_p, _c.c_void_p]),
    ("dprc_embed_plan", _c.c_int,
     [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_embed_norm", _c.c_int,
     [_c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_float,
      _c.c_void_p, _c.c_size_t, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_embed_grad", _c.c_int,
     [_c.c_void_p, _c.c_int, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int64,
      _c.c_float, _c.c_void_p, _c.c_size_t, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t,
      _c.c_void_p]),
    ("dprc_dropout", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_uint64, _c.c_double, _c.c_uint64,
      _c.c_uint64, _c.c_void_p, _c.c_void_p]),
    ("dprc_linear_workspace_bytes", _c.c_size_t,
     [_c.c_int, _c.c_int64, _c.c_int64, _c.c_int64, _c.c_int]),
    ("dprc_linear", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int, _c.c_double, _c.c_uint64, _c.c_uint64, _c.c_void_p, _c.c_void_p,
      _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("dprc_linear_grad", _c.c_int,
     [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int64, _c.c_int64,
      _c.c_int64, _c.c_int, _c.c_double, _c.c_uint64, _c.c_uint64, _c.c_void_p, _c.c_void_p,
      _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
]
EXPORTED = tuple(name for name, _, _ in _PROTOS)

_lib = None
_lock = threading.Lock()


class DprcError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed with status {status} ({STATUS.get(status, '?')})")
        self.status = status


def lib():
    """The loaded libdprc (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with `python -c "
                        "\"import __graft_entry__ as g; g.build()\"`")
                h = ctypes.CDLL(LIB_PATH)
                for name, res, args in _PROTOS:
                    f = getattr(h, name)
                    f.restype = res
                    f.argtypes = args
                _lib = h
    return _lib


_CODES = {torch.float32: DPRC_F32, torch.bfloat16: DPRC_BF16}


def _dtype_code(t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t, stream):
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    if _raw_stream is not None:  # the current stream's handle without a Stream object
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _check(fn, status):
    if status != 0:
        raise DprcError(fn, status)


def _need_cuda(*ts):
    for t in ts:
        if t is None or (t.is_cuda and t.is_contiguous()):
            continue
        raise ValueError("libdprc takes device tensors" if not t.is_cuda
                         else "libdprc takes contiguous tensors")


def dprc_abi_version():
    return lib().dprc_abi_version()


def dprc_workspace_bytes(op, dtype_code, B, T, d, p, k):
    return int(lib().dprc_workspace_bytes(op, dtype_code, B, T, d, p, k))


def workspace(op, like, B, T, d, p, k):
    """A zeroed device byte buffer of dprc_workspace_bytes(...) bytes (torch
    allocation).  Workspaces must be zero before their first use; calls leave
    their counter block zero again, so the buffer can be reused."""
    n = dprc_workspace_bytes(op, _dtype_code(like), B, T, d, p, k)
    if n == 0:
        raise DprcError("dprc_workspace_bytes", 2)
    return torch.zeros(n, dtype=torch.uint8, device=like.device)


def dprc_norm_hutch_clip(A, G, P, n, C, c, accumulate=False, nonfinite=None, ws=None,
                         stream=None):
    """n[i] (+)= ||A_i^T (G_i P)||_F^2, then c[i] = min(1, C / sqrt(n[i]))
    (see include/dprc.h)."""
    _need_cuda(A, G, P, n, c, nonfinite)
    B, T, d = A.shape
    p, k = P.shape
    if ws is None:
        ws = workspace(DPRC_OP_HUTCH, A, B, T, d, p, k)
    st = lib().dprc_norm_hutch_clip(_ptr(A), _ptr(G), _ptr(P), _dtype_code(A), B, T, d, p, k,
                                    _ptr(n), int(bool(accumulate)), float(C), _ptr(c),
                                    _ptr(nonfinite) if nonfinite is not None else None,
                                    _ptr(ws), ws.numel(), _stream(A, stream))
    _check("dprc_norm_hutch_clip", st)
    return n, c


def host_stage(A, T, d, p, k, B=None, device=None):
    """A zeroed device stage buffer for dprc_norm_hutch_clip_host with the
    sizes of host tensor A ([B][T][d]) and P [p][k]."""
    B = A.shape[0] if B is None else B
    n = dprc_workspace_bytes(DPRC_OP_HUTCH_HOST, _dtype_code(A), B, T, d, p, k)
    if n == 0:
        raise DprcError("dprc_workspace_bytes", 2)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def dprc_norm_hutch_clip_host(A, G, P, C, n, c, stage=None, stream=None):
    """Host tensors A [B][T][d], G [B][T][p], P [p][k] (pinned for asynchronous
    copies) -> host float32 n, c [B]: n[i] = ||A_i^T (G_i P)||_F^2 and
    c[i] = min(1, C / sqrt(n[i])), copied back at the end of the work enqueued
    on the stream (see include/dprc.h); n may be None.  Synchronise the
    stream before reading n and c."""
    ts = [t for t in (A, G, P, n, c) if t is not None]
    for t in ts:
        if t.is_cuda:
            raise ValueError("dprc_norm_hutch_clip_host takes host tensors")
        if not t.is_contiguous():
            raise ValueError("host tensors must be contiguous")
    if (n is not None and n.dtype != torch.float32) or c.dtype != torch.float32:
        raise ValueError("n and c must be float32")
    B, T, d = A.shape
    p, k = P.shape
    if stage is None:
        stage = host_stage(A, T, d, p, k)
    st = lib().dprc_norm_hutch_clip_host(_ptr(A), _ptr(G), _ptr(P), _dtype_code(A), B, T, d, p, k,
                                         float(C), _ptr(n), _ptr(c), _ptr(stage), stage.numel(),
                                         _stream(stage, stream))
    _check("dprc_norm_hutch_clip_host", st)
    return n, c


def dprc_norm_hutch_pm1(A, G, k, seed, step, n, accumulate=False, ws=None, stream=None):
    """n[i] (+)= (1/k) ||A_i^T (G_i S)||_F^2 with the +-1 projection S of
    (seed, step) (see include/dprc.h)."""
    _need_cuda(A, G, n)
    B, T, d = A.shape
    p = G.shape[2]
    if ws is None:
        ws = workspace(DPRC_OP_HUTCH_PM1, A, B, T, d, p, k)
    st = lib().dprc_norm_hutch_pm1(_ptr(A), _ptr(G), int(seed) & (2**64 - 1),
                                   int(step) & (2**64 - 1), _dtype_code(A), B, T, d, p, k,
                                   _ptr(n), int(bool(accumulate)), _ptr(ws), ws.numel(),
                                   _stream(A, stream))
    _check("dprc_norm_hutch_pm1", st)
    return n


def dprc_norm_hutch_layers(As, Gs, Ps, n, accumulate=False, ws=None, stream=None, C=None,
                           c=None, nonfinite=None):
    """n[i] (+)= sum_l ||A_l,i^T (G_l,i P_l)||_F^2 over the layers (see
    include/dprc.h); with C and c also c[i] = min(1, C / sqrt(n[i])) of the sum
    (dprc_norm_hutch_layers_clip)."""
    if (C is None) != (c is None):
        raise ValueError("give both C and c, or neither")
    L = len(As)
    if not (L == len(Gs) == len(Ps)) or L == 0:
        raise ValueError("As, Gs and Ps must be non-empty lists of the same length")
    _need_cuda(*As, *Gs, *Ps, n)
    B, T = As[0].shape[0], As[0].shape[1]
    k = Ps[0].shape[1]
    d = (ctypes.c_int64 * L)(*[a.shape[2] for a in As])
    p = (ctypes.c_int64 * L)(*[g.shape[2] for g in Gs])
    ap = (ctypes.c_void_p * L)(*[_ptr(a) for a in As])
    gp = (ctypes.c_void_p * L)(*[_ptr(g) for g in Gs])
    pp = (ctypes.c_void_p * L)(*[_ptr(x) for x in Ps])
    if ws is None:
        ws = workspace(DPRC_OP_HUTCH_LAYERS, As[0], B, T, max(d), max(p), k)
    if C is None:
        st = lib().dprc_norm_hutch_layers(L, ap, gp, pp, d, p, _dtype_code(As[0]), B, T, k,
                                          _ptr(n), int(bool(accumulate)), _ptr(ws), ws.numel(),
                                          _stream(As[0], stream))
        _check("dprc_norm_hutch_layers", st)
        return n
    _need_cuda(c, nonfinite)
    st = lib().dprc_norm_hutch_layers_clip(L, ap, gp, pp, d, p, _dtype_code(As[0]), B, T, k,
                                           _ptr(n), int(bool(accumulate)), float(C), _ptr(c),
                                           _ptr(nonfinite) if nonfinite is not None else None,
                                           _ptr(ws), ws.numel(), _stream(As[0], stream))
    _check("dprc_norm_hutch_layers_clip", st)
    return n, c


def dprc_norm_hutch_launches(dtype_code, B, T, d, p, k):
    """Kernels one dprc_norm_hutch call with these sizes enqueues on the
    current device (1 fused, 2 sketch + projection, 3 CUDA cores; 0 invalid)."""
    return int(lib().dprc_norm_hutch_launches(dtype_code, B, T, d, p, k))


def dprc_norm_hutchpp_launches(dtype_code, B, T, d, p, r):
    """Kernels one dprc_norm_hutchpp call with these sizes enqueues on the
    current device (5 with passes 1 and 2 fused, 7 or 8 otherwise; 0 invalid)."""
    return int(lib().dprc_norm_hutchpp_launches(dtype_code, B, T, d, p, r))


def dprc_norm_hutch(A, G, P, n, accumulate=False, ws=None, stream=None):
    """n[i] (+)= ||A_i^T (G_i P)||_F^2 (see include/dprc.h)."""
    _need_cuda(A, G, P, n)
    B, T, d = A.shape
    p, k = P.shape
    if ws is None:
        ws = workspace(DPRC_OP_HUTCH, A, B, T, d, p, k)
    st = lib().dprc_norm_hutch(_ptr(A), _ptr(G), _ptr(P), _dtype_code(A), B, T, d, p, k,
                               _ptr(n), int(bool(accumulate)), _ptr(ws), ws.numel(),
                               _stream(A, stream))
    _check("dprc_norm_hutch", st)
    return n


def dprc_norm_hutchpp(A, G, S, P, n, accumulate=False, ws=None, stream=None):
    """n[i] (+)= Hutch++ head + tail / r (see include/dprc.h)."""
    _need_cuda(A, G, S, P, n)
    B, T, d = A.shape
    p, r = P.shape
    if ws is None:
        ws = workspace(DPRC_OP_HUTCHPP, A, B, T, d, p, r)
    st = lib().dprc_norm_hutchpp(_ptr(A), _ptr(G), _ptr(S), _ptr(P), _dtype_code(A), B, T, d, p,
                                 r, _ptr(n), int(bool(accumulate)), _ptr(ws), ws.numel(),
                                 _stream(A, stream))
    _check("dprc_norm_hutchpp", st)
    return n


def dprc_norm_hutch_noalloc(A, G, P, n, accumulate=False, stream=None):
    """dprc_norm_hutch with the library's built-in scratch instead of a workspace,
    for callers that cannot allocate device memory (see include/dprc.h)."""
    _need_cuda(A, G, P, n)
    B, T, d = A.shape
    p, k = P.shape
    st = lib().dprc_norm_hutch_noalloc(_ptr(A), _ptr(G), _ptr(P), _dtype_code(A), B, T, d, p, k,
                                       _ptr(n), int(bool(accumulate)), _stream(A, stream))
    _check("dprc_norm_hutch_noalloc", st)
    return n


# Device error codes (DPRC_DEVERR_* of include/dprc.h).
(DPRC_DEVERR_PIPE_FULL, DPRC_DEVERR_PIPE_EMPTY, DPRC_DEVERR_ACCUM, DPRC_DEVERR_CLUSTER,
 DPRC_DEVERR_READY, DPRC_DEVERR_LAUNCH, DPRC_DEVERR_BOUNDS,
 DPRC_DEVERR_TOKEN) = (1, 2, 3, 4, 5, 6, 7, 8)
FAULT_READY_NEVER_MET, FAULT_CLUSTER_SHAPE = 0, 1


def dprc_test_hutch_fault(mode, wait_ns, As, Gs, Ps, n, ws, stream=None):
    """Failure-detection test of the one-launch Hutchinson kernel (see
    include/dprc.h): mode FAULT_READY_NEVER_MET makes every projection's wait
    for its sample's sketch run out after wait_ns; mode FAULT_CLUSTER_SHAPE
    launches a plan without clusters as clusters of 2.  Read the outcome with
    dprc_device_error(reset=True)."""
    L = len(As)
    if not (L == len(Gs) == len(Ps)) or L == 0:
        raise ValueError("As, Gs and Ps must be non-empty lists of the same length")
    _need_cuda(*As, *Gs, *Ps, n, ws)
    B, T = As[0].shape[0], As[0].shape[1]
    k = Ps[0].shape[1]
    d = (ctypes.c_int64 * L)(*[a.shape[2] for a in As])
    p = (ctypes.c_int64 * L)(*[g.shape[2] for g in Gs])
    ap = (ctypes.c_void_p * L)(*[_ptr(a) for a in As])
    gp = (ctypes.c_void_p * L)(*[_ptr(g) for g in Gs])
    pp = (ctypes.c_void_p * L)(*[_ptr(x) for x in Ps])
    st = lib().dprc_test_hutch_fault(int(mode), int(wait_ns), L, ap, gp, pp, d, p, B, T, k,
                                     _ptr(n), _ptr(ws), ws.numel(), _stream(As[0], stream))
    _check("dprc_test_hutch_fault", st)
    return n


def dprc_exact_norm(A, G, n, accumulate=False, ws=None, stream=None, form=DPRC_EXACT_AUTO):
    """n[i] (+)= ||A_i^T G_i||_F^2 exactly, by the direct form A_i^T G_i or the
    ghost form sum_{t,s} (A_i A_i^T)_{ts} (G_i G_i^T)_{ts} (form: one of
    DPRC_EXACT_*; AUTO takes the one with less work, see include/dprc.h)."""
    _need_cuda(A, G, n)
    B, T, d = A.shape
    p = G.shape[2]
    if ws is None:
        ws = workspace(DPRC_OP_EXACT, A, B, T, d, p, 0)
    if form == DPRC_EXACT_AUTO:
        st = lib().dprc_exact_norm(_ptr(A), _ptr(G), _dtype_code(A), B, T, d, p, _ptr(n),
                                   int(bool(accumulate)), _ptr(ws), ws.numel(),
                                   _stream(A, stream))
        _check("dprc_exact_norm", st)
    else:
        st = lib().dprc_exact_norm_form(_ptr(A), _ptr(G), _dtype_code(A), B, T, d, p, int(form),
                                        _ptr(n), int(bool(accumulate)), _ptr(ws), ws.numel(),
                                        _stream(A, stream))
        _check("dprc_exact_norm_form", st)
    return n


def dprc_exact_norm_plan(dtype, B, T, d, p, form=DPRC_EXACT_AUTO):
    """The form (DPRC_EXACT_DIRECT, _GHOST_N128 or _GHOST_N256 on tensor cores,
    _GHOST on CUDA cores) an exact-norm call with these sizes runs on the
    current device, 0 if it would be rejected."""
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return lib().dprc_exact_norm_plan(code, B, T, d, p, int(form))


def dprc_clip_factors(n, C, c, nonfinite=None, stream=None):
    """c[i] = min(1, C / sqrt(n[i])); non-finite or negative n gives 0."""
    _need_cuda(n, c, nonfinite)
    st = lib().dprc_clip_factors(_ptr(n), n.numel(), float(C), _ptr(c), _ptr(nonfinite),
                                 _stream(n, stream))
    _check("dprc_clip_factors", st)
    return c


def dprc_add_noise(grad, sigma, C, seed, step, stream=None):
    """grad += sigma * C * z (Philox4x32-10 + Box-Muller), in place."""
    _need_cuda(grad)
    st = lib().dprc_add_noise(_ptr(grad), grad.numel(), float(sigma), float(C),
                              int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
                              _stream(grad, stream))
    _check("dprc_add_noise", st)
    return grad


def dprc_add_noise_at(grad, first_element, sigma, C, seed, step, stream=None):
    """grad += sigma * C * z[first_element : first_element + grad.numel()], in
    place (float32 or bfloat16): the noise of one piece of a gradient kept in
    several buffers (see include/dprc.h)."""
    _need_cuda(grad)
    st = lib().dprc_add_noise_at(_ptr(grad), _dtype_code(grad), grad.numel(),
                                 int(first_element) & (2**64 - 1), float(sigma), float(C),
                                 int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
                                 _stream(grad, stream))
    _check("dprc_add_noise_at", st)
    return grad


def dprc_philox_words(out, first_block, seed, step, stream=None):
    """Fills out (int32 [n, 4]) with Philox blocks first_block .. first_block + n - 1."""
    _need_cuda(out)
    n_blocks = out.numel() // 4
    st = lib().dprc_philox_words(_ptr(out), n_blocks, int(first_block), int(seed) & (2**64 - 1),
                                 int(step) & (2**64 - 1), _stream(out, stream))
    _check("dprc_philox_words", st)
    return out


def dprc_device_error(reset=False):
    v = ctypes.c_int32(0)
    st = lib().dprc_device_error(ctypes.byref(v), int(bool(reset)))
    _check("dprc_device_error", st)
    return v.value


_events_keepalive = None


def dprc_set_phase_events(events):
    """Record these torch.cuda.Event objects between the stages of later calls
    on this thread (None turns it off)."""
    global _events_keepalive
    if not events:
        _events_keepalive = None
        _check("dprc_set_phase_events", lib().dprc_set_phase_events(None, 0))
        return
    for e in events:
        if not e.cuda_event:  # torch creates the event on its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _events_keepalive = (arr, events)
    _check("dprc_set_phase_events", lib().dprc_set_phase_events(arr, len(events)))


# ---------------------------------------------------------------------------
# The operators around the norm path (include/dprc.h says what each computes).
# ---------------------------------------------------------------------------
DPRC_ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
_U64 = 2**64 - 1


_scratch_kept = threading.local()
_SCRATCH_KEEP = 64 << 20  # larger workspaces are allocated per call
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)


def _empty(like, shape, stream, given, dtype=None):
    """An uninitialised tensor on like's device, of its dtype if none is given,
    for a call on the stream handle `stream`: allocated on that stream where the
    caller gave one (`given` not None), so that the memory's earlier and later
    uses are ordered against the call."""
    if dtype is None:
        dtype = like.dtype
    if given is None:  # (sizes as arguments of their own: 1 to 2 us less than a tuple or Size)
        return torch.empty(*shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)):
        return torch.empty(*shape, dtype=dtype, device=like.device)


def _current_stream_id(device):
    """torch's number of the current stream: the handle itself for a stream that
    torch does not own."""
    return torch._C._cuda_getCurrentStream(device)[0]


def _keeps_scratch(like, stream, given):
    """Whether a workspace may be kept for the stream: one of torch's own, which
    are never destroyed (the handle of another may come to name a new stream while
    the old one's work is pending), and not being captured, since a graph owns
    what it allocates."""
    if _capturing is None:
        return False
    if given is None:
        return not _capturing() and (stream == 0 or _current_stream_id(like.get_device()) != stream)
    if not isinstance(given, torch.cuda.Stream) or isinstance(given, torch.cuda.ExternalStream):
        return False
    with torch.cuda.stream(given):
        return not _capturing()


def _scratch(nbytes, like, stream, given):
    """A device workspace of nbytes for one call without a ws argument: kept
    per host thread, device and stream (calls of one thread on one stream run
    one after the other) and grown as needed, so that a call does not pay for
    an allocation.  Large ones are allocated fresh."""
    if nbytes > _SCRATCH_KEEP or not _keeps_scratch(like, stream, given):
        return _empty(like, (nbytes,), stream, given, torch.uint8)
    kept = _scratch_kept.__dict__
    key = (like.get_device(), stream)
    have = kept.get(key)
    if have is None or have.numel() < nbytes:
        size = 1 << max(16, (nbytes - 1).bit_length())
        # (the outgrown one was allocated on this stream, and its memory goes to later
        # work there, behind what may still use it)
        have = kept[key] = _empty(like, (size,), stream, given, torch.uint8)
    return have


def _same(name, t, dtype, shape, device):
    """An optional tensor of the call's dtype, shape and device."""
    if t is None or (t.dtype is dtype and (shape is None or t.shape == shape)
                     and t.device == device):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, the call's tensors are {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors are on {device}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} is needed")


def _beside(name, t, like):
    """A tensor on the call's device, of whatever type."""
    if t is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors are on {like.device}")


def _act(name):
    code = DPRC_ACTS.get(name)
    if code is None:
        raise ValueError(f"act is one of {sorted(DPRC_ACTS)}, not {name!r}")
    return code


def _token_bytes(tokens):
    if tokens.dtype == torch.int64:
        return 8
    if tokens.dtype == torch.int32:
        return 4
    raise TypeError(f"tokens are int32 or int64, not {tokens.dtype}")


def dprc_embed_lookup(W, tokens, scale=1.0, out=None, stream=None):
    """out[..., :] = scale * W[tokens[...]], zero rows for negative tokens."""
    V, d = W.shape
    _need_cuda(W, tokens, out)
    _beside("tokens", tokens, W)
    st = _stream(W, stream)
    shape = (*tokens.shape, d)
    if out is None:
        out = _empty(W, shape, st, stream)
    else:
        _same("out", out, W.dtype, shape, W.device)
    _check("dprc_embed_lookup",
           lib().dprc_embed_lookup(W.data_ptr(), _dtype_code(W), tokens.data_ptr(),
                                   _token_bytes(tokens), tokens.numel(), V, d, scale,
                                   out.data_ptr(), st))
    return out


class EmbedPlan:
    """The sorted token order of tokens [B][T] over a vocabulary of V
    (dprc_embed_plan), as dprc_embed_norm and dprc_embed_grad take it."""

    __slots__ = ("B", "T", "V", "buf")

    def __init__(self, B, T, V, buf):
        self.B, self.T, self.V, self.buf = B, T, V, buf


def dprc_embed_plan(tokens, V, buf=None, stream=None):
    """Sorts tokens [B][T]; returns an EmbedPlan.  buf: a uint8 device buffer
    of dprc_embed_plan_bytes(B * T, V) bytes to keep it in."""
    B, T = tokens.shape
    size = _token_bytes(tokens)
    _need_cuda(tokens, buf)
    _beside("buf", buf, tokens)
    st = _stream(tokens, stream)
    if buf is None:
        n = lib().dprc_embed_plan_bytes(B * T, V)
        if n == 0:
            raise DprcError("dprc_embed_plan_bytes", 2)
        buf = _empty(tokens, (n,), st, stream, torch.uint8)
    _check("dprc_embed_plan",
           lib().dprc_embed_plan(tokens.data_ptr(), size, B * T, V,
                                 buf.data_ptr(), buf.numel(), st))
    return EmbedPlan(B, T, int(V), buf)


def _embed_ws(G, plan, ws, stream, given):
    if G.dim() != 3 or G.shape[0] != plan.B or G.shape[1] != plan.T:
        raise ValueError(f"G has shape {tuple(G.shape)}, the plan is of {plan.B} x {plan.T} tokens")
    _beside("the plan", plan.buf, G)
    _beside("ws", ws, G)
    if ws is None:
        n = lib().dprc_embed_workspace_bytes(_dtype_code(G), plan.B, plan.T, G.shape[2])
        if n == 0:
            raise DprcError("dprc_embed_workspace_bytes", 2)
        ws = _scratch(n, G, stream, given)
    return ws


def dprc_embed_norm(G, plan, n, scale=1.0, accumulate=False, ws=None, stream=None):
    """n[i] (+)= scale^2 sum_v ||sum_{t: tok_it = v} G_it||^2, exactly."""
    _need_cuda(G, n, ws, plan.buf)
    _same("n", n, torch.float32, (plan.B,), G.device)
    st = _stream(G, stream)
    ws = _embed_ws(G, plan, ws, st, stream)
    _check("dprc_embed_norm",
           lib().dprc_embed_norm(G.data_ptr(), _dtype_code(G), plan.B, plan.T, plan.V, G.shape[2],
                                 scale, plan.buf.data_ptr(), plan.buf.numel(), n.data_ptr(),
                                 1 if accumulate else 0, ws.data_ptr(), ws.numel(), st))
    return n


def dprc_embed_grad(G, plan, dW, c=None, scale=1.0, accumulate=False, ws=None, stream=None):
    """dW[v] (+)= scale sum_i c[i] sum_{t: tok_it = v} G_it (c None: all 1)."""
    _need_cuda(G, dW, c, ws, plan.buf)
    _same("dW", dW, G.dtype, (plan.V, G.shape[2]), G.device)
    _same("c", c, torch.float32, (plan.B,), G.device)
    st = _stream(G, stream)
    ws = _embed_ws(G, plan, ws, st, stream)
    _check("dprc_embed_grad",
           lib().dprc_embed_grad(G.data_ptr(), _dtype_code(G), _ptr(c), plan.B, plan.T, plan.V,
                                 G.shape[2], scale, plan.buf.data_ptr(), plan.buf.numel(),
                                 dW.data_ptr(), 1 if accumulate else 0, ws.data_ptr(), ws.numel(),
                                 st))
    return dW


def dprc_dropout(x, p, seed, step, residual=None, first_element=0, out=None, stream=None):
    """residual + dropout(x) with the mask of (seed, step) from element
    first_element on; the gradient is the same call on dy without residual."""
    _need_cuda(x, residual, out)
    st = _stream(x, stream)
    if out is None:
        out = _empty(x, x.shape, st, stream) if x.dim() > 0 else torch.empty_like(x)
    else:
        _same("out", out, x.dtype, x.shape, x.device)
    if residual is not None:
        _same("residual", residual, x.dtype, x.shape, x.device)
    _check("dprc_dropout",
           lib().dprc_dropout(x.data_ptr(), _ptr(residual), _dtype_code(x), x.numel(),
                              int(first_element) & _U64, p, int(seed) & _U64, int(step) & _U64,
                              out.data_ptr(), st))
    return out


def _linear_ws(like, M, K, N, grad, ws, stream, given):
    _beside("ws", ws, like)
    if ws is None:
        n = lib().dprc_linear_workspace_bytes(_dtype_code(like), M, K, N, grad)
        if n == 0:
            raise DprcError("dprc_linear_workspace_bytes", 2)
        ws = _scratch(n, like, stream, given)
    return ws


def dprc_linear(X, W, bias=None, act="none", p=0.0, seed=0, step=0, residual=None, Z=None,
                out=None, ws=None, stream=None):
    """Y = residual + dropout(act(X W^T + bias)) for X [..., K], W [N][K]; Z
    receives X W^T + bias (needed by the gradient of an activation)."""
    N, K = W.shape
    if X.shape[-1] != K:
        raise ValueError(f"X has width {X.shape[-1]}, W {K}")
    shape = (*X.shape[:-1], N)
    M = X.numel() // K if K > 0 else 0
    dt, dev = X.dtype, X.device
    _need_cuda(X, W, bias, residual, Z, out, ws)
    st = _stream(X, stream)
    _same("W", W, dt, None, dev)
    _same("bias", bias, dt, (N,), dev)
    _same("residual", residual, dt, shape, dev)
    _same("Z", Z, dt, shape, dev)
    _same("out", out, dt, shape, dev)
    if out is None:
        out = _empty(X, shape, st, stream)
    ws = _linear_ws(X, M, K, N, 0, ws, st, stream)
    _check("dprc_linear",
           lib().dprc_linear(X.data_ptr(), W.data_ptr(), _ptr(bias), _ptr(residual),
                             _dtype_code(X), M, K, N, _act(act), p, int(seed) & _U64,
                             int(step) & _U64, _ptr(Z), out.data_ptr(), ws.data_ptr(), ws.numel(),
                             st))
    return out


def dprc_linear_grad(dY, X, W, Z=None, act="none", p=0.0, seed=0, step=0, dX=None, dW=None,
                     db=None, dZ=None, ws=None, stream=None):
    """Gradient of dprc_linear into those of dX [..., K], dW [N][K], db [N] and
    dZ [..., N] that are given (act, p, seed, step as in its call)."""
    N, K = W.shape
    M = dY.numel() // N if N > 0 else 0
    lead = dY.shape[:-1]
    dt, dev = dY.dtype, dY.device
    if dY.shape[-1] != N:
        raise ValueError(f"dY has width {dY.shape[-1]}, W {N} rows")
    _need_cuda(dY, X, W, Z, dX, dW, db, dZ, ws)
    _same("X", X, dt, (*lead, K), dev)
    _same("W", W, dt, None, dev)
    _same("Z", Z, dt, dY.shape, dev)
    _same("dX", dX, dt, (*lead, K), dev)
    _same("dW", dW, dt, (N, K), dev)
    _same("db", db, dt, (N,), dev)
    _same("dZ", dZ, dt, dY.shape, dev)
    st = _stream(dY, stream)
    ws = _linear_ws(dY, M, K, N, 1, ws, st, stream)
    _check("dprc_linear_grad",
           lib().dprc_linear_grad(dY.data_ptr(), _ptr(X), W.data_ptr(), _ptr(Z), _dtype_code(dY),
                                  M, K, N, _act(act), p, int(seed) & _U64, int(step) & _U64,
                                  _ptr(dX), _ptr(dW), _ptr(db), _ptr(dZ), ws.data_ptr(),
                                  ws.numel(), st))
