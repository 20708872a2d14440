"""gated_delta_rule_21_gb300 -- Python binding of libkda, the GB300 (sm_103a)
chunked Kimi Delta Attention forward.

The binding only marshals arguments: it checks dtypes/shapes/devices of torch
tensors, allocates outputs and the workspace with torch (device memory and
streams are all torch is used for), and calls the C ABI declared in
``include/kda.h`` through ctypes.  Every step of the computation runs in the
library's CUDA kernels; there is no CPU or eager fallback, and importing this
package fails loudly when ``libkda.so`` has not been built.

Entry points (same names as the C ABI, minus the ``kda_`` prefix):

* :func:`chunk_fwd` -- the chunked KDA forward (``kda_chunk_fwd[_ex]``).
* :func:`chunk_bwd` -- its gradient (``kda_chunk_bwd``).
* :func:`short_conv_silu` -- the causal conv + SiLU (+ L2) prologue.
* :func:`step` -- one token per sequence through the delta rule
  (``kda_step``), on cached states.
* :func:`ssm_fwd`, :func:`ssm_step` -- the selective state space operator
  with its short convolution, on prompts and on single tokens.
* :func:`block_norm`, :func:`block_norm_bwd` -- the norms before and after a
  block fused with its gate and residual scale, and their gradients.
* :func:`workspace_size`, :func:`read_device_status`,
  :func:`clear_device_status`, :func:`status_string`, :func:`version`.
* :func:`lib` -- the raw ctypes library with typed signatures.

``stream`` is a ``torch.cuda.Stream`` (None: the current one).  What a call
allocates belongs to that stream, as under ``torch.cuda.stream(stream)``: wait
for it, and ``record_stream`` outputs that another stream goes on to use.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK = 0
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED",
                3: "KDA_ERR_ALIGNMENT", 4: "KDA_ERR_WORKSPACE", 5: "KDA_ERR_CUDA",
                6: "KDA_ERR_TIMEOUT", 7: "KDA_ERR_DEVICE"}
IMPLS = {"auto": 0, "simt": 1, "tc": 2, "split": 3}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
CHUNK = 64


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({status_string(status)})")


class kda_ssm_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "H", "P", "N", "G", "dtype")] + \
        [(n, ctypes.c_longlong) for n in ("xbc_stride_b", "xbc_stride_t", "z_stride_b",
                                          "z_stride_t", "dt_stride_b", "dt_stride_t")]


class kda_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("gate_act", ctypes.c_int), ("gate_rows", ctypes.c_longlong),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class kda_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("K", ctypes.c_int), ("V", ctypes.c_int),
                ("qkv_dtype", ctypes.c_int)]


_lib = None
_lock = threading.Lock()


def lib():
    """Load libkda.so (raising if it is missing) and return the typed CDLL."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"libkda.so is not built ({LIB_PATH}); run "
                "`python -c 'import __graft_entry__ as g; g.build()'` or "
                "`python -m gated_delta_rule_21_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, u64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        sp = ctypes.POINTER(kda_shape)
        L.kda_chunk_fwd_workspace_size.argtypes = [sp, i]
        L.kda_chunk_fwd_workspace_size.restype = u64
        L.kda_chunk_fwd_workspace_size_for.argtypes = [sp, i, i]
        L.kda_chunk_fwd_workspace_size_for.restype = u64
        L.kda_chunk_fwd_workspace_size_packed.argtypes = [sp, i]
        L.kda_chunk_fwd_workspace_size_packed.restype = u64
        L.kda_chunk_fwd.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp,
                                    vp, vp, u64, vp]
        L.kda_chunk_fwd.restype = i
        L.kda_chunk_fwd_ex.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp,
                                       vp, vp, vp, u64, i, i, vp]
        L.kda_chunk_fwd_ex.restype = i
        L.kda_short_conv_silu.argtypes = [sp, vp, vp, vp, vp, vp, i, vp, vp,
                                          vp, vp]
        L.kda_short_conv_silu.restype = i
        L.kda_read_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.kda_read_device_status.restype = i
        L.kda_clear_device_status.argtypes = [vp, vp]
        L.kda_clear_device_status.restype = i
        L.kda_status_string.argtypes = [i]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_impl_available.argtypes = [i, sp, i]
        L.kda_impl_available.restype = i
        L.kda_version.argtypes = []
        L.kda_version.restype = i
        L.kda_chunk_fwd_host_buffer_size.argtypes = [sp, i]
        L.kda_chunk_fwd_host_buffer_size.restype = u64
        L.kda_chunk_fwd_host.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp,
                                         vp, vp, u64, vp]
        L.kda_chunk_fwd_host.restype = i
        L.kda_chunk_bwd_workspace_size.argtypes = [sp, i]
        L.kda_chunk_bwd_workspace_size.restype = u64
        L.kda_chunk_bwd.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp, vp, vp,
                                    vp, vp, vp, vp, u64, vp]
        L.kda_chunk_bwd.restype = i
        L.kda_chunk_bwd_workspace_size_for.argtypes = [sp, i, i]
        L.kda_chunk_bwd_workspace_size_for.restype = u64
        L.kda_chunk_bwd_workspace_size_packed.argtypes = [sp, i]
        L.kda_chunk_bwd_workspace_size_packed.restype = u64
        L.kda_chunk_fwd_save_workspace_size.argtypes = [sp, i]
        L.kda_chunk_fwd_save_workspace_size.restype = u64
        L.kda_chunk_fwd_save.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp, u64, vp]
        L.kda_chunk_fwd_save.restype = i
        L.kda_chunk_bwd_from_saved.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp, vp, vp, u64, vp]
        L.kda_chunk_bwd_from_saved.restype = i
        L.kda_chunk_bwd_ex.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, vp, u64, i, vp]
        L.kda_chunk_bwd_ex.restype = i
        L.kda_chunk_fwd_scan_workspace_size.argtypes = [sp, i]
        L.kda_chunk_fwd_scan_workspace_size.restype = u64
        L.kda_chunk_fwd_scan_segments.argtypes = [sp, i]
        L.kda_chunk_fwd_scan_segments.restype = i
        L.kda_chunk_fwd_scan.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, i, vp, u64, vp]
        L.kda_chunk_fwd_scan.restype = i
        L.kda_chunk_fwd_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp]
        L.kda_chunk_fwd_noalloc.restype = i
        L.kda_chunk_fwd_noalloc_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        L.kda_chunk_fwd_noalloc_status.restype = i
        ssp, ndp, ll = ctypes.POINTER(kda_ssm_shape), ctypes.POINTER(kda_norm_desc), ctypes.c_longlong
        L.kda_ssm_fwd_workspace_size.argtypes = [ssp, i]
        L.kda_ssm_fwd_workspace_size.restype = u64
        L.kda_ssm_fwd.argtypes = [ssp] + [vp] * 15 + [u64, i, vp]
        L.kda_ssm_fwd.restype = i
        L.kda_step_workspace_size.argtypes = [i, i]
        L.kda_step_workspace_size.restype = u64
        L.kda_ssm_step.argtypes = [ssp] + [vp] * 9 + [i] + [vp] * 4 + [u64, vp]
        L.kda_ssm_step.restype = i
        L.kda_step.argtypes = [sp, vp, vp, vp, ll, ll, ll, vp, vp, f, vp, vp, i, vp, i, vp, vp, vp,
                               u64, vp]
        L.kda_step.restype = i
        L.kda_block_norm_fwd.argtypes = [ndp] + [vp] * 9
        L.kda_block_norm_fwd.restype = i
        L.kda_block_norm_bwd_workspace_size.argtypes = [ndp, i]
        L.kda_block_norm_bwd_workspace_size.restype = u64
        L.kda_block_norm_bwd.argtypes = [ndp] + [vp] * 14 + [u64, vp]
        L.kda_block_norm_bwd.restype = i
        L.kda_selftest_wait_timeout.argtypes = [vp, ctypes.c_longlong, vp]
        L.kda_selftest_wait_timeout.restype = i
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def version() -> int:
    return lib().kda_version()


def impl_available(impl, B, T, H, K, V, dtype=torch.bfloat16, v_tile=0) -> bool:
    """Whether implementation ``impl`` ("auto"/"simt"/"tc") runs this shape."""
    s = make_shape(B, T, H, K, V, dtype)
    return bool(lib().kda_impl_available(IMPLS[impl], ctypes.byref(s), int(v_tile)))


def make_shape(B, T, H, K, V, dtype) -> kda_shape:
    if dtype not in DTYPES:
        raise TypeError(f"q/k/v dtype must be float32 or bfloat16, got {dtype}")
    return kda_shape(int(B), int(T), int(H), int(K), int(V), DTYPES[dtype])


def workspace_size(B, T, H, K, V, dtype=torch.bfloat16, has_segment_ids=False,
                   impl=None) -> int:
    """Workspace bytes: what the fastest kernel needs (impl None, the C
    default query) or what ``impl`` needs ("simt" gives the smallest size
    any path accepts)."""
    s = make_shape(B, T, H, K, V, dtype)
    if impl is None:
        return int(lib().kda_chunk_fwd_workspace_size(ctypes.byref(s), int(bool(has_segment_ids))))
    return int(lib().kda_chunk_fwd_workspace_size_for(ctypes.byref(s), int(bool(has_segment_ids)),
                                                      IMPLS[impl]))


def workspace_size_packed(B, T, H, K, V, max_runs_per_row, dtype=torch.bfloat16) -> int:
    """Split-path workspace for packed inputs with at most ``max_runs_per_row``
    runs per row."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_fwd_workspace_size_packed(ctypes.byref(s), int(max_runs_per_row)))


def alloc_workspace(B, T, H, K, V, dtype=torch.bfloat16, has_segment_ids=False,
                    device=None, impl=None, max_runs_per_row=None) -> torch.Tensor:
    """Zero-filled workspace of the size ``impl`` needs (uint8 device tensor);
    with ``max_runs_per_row`` the split path's packed bound is used."""
    n = 0
    if max_runs_per_row is not None and has_segment_ids and impl in ("auto", "split"):
        n = workspace_size_packed(B, T, H, K, V, max_runs_per_row, dtype)
    if n == 0:
        n = workspace_size(B, T, H, K, V, dtype, has_segment_ids, impl)
    if n == 0:
        raise KdaError(1, "workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_its_stream(f):
    """A call with ``stream`` is the call made under ``torch.cuda.stream(stream)``:
    the outputs and scratch memory that it allocates belong to that stream, and
    scratch memory is zeroed there before the kernels that count on it."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None or not _elsewhere(stream):
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)

    return call


def _elsewhere(stream):
    return stream != torch.cuda.current_stream(stream.device)


@_on_its_stream
def chunk_fwd(q, k, v, g, beta, scale=None, chunk_size=CHUNK, initial_state=None,
              segment_ids=None, output_final_state=False, out=None,
              final_state_out=None, workspace=None, impl="auto", v_tile=0,
              stream=None, max_runs_per_row=None):
    """Chunked KDA forward on the GPU.

    q, k: [B,T,H,K]; v: [B,T,H,V] (bf16 or fp32, same dtype); g: [B,T,H,K]
    fp32 log-decay in [-5, 0]; beta: [B,T,H] fp32; initial_state: [B,H,K,V]
    fp32 or None; segment_ids: [B,T] int32 (1-based, 0 = padding) or None.
    ``scale`` None means K**-0.5.  ``max_runs_per_row`` bounds the runs
    per row when the workspace is allocated here for packed inputs.
    Returns ``(o, final_state or None)``.
    """
    B, T, H, K = q.shape
    V = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("chunk_fwd needs CUDA tensors")
    dt = q.dtype
    _check(q, "q", (B, T, H, K), dt, dev)
    _check(k, "k", (B, T, H, K), dt, dev)
    _check(v, "v", (B, T, H, V), dt, dev)
    _check(g, "g", (B, T, H, K), torch.float32, dev)
    _check(beta, "beta", (B, T, H), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H, K, V), torch.float32, dev)
    _check(segment_ids, "segment_ids", (B, T), torch.int32, dev)
    if scale is None:
        scale = K ** -0.5
    o = out if out is not None else torch.empty(B, T, H, V, dtype=dt, device=dev)
    _check(o, "out", (B, T, H, V), dt, dev)
    fs = None
    if output_final_state:
        fs = final_state_out if final_state_out is not None else torch.empty(
            B, H, K, V, dtype=torch.float32, device=dev)
        _check(fs, "final_state_out", (B, H, K, V), torch.float32, dev)
    if workspace is None:
        workspace = alloc_workspace(B, T, H, K, V, dt, segment_ids is not None, dev, impl=impl,
                                    max_runs_per_row=max_runs_per_row)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_fwd_ex(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        float(scale), int(chunk_size), _ptr(initial_state), _ptr(segment_ids),
        _ptr(o), _ptr(fs), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        IMPLS[impl], int(v_tile), _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd")
    return o, fs


def scan_workspace_size(B, T, H, K, V, dtype=torch.bfloat16, n_segments=0) -> int:
    """Workspace bytes of chunk_fwd_scan (0 when the shape is not served)."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_fwd_scan_workspace_size(ctypes.byref(s), int(n_segments)))


def scan_segments(B, T, H, K, V, dtype=torch.bfloat16, n_segments=0) -> int:
    """Segments per row chunk_fwd_scan uses for this request (0: not served)."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_fwd_scan_segments(ctypes.byref(s), int(n_segments)))


@_on_its_stream
def chunk_fwd_scan(q, k, v, g, beta, scale=None, chunk_size=CHUNK, initial_state=None,
                   output_final_state=False, n_segments=0, out=None, final_state_out=None,
                   workspace=None, stream=None):
    """The chunked forward as a chunk-parallel state scan over ``n_segments``
    segments per row (0: chosen to fill the GPU); rows without segment ids,
    bf16 with K = V = 128.  Same results as chunk_fwd up to rounding.
    Returns ``(o, final_state or None)``."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("chunk_fwd_scan needs CUDA tensors")
    _check(q, "q", (B, T, H, K), dt, dev)
    _check(k, "k", (B, T, H, K), dt, dev)
    _check(v, "v", (B, T, H, V), dt, dev)
    _check(g, "g", (B, T, H, K), torch.float32, dev)
    _check(beta, "beta", (B, T, H), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H, K, V), torch.float32, dev)
    if scale is None:
        scale = K ** -0.5
    o = out if out is not None else torch.empty(B, T, H, V, dtype=dt, device=dev)
    _check(o, "out", (B, T, H, V), dt, dev)
    fs = None
    if output_final_state:
        fs = final_state_out if final_state_out is not None else torch.empty(
            B, H, K, V, dtype=torch.float32, device=dev)
        _check(fs, "final_state_out", (B, H, K, V), torch.float32, dev)
    if workspace is None:
        n = scan_workspace_size(B, T, H, K, V, dt, n_segments)
        if n == 0:
            raise KdaError(2, "kda_chunk_fwd_scan_workspace_size")
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_fwd_scan(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        int(chunk_size), _ptr(initial_state), _ptr(o), _ptr(fs), int(n_segments),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_scan")
    return o, fs


def bwd_workspace_size(B, T, H, K, V, dtype=torch.bfloat16, has_segment_ids=False,
                       impl=None) -> int:
    """Workspace bytes of chunk_bwd for this shape (0 when unsupported):
    the AUTO choice (impl None) or what ``impl`` ("auto", "simt", "tc")
    needs."""
    s = make_shape(B, T, H, K, V, dtype)
    if impl is None:
        return int(lib().kda_chunk_bwd_workspace_size(ctypes.byref(s), int(bool(has_segment_ids))))
    return int(lib().kda_chunk_bwd_workspace_size_for(ctypes.byref(s), int(bool(has_segment_ids)),
                                                      IMPLS[impl]))


def bwd_workspace_size_packed(B, T, H, K, V, max_runs_per_row, dtype=torch.bfloat16) -> int:
    """Tensor-core backward workspace for inputs with segment ids and at most
    ``max_runs_per_row`` runs per row (0 when that path does not apply)."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_bwd_workspace_size_packed(ctypes.byref(s), int(max_runs_per_row)))


@_on_its_stream
def chunk_bwd(q, k, v, g, beta, d_o, scale=None, chunk_size=CHUNK, initial_state=None,
              segment_ids=None, d_final=None, want_d_initial=True, workspace=None,
              stream=None, impl="auto"):
    """Gradient of chunk_fwd on the GPU: given ``d_o`` [B,T,H,V] (dtype of q)
    and ``d_final`` [B,H,K,V] fp32 or None, returns fp32 ``(dq, dk, dv, dg,
    dbeta, d_initial or None)`` of ``sum(d_o * o) + sum(d_final *
    final_state)``.  Inputs as chunk_fwd; ``impl``: "auto" (the tensor cores
    where they apply), "tc" or "simt"."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("chunk_bwd needs CUDA tensors")
    dt = q.dtype
    _check(q, "q", (B, T, H, K), dt, dev)
    _check(k, "k", (B, T, H, K), dt, dev)
    _check(v, "v", (B, T, H, V), dt, dev)
    _check(d_o, "d_o", (B, T, H, V), dt, dev)
    _check(g, "g", (B, T, H, K), torch.float32, dev)
    _check(beta, "beta", (B, T, H), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H, K, V), torch.float32, dev)
    _check(d_final, "d_final", (B, H, K, V), torch.float32, dev)
    _check(segment_ids, "segment_ids", (B, T), torch.int32, dev)
    if scale is None:
        scale = K ** -0.5
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk, dg = (torch.empty(B, T, H, K, **f32) for _ in range(3))
    dv = torch.empty(B, T, H, V, **f32)
    dbeta = torch.empty(B, T, H, **f32)
    d_init = torch.empty(B, H, K, V, **f32) if want_d_initial else None
    if workspace is None:
        n = bwd_workspace_size(B, T, H, K, V, dt, segment_ids is not None, impl)
        if n == 0:
            raise KdaError(2, "kda_chunk_bwd_workspace_size")
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_bwd_ex(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        int(chunk_size), _ptr(initial_state), _ptr(segment_ids), _ptr(d_o), _ptr(d_final),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(d_init), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), IMPLS[impl],
        _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd_ex")
    return dq, dk, dv, dg, dbeta, d_init


def fwd_save_workspace_size(B, T, H, K, V, dtype=torch.bfloat16, has_segment_ids=False) -> int:
    """Workspace bytes of chunk_fwd_save (0 when that path does not apply)."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_fwd_save_workspace_size(ctypes.byref(s), int(bool(has_segment_ids))))


@_on_its_stream
def chunk_fwd_save(q, k, v, g, beta, scale=None, chunk_size=CHUNK, initial_state=None,
                   segment_ids=None, output_final_state=True, workspace=None, stream=None):
    """The forward of a training step (``kda_chunk_fwd_save``): returns
    ``(o, final_state or None, workspace)``, o and the final state as
    chunk_fwd's split path computes them, the workspace holding what
    chunk_bwd_from_saved reads.  bf16, K = V = 128."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("chunk_fwd_save needs CUDA tensors")
    dt = q.dtype
    _check(q, "q", (B, T, H, K), dt, dev)
    _check(k, "k", (B, T, H, K), dt, dev)
    _check(v, "v", (B, T, H, V), dt, dev)
    _check(g, "g", (B, T, H, K), torch.float32, dev)
    _check(beta, "beta", (B, T, H), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H, K, V), torch.float32, dev)
    _check(segment_ids, "segment_ids", (B, T), torch.int32, dev)
    if scale is None:
        scale = K ** -0.5
    o = torch.empty(B, T, H, V, dtype=dt, device=dev)
    fs = torch.empty(B, H, K, V, dtype=torch.float32, device=dev) if output_final_state else None
    if workspace is None:
        n = fwd_save_workspace_size(B, T, H, K, V, dt, segment_ids is not None)
        if n == 0:
            raise KdaError(2, "kda_chunk_fwd_save_workspace_size")
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_fwd_save(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        int(chunk_size), _ptr(initial_state), _ptr(segment_ids), _ptr(o), _ptr(fs),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_save")
    return o, fs, workspace


@_on_its_stream
def chunk_bwd_from_saved(q, k, v, g, beta, d_o, workspace, scale=None, chunk_size=CHUNK,
                         initial_state=None, segment_ids=None, d_final=None,
                         want_d_initial=True, stream=None):
    """The backward of a training step (``kda_chunk_bwd_from_saved``) on the
    workspace a chunk_fwd_save of the same inputs left: returns the
    gradients as chunk_bwd."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    dev = q.device
    dt = q.dtype
    _check(d_o, "d_o", (B, T, H, V), dt, dev)
    _check(d_final, "d_final", (B, H, K, V), torch.float32, dev)
    if scale is None:
        scale = K ** -0.5
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk, dg = (torch.empty(B, T, H, K, **f32) for _ in range(3))
    dv = torch.empty(B, T, H, V, **f32)
    dbeta = torch.empty(B, T, H, **f32)
    d_init = torch.empty(B, H, K, V, **f32) if want_d_initial else None
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_bwd_from_saved(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        int(chunk_size), _ptr(initial_state), _ptr(segment_ids), _ptr(d_o), _ptr(d_final),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(d_init), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd_from_saved")
    return dq, dk, dv, dg, dbeta, d_init


@_on_its_stream
def short_conv_silu(x_q, x_k, x_v, w, segment_ids=None, l2norm_qk=True,
                    stream=None):
    """Segment-aware causal depthwise conv (width 4) + SiLU on q, k, v, then
    optional L2 norm of q and k.  x_q, x_k: [B,T,H,K]; x_v: [B,T,H,V];
    w: fp32 [3, H*K, 4] (q, k, v weight blocks; needs K == V) or a flat
    tensor of 4*(2*H*K + H*V) floats.  Returns (q, k, v)."""
    B, T, H, K = x_q.shape
    V = x_v.shape[-1]
    dev, dt = x_q.device, x_q.dtype
    _check(x_q, "x_q", (B, T, H, K), dt, dev)
    _check(x_k, "x_k", (B, T, H, K), dt, dev)
    _check(x_v, "x_v", (B, T, H, V), dt, dev)
    _check(segment_ids, "segment_ids", (B, T), torch.int32, dev)
    if w.dtype != torch.float32 or w.device != dev or not w.is_contiguous() \
            or w.numel() != 4 * (2 * H * K + H * V):
        raise ValueError("w must be contiguous fp32 with 4*(2*H*K + H*V) elements")
    q = torch.empty_like(x_q)
    k = torch.empty_like(x_k)
    v = torch.empty_like(x_v)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_short_conv_silu(
        ctypes.byref(s), _ptr(x_q), _ptr(x_k), _ptr(x_v), _ptr(w),
        _ptr(segment_ids), int(bool(l2norm_qk)), _ptr(q), _ptr(k), _ptr(v),
        _stream_ptr(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_short_conv_silu")
    return q, k, v


def host_buffer_size(B, T, H, K, V, dtype=torch.bfloat16, has_segment_ids=False) -> int:
    """Bytes of device memory chunk_fwd_host needs for this shape."""
    s = make_shape(B, T, H, K, V, dtype)
    return int(lib().kda_chunk_fwd_host_buffer_size(ctypes.byref(s), 1 if has_segment_ids else 0))


@_on_its_stream
def chunk_fwd_host(q, k, v, g, beta, scale=None, chunk_size=CHUNK, initial_state=None,
                   segment_ids=None, output_final_state=False, out=None,
                   final_state_out=None, device_buffer=None, stream=None):
    """End-to-end forward on HOST tensors (pin them for asynchronous copies):
    the library copies the inputs in, runs the forward and copies o (and the
    final state) back, pipelined over token ranges (over head groups with
    segment ids).  ``device_buffer`` is a
    zero-filled CUDA uint8 tensor of host_buffer_size() bytes (allocated here
    when None).  The host outputs are valid once ``stream`` synchronises.
    Returns ``(o, final_state or None)`` (CPU tensors)."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    cpu = torch.device("cpu")
    dt = q.dtype
    for t, name, shape, tdt in ((q, "q", (B, T, H, K), dt), (k, "k", (B, T, H, K), dt),
                                (v, "v", (B, T, H, V), dt),
                                (g, "g", (B, T, H, K), torch.float32),
                                (beta, "beta", (B, T, H), torch.float32),
                                (initial_state, "initial_state", (B, H, K, V), torch.float32),
                                (segment_ids, "segment_ids", (B, T), torch.int32)):
        _check(t, name, shape, tdt, cpu)
    if scale is None:
        scale = K ** -0.5
    o = out if out is not None else torch.empty(B, T, H, V, dtype=dt).pin_memory()
    _check(o, "out", (B, T, H, V), dt, cpu)
    fs = None
    if output_final_state:
        fs = final_state_out if final_state_out is not None else torch.empty(
            B, H, K, V, dtype=torch.float32).pin_memory()
        _check(fs, "final_state_out", (B, H, K, V), torch.float32, cpu)
    n = host_buffer_size(B, T, H, K, V, dt, segment_ids is not None)
    if n == 0:
        raise KdaError(2, "kda_chunk_fwd_host_buffer_size")
    dev = torch.device("cuda", torch.cuda.current_device())
    if device_buffer is None:
        device_buffer = torch.zeros(n, dtype=torch.uint8, device=dev)
    s = make_shape(B, T, H, K, V, dt)
    st = lib().kda_chunk_fwd_host(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        int(chunk_size), _ptr(initial_state), _ptr(segment_ids), _ptr(o), _ptr(fs),
        _ptr(device_buffer), int(device_buffer.numel() * device_buffer.element_size()),
        _stream_ptr(stream, device_buffer.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_host")
    return o, fs


def read_device_status(workspace, stream=None) -> int:
    """Synchronise the stream and return the device status bits (0 = clean)."""
    bits = ctypes.c_uint32(0)
    st = lib().kda_read_device_status(_ptr(workspace), _stream_ptr(stream, workspace.device),
                                      ctypes.byref(bits))
    if st not in (KDA_OK, 4, 6, 7):
        raise KdaError(st, "kda_read_device_status")
    return int(bits.value)


def selftest_wait_timeout(workspace, limit_cycles=1 << 20, stream=None) -> None:
    """Enqueue the bounded-wait self-test: one device wait that nothing ends,
    given up after ``limit_cycles`` SM clocks, reported as KDA_DEVICE_TIMEOUT
    in ``workspace``'s status word (read it with read_device_status)."""
    st = lib().kda_selftest_wait_timeout(_ptr(workspace), int(limit_cycles),
                                         _stream_ptr(stream, workspace.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_wait_timeout")


def clear_device_status(workspace, stream=None) -> None:
    st = lib().kda_clear_device_status(_ptr(workspace), _stream_ptr(stream, workspace.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_clear_device_status")


# ---------------------------------------------------------------------------
# one token per sequence, the state space operator, the norms around a block
#
# Single-token calls take a few microseconds on the GPU, so the host side of
# these calls is kept short: descriptors are made once per shape, a tensor is
# checked by four attribute reads, messages are made only to be raised, and a
# call with a stream calls itself under it instead of being wrapped.

_f32, _i32 = torch.float32, torch.int32


def _lib_now():
    return _lib if _lib is not None else lib()


def _refuse(t, name, shape, dtype, device, contiguous):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _at(t, name, shape, dtype, device):
    """Address of a contiguous tensor of this shape, or None for None."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == device):
        _refuse(t, name, shape, dtype, device, True)
    return t.data_ptr()


def _rows(t, name, shape, dtype, device):
    """Address and row stride of a tensor whose dimensions after the first
    are contiguous (the rows may be slices of something wider)."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device):
        _refuse(t, name, shape, dtype, device, False)
    st = t.stride()
    n = 1
    for d in range(len(shape) - 1, 0, -1):
        if st[d] != n and shape[d] != 1:
            raise ValueError(f"the dimensions of {name} after the first must be contiguous")
        n *= shape[d]
    return t.data_ptr(), st[0]


def _start(t, where):
    """Device index and dtype of a call's first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{where} needs CUDA tensors")
    if t.dtype not in DTYPES:
        raise TypeError(f"{where}: dtype must be float32 or bfloat16, got {t.dtype}")
    return t.get_device(), t.dtype


def _scratch(workspace, need, device, where, zeros):
    """The workspace, or a new one whose first ``zeros`` bytes are zero."""
    if workspace is None:
        if need == 0:
            raise KdaError(2, where)
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if zeros:
            workspace[:zeros].zero_()
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


@functools.lru_cache(maxsize=1024)
def _shape_ref(*fields):
    return ctypes.byref(kda_shape(*fields))


@functools.lru_cache(maxsize=1024)
def _ssm_ref(*fields):
    return ctypes.byref(kda_ssm_shape(*fields))


@functools.lru_cache(maxsize=1024)
def _norm_ref(*fields):
    return ctypes.byref(kda_norm_desc(*fields))


def step_workspace_size(B, H) -> int:
    """Workspace bytes of :func:`step` and :func:`ssm_step`."""
    return int(lib().kda_step_workspace_size(int(B), int(H)))


def alloc_step_workspace(B, H, device=None) -> torch.Tensor:
    """Zero-filled workspace of :func:`step` and :func:`ssm_step` (one for
    each stream that makes such calls)."""
    n = step_workspace_size(B, H)
    if n == 0:
        raise KdaError(1, "kda_step_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def step(q, k, v, g, beta, state, scale=None, slots=None, conv_w=None, conv_state=None,
         l2norm_qk=False, out=None, workspace=None, stream=None):
    """One token per sequence through the delta rule, on cached states.

    q, k: [B,H,K]; v: [B,H,V] (bf16 or fp32; any stride between the rows);
    g: [B,H,K] fp32 log-decay; beta: [B,H] fp32; state: [n_slots,H,K,V] fp32,
    moved on in place.  ``slots`` [B] int32 gives each sequence's place in
    the cache (None: its row; a place outside the cache marks an idle
    sequence, whose output is 0).  With ``conv_w`` (as short_conv_silu) and
    ``conv_state`` [n_slots,3,H*(2K+V)] (moved on in place) q, k, v are the
    inputs of the convolution; after a prompt it holds the last three inputs of
    short_conv_silu of each sequence, zeros where there were fewer.  Returns o
    [B,H,V]."""
    if stream is not None and _elsewhere(stream):
        with torch.cuda.stream(stream):
            return step(q, k, v, g, beta, state, scale, slots, conv_w, conv_state, l2norm_qk, out,
                        workspace)
    dev, dt = _start(q, "step")
    B, H, K = q.shape
    V = v.shape[-1]
    n_slots, C = state.shape[0], H * (2 * K + V)
    qp, qs = _rows(q, "q", (B, H, K), dt, dev)
    kp, ks = _rows(k, "k", (B, H, K), dt, dev)
    vp, vs = _rows(v, "v", (B, H, V), dt, dev)
    wp = None
    if conv_w is not None:
        if conv_w.numel() != 4 * C or not conv_w.is_contiguous():
            raise ValueError(f"conv_w must be contiguous with 4*{C} elements")
        wp = _at(conv_w, "conv_w", conv_w.shape, _f32, dev)
    o = v.new_empty((B, H, V)) if out is None else out
    ws, n = _scratch(workspace, step_workspace_size(B, H) if workspace is None else 0, dev,
                     "kda_step_workspace_size", 1 << 40)
    st = _lib_now().kda_step(
        _shape_ref(B, 1, H, K, V, DTYPES[dt]), qp, kp, vp, qs, ks, vs,
        _at(g, "g", (B, H, K), _f32, dev), _at(beta, "beta", (B, H), _f32, dev),
        K ** -0.5 if scale is None else scale, wp,
        _at(conv_state, "conv_state", (n_slots, 3, C), dt, dev), 1 if l2norm_qk else 0,
        _at(slots, "slots", (B,), _i32, dev), n_slots,
        _at(state, "state", (n_slots, H, K, V), _f32, dev), _at(o, "out", (B, H, V), dt, dev),
        ws.data_ptr(), n, _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_step")
    return o


def _ssm_dims(xbc, A, head_dim, state_dim):
    H, P, N = A.numel(), head_dim, state_dim
    C = xbc.shape[-1]
    groups, rest = divmod(C - H * P, 2 * N)
    if rest or groups < 1:
        raise ValueError(f"xbc has {C} channels, expected {H}*{P} + 2*G*{N}")
    return H, P, N, groups, C


def ssm_workspace_size(B, T, H, P, N, G, dtype=torch.bfloat16, impl="auto") -> int:
    """Workspace bytes of :func:`ssm_fwd` (0 when the shape is not served)."""
    s = kda_ssm_shape(int(B), int(T), int(H), int(P), int(N), int(G), DTYPES[dtype])
    return int(lib().kda_ssm_fwd_workspace_size(s, IMPLS[impl]))


def alloc_ssm_workspace(B, T, H, P, N, G, dtype=torch.bfloat16, impl="auto",
                        device=None) -> torch.Tensor:
    """Workspace of :func:`ssm_fwd`, its header zero-filled."""
    return _scratch(None, ssm_workspace_size(B, T, H, P, N, G, dtype, impl), device or "cuda",
                    "kda_ssm_fwd_workspace_size", 256)[0]


def _tokens(t, name, shape, dtype, device):
    """Address and strides of a [B,T,width] tensor with contiguous channels."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device):
        _refuse(t, name, shape, dtype, device, False)
    st = t.stride()
    if st[2] != 1 and shape[2] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # the stride of a dimension of 1 means nothing
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0


def ssm_fwd(xbc, dt, conv_w, A, *, head_dim, state_dim, conv_bias=None, dt_bias=None, D=None,
            z=None, initial_state=None, conv_state=None, segment_ids=None,
            output_final_state=False, out=None, workspace=None, impl="auto", stream=None):
    """The selective state space operator on prompts (see include/kda.h).

    xbc: [B,T,H*P+2*G*N], z: [B,T,H*P] or None, dt: [B,T,H], all of one dtype
    (bf16 or fp32) and possibly slices of one projection (last dimension
    contiguous; xbc and z begin and lie on multiples of 16 bytes unless
    ``impl="simt"``, which serves any place and width); conv_w: [channels,4], conv_bias: [channels], A, D, dt_bias:
    [H], all fp32; initial_state: [B,H,N,P] fp32; conv_state: [B,3,channels].
    ``impl``: "simt" computes in fp32 on the CUDA cores, "tc" on the tensor cores,
    the state as fp32 arithmetic does (1.5e-7 off), y from operands of fewer bits
    (of bf16 inputs 1.8e-3 to 2.2e-3 off, 1.7e-3 of it its own rounding; of fp32
    inputs 2e-7 to 7e-7); "auto" takes "tc" but for long rows of few heads
    and fp32 problems of up to 2^26 products of states and tokens.
    Returns ``(y [B,T,H,P], final_state, conv_state_out)``, the last two None
    unless ``output_final_state``."""
    if stream is not None and _elsewhere(stream):
        with torch.cuda.stream(stream):
            return ssm_fwd(xbc, dt, conv_w, A, head_dim=head_dim, state_dim=state_dim,
                           conv_bias=conv_bias, dt_bias=dt_bias, D=D, z=z,
                           initial_state=initial_state, conv_state=conv_state,
                           segment_ids=segment_ids, output_final_state=output_final_state,
                           out=out, workspace=workspace, impl=impl)
    dev, ty = _start(xbc, "ssm_fwd")
    B, T, _ = xbc.shape
    H, P, N, G, C = _ssm_dims(xbc, A, head_dim, state_dim)
    xp, xb, xt = _tokens(xbc, "xbc", (B, T, C), ty, dev)
    dp, db, dtt = _tokens(dt, "dt", (B, T, H), ty, dev)
    zp, zb, zt = (None, 0, 0) if z is None else _tokens(z, "z", (B, T, H * P), ty, dev)
    y = xbc.new_empty((B, T, H, P)) if out is None else out
    fs = conv = fp = cp = None
    if output_final_state:
        fs = A.new_empty((B, H, N, P))
        conv = xbc.new_empty((B, 3, C))
        fp, cp = fs.data_ptr(), conv.data_ptr()
    s = _ssm_ref(B, T, H, P, N, G, DTYPES[ty], xb, xt, zb, zt, db, dtt)
    L, way, one = _lib_now(), IMPLS[impl], (H,)
    ws, n = _scratch(workspace, L.kda_ssm_fwd_workspace_size(s, way) if workspace is None else 0,
                     dev, "kda_ssm_fwd_workspace_size", 256)
    st = L.kda_ssm_fwd(
        s, xp, dp, zp, _at(conv_w, "conv_w", (C, 4), _f32, dev),
        _at(conv_bias, "conv_bias", (C,), _f32, dev), _at(A, "A", one, _f32, dev),
        _at(D, "D", one, _f32, dev), _at(dt_bias, "dt_bias", one, _f32, dev),
        _at(initial_state, "initial_state", (B, H, N, P), _f32, dev),
        _at(conv_state, "conv_state", (B, 3, C), ty, dev),
        _at(segment_ids, "segment_ids", (B, T), _i32, dev), _at(y, "out", (B, T, H, P), ty, dev),
        fp, cp, ws.data_ptr(), n, way, _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_ssm_fwd")
    return y, fs, conv


def ssm_step(xbc, dt, conv_w, A, state, conv_state, *, head_dim, state_dim, conv_bias=None,
             dt_bias=None, D=None, z=None, slots=None, out=None, workspace=None, stream=None):
    """One token per sequence through the state space operator, on cached
    states: xbc [B,H*P+2*G*N], z [B,H*P] or None, dt [B,H] (any stride between
    the rows); state [n_slots,H,N,P] fp32 and conv_state [n_slots,3,channels]
    are moved on in place; ``slots`` as :func:`step`.  Returns y [B,H,P]."""
    if stream is not None and _elsewhere(stream):
        with torch.cuda.stream(stream):
            return ssm_step(xbc, dt, conv_w, A, state, conv_state, head_dim=head_dim,
                            state_dim=state_dim, conv_bias=conv_bias, dt_bias=dt_bias, D=D, z=z,
                            slots=slots, out=out, workspace=workspace)
    dev, ty = _start(xbc, "ssm_step")
    B = xbc.shape[0]
    H, P, N, G, C = _ssm_dims(xbc, A, head_dim, state_dim)
    n_slots, one = state.shape[0], (H,)
    xp, xs = _rows(xbc, "xbc", (B, C), ty, dev)
    dp, ds = _rows(dt, "dt", (B, H), ty, dev)
    zp, zs = (None, 0) if z is None else _rows(z, "z", (B, H * P), ty, dev)
    y = xbc.new_empty((B, H, P)) if out is None else out
    ws, n = _scratch(workspace, step_workspace_size(B, H) if workspace is None else 0, dev,
                     "kda_step_workspace_size", 1 << 40)
    st = _lib_now().kda_ssm_step(
        _ssm_ref(B, 1, H, P, N, G, DTYPES[ty], xs, 0, zs, 0, ds, 0), xp, dp, zp,
        _at(conv_w, "conv_w", (C, 4), _f32, dev), _at(conv_bias, "conv_bias", (C,), _f32, dev),
        _at(A, "A", one, _f32, dev), _at(D, "D", one, _f32, dev),
        _at(dt_bias, "dt_bias", one, _f32, dev), _at(slots, "slots", (B,), _i32, dev), n_slots,
        _at(conv_state, "conv_state", (n_slots, 3, C), ty, dev),
        _at(state, "state", (n_slots, H, N, P), _f32, dev), _at(y, "out", (B, H, P), ty, dev),
        ws.data_ptr(), n, _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_ssm_step")
    return y


GATE_ACTS = {"none": 0, "sigmoid": 1, "silu": 2, "tanh": 3}


def _norm_desc(y, gate, gate_act, scale, eps):
    D, n = y.shape[-1], y.numel()
    if n == 0:
        raise ValueError("y must not be empty")
    rows, grows = n // D, 0
    if gate is not None:
        grows = gate.numel() // D
        if gate.shape[-1] != D or grows == 0 or rows % grows:
            raise ValueError(
                f"gate {tuple(gate.shape)} does not divide the rows of {tuple(y.shape)}")
        if grows != rows and gate.dim() == y.dim():
            # [1, T, D] beside [B, T, D] would serve other rows than broadcasting does
            g, n = gate.shape[:-1], y.shape[:-1]
            k = next(i for i in range(len(n)) if g[i] != n[i])
            if g[k] == 1 and any(v != 1 for v in g[k:]):
                raise ValueError(f"gate {tuple(gate.shape)} does not serve consecutive rows of "
                                 f"{tuple(y.shape)}")
    act = GATE_ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}, got {gate_act!r}")
    return _norm_ref(rows, D, DTYPES[y.dtype], act, grows, scale, eps), rows, (D,)


def block_norm(y, w_post, *, residual=None, gate=None, gate_act="sigmoid", scale=1.0, w_pre=None,
               eps=1e-6, save_stats=False, out=None, stream=None):
    """The norm after a block, its gate and residual scale, and the norm
    before the next block: ``out = residual + scale * act(gate) * rms(y) *
    w_post``, ``x = rms(out) * w_pre``.

    y, residual: [..., D] (bf16 or fp32, contiguous); gate: [..., D] with as
    many rows as y, or fewer that divide them (each then serves as many
    consecutive rows: [B, 1, D] beside [B, T, D], not [1, T, D]); w_post, w_pre: [D] fp32.  residual, gate and w_pre may be
    None.  ``out`` may be the residual itself, but not with ``save_stats``:
    block_norm_bwd reads the residual.  Returns ``(out, x or None)``, and the
    statistics block_norm_bwd reads when ``save_stats``."""
    if stream is not None and _elsewhere(stream):
        with torch.cuda.stream(stream):
            return block_norm(y, w_post, residual=residual, gate=gate, gate_act=gate_act,
                              scale=scale, w_pre=w_pre, eps=eps, save_stats=save_stats, out=out)
    dev, ty = _start(y, "block_norm")
    shape = y.shape
    d, rows, width = _norm_desc(y, gate, gate_act, scale, eps)
    yp = _at(y, "y", shape, ty, dev)
    if out is None:
        out = torch.empty_like(y)
    x = stats = xp = sp = None
    if w_pre is not None:
        x = torch.empty_like(y)
        xp = x.data_ptr()
    if save_stats:
        stats = w_post.new_empty((2, rows))
        sp = stats.data_ptr()
    st = _lib_now().kda_block_norm_fwd(
        d, yp, _at(w_post, "w_post", width, _f32, dev),
        _at(residual, "residual", shape, ty, dev),
        None if gate is None else _at(gate, "gate", gate.shape, ty, dev),
        _at(w_pre, "w_pre", width, _f32, dev), _at(out, "out", shape, ty, dev), xp, sp,
        _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_block_norm_fwd")
    return (out, x, stats) if save_stats else (out, x)


def block_norm_workspace_size(rows, D, gate_rows=0) -> int:
    """Workspace bytes of :func:`block_norm_bwd` for either type (gate_rows
    0: no gate)."""
    d = kda_norm_desc(int(rows), int(D), 0, 1, int(gate_rows), 1.0, 0.0)
    return int(lib().kda_block_norm_bwd_workspace_size(d, int(gate_rows > 0)))


def alloc_block_norm_workspace(rows, D, gate_rows=0, device=None) -> torch.Tensor:
    """Workspace of :func:`block_norm_bwd` (needs no initialisation)."""
    return _scratch(None, block_norm_workspace_size(rows, D, gate_rows), device or "cuda",
                    "kda_block_norm_bwd_workspace_size", 0)[0]


def block_norm_bwd(y, w_post, stats, d_out, *, d_x=None, residual=None, gate=None,
                   gate_act="sigmoid", scale=1.0, w_pre=None, eps=1e-6, workspace=None,
                   stream=None):
    """Gradients of block_norm from its inputs and statistics, given the
    gradients of ``out`` and ``x`` (one of them may be None): ``(dy, d_residual,
    d_gate, dw_post, dw_pre)``, None in the place of an input that was None."""
    if stream is not None and _elsewhere(stream):
        with torch.cuda.stream(stream):
            return block_norm_bwd(y, w_post, stats, d_out, d_x=d_x, residual=residual, gate=gate,
                                  gate_act=gate_act, scale=scale, w_pre=w_pre, eps=eps,
                                  workspace=workspace)
    dev, ty = _start(y, "block_norm_bwd")
    shape = y.shape
    d, rows, width = _norm_desc(y, gate, gate_act, scale, eps)
    yp = _at(y, "y", shape, ty, dev)
    dy, dw_post = torch.empty_like(y), torch.empty_like(w_post)
    dres = dgate = dw_pre = rp = gp = gop = wp = None
    if residual is not None:
        dres = torch.empty_like(y)
        rp = dres.data_ptr()
    if gate is not None:
        gp = _at(gate, "gate", gate.shape, ty, dev)
        dgate = torch.empty_like(gate)
        gop = dgate.data_ptr()
    if w_pre is not None:
        dw_pre = torch.empty_like(w_pre)
        wp = dw_pre.data_ptr()
    L = _lib_now()
    ws, n = _scratch(workspace, L.kda_block_norm_bwd_workspace_size(d, int(gate is not None))
                     if workspace is None else 0, dev, "kda_block_norm_bwd_workspace_size", 0)
    st = L.kda_block_norm_bwd(
        d, yp, _at(w_post, "w_post", width, _f32, dev), _at(residual, "residual", shape, ty, dev),
        gp, _at(w_pre, "w_pre", width, _f32, dev), _at(stats, "stats", (2, rows), _f32, dev),
        _at(d_out, "d_out", shape, ty, dev), _at(d_x, "d_x", shape, ty, dev), dy.data_ptr(), rp,
        gop, dw_post.data_ptr(), wp, ws.data_ptr(), n, _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_block_norm_bwd")
    return dy, dres, dgate, dw_post, dw_pre
