"""Python binding of libkda (ctypes).  Argument marshalling only.

Every step of the recurrence runs in the CUDA kernels behind the C ABI in
``include/kda.h``.  PyTorch supplies device memory and the stream; nothing
here computes any part of the method, and there is no CPU fallback: if the
library is missing or a call fails, an exception is raised.

The names follow the C ABI: ``prefill`` / ``prefill_into`` wrap
``kda_prefill`` / ``kda_prefill_ex``, ``decode_step`` wraps
``kda_decode_step``, ``workspace_size`` wraps ``kda_prefill_workspace_size``
(``kda_prefill_workspace_size_tokens`` when given the token count),
``device_status`` wraps ``kda_prefill_device_status`` and ``backward`` /
``backward_into`` / ``backward_workspace_size`` wrap ``kda_backward`` and
``kda_backward_workspace_size``; ``attnres_layer`` wraps the Blocked Attention
Residuals call of ``include/attnres.h``; the ``linrec_*`` functions wrap the
gated linear recurrence of ``include/linrec.h``, and ``beam_select``,
``beam_reorder`` and ``decode_step_parents`` the beam search calls of
``include/beam.h``.  What a layer has around its recurrence: the ``causalconv_*``
functions wrap the short causal convolution of ``include/causalconv.h``, the
``selscan_*`` functions the selective scan of ``include/selscan.h`` and the
``groupnorm_*`` functions the gated group norm of ``include/groupnorm.h``.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_INPUT, ERR_DEVICE_TIMEOUT = 0, 1, 2, 3, 4, 5
ERR_DEVICE_RANGE = 6
BF16, FP32 = 0, 1
KERNEL_AUTO, KERNEL_CHUNK_SIMT, KERNEL_CHUNK_TC, KERNEL_CHUNK_TC_SPLIT = 0, 1, 2, 3
_KERNELS = {"auto": KERNEL_AUTO, "simt": KERNEL_CHUNK_SIMT, "tc": KERNEL_CHUNK_TC,
            "tc_split": KERNEL_CHUNK_TC_SPLIT}
GATE_CHANNEL_F32, GATE_HEAD_F32, GATE_CHANNEL_LOG_BF16 = 0, 1, 2
# gate layout -> (code, dtype, alpha tensor rank)
_GATES = {"channel": (GATE_CHANNEL_F32, torch.float32, 3),
          "head": (GATE_HEAD_F32, torch.float32, 2),
          "log_bf16": (GATE_CHANNEL_LOG_BF16, torch.bfloat16, 3)}

_lib = None


class _ScanRows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "dt", "B", "C", "z")] + \
        [(n, ctypes.c_int64) for n in ("ldx", "lddt", "ldB", "ldC", "ldz")]


class _ScanGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "ddt", "dB", "dC", "dz", "dA", "dD",
                                               "ddt_bias", "dS0")]


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def load(path: str | None = None):
    """Load libkda.so (built by ``gated_delta_rule_45_gb300.build``); raise if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libkda.so not found at {p}: build it with "
                           "`python -m gated_delta_rule_45_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kda_prefill_workspace_size.restype = sz
    lib.kda_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.kda_prefill_workspace_size_tokens.restype = sz
    lib.kda_prefill_workspace_size_tokens.argtypes = [i32, i64, i32, i32, i32, i32]
    prefill_args = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, ctypes.c_int, i32,
                    vp, vp, vp, sz]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = prefill_args + [vp]
    lib.kda_prefill_ex.restype = ctypes.c_int
    lib.kda_prefill_ex.argtypes = prefill_args + [ctypes.c_int, vp]
    lib.kda_prefill_gates.restype = ctypes.c_int
    lib.kda_prefill_gates.argtypes = [vp, vp, vp, vp, ctypes.c_int] + prefill_args[4:] + \
        [ctypes.c_int, vp]
    lib.kda_prefill_noalloc.restype = ctypes.c_int
    lib.kda_prefill_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                        ctypes.c_int, i32, vp, vp, vp]
    lib.kda_prefill_supported.restype = ctypes.c_int
    lib.kda_prefill_supported.argtypes = [ctypes.c_int, i32, i32, i32, ctypes.c_int, i32]
    lib.kda_segment_combine.restype = ctypes.c_int
    lib.kda_segment_combine.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.kda_check_wait_timeout.restype = ctypes.c_int
    lib.kda_check_wait_timeout.argtypes = [vp, sz, ctypes.c_uint64, vp]
    lib.kda_check_scan_timeout.restype = ctypes.c_int
    lib.kda_check_scan_timeout.argtypes = [vp, sz, ctypes.c_uint64, vp]
    lib.kda_prefill_device_status.restype = ctypes.c_int
    lib.kda_prefill_device_status.argtypes = [vp, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_int,
                                    vp, vp]
    lib.kda_decode_step_gates.restype = ctypes.c_int
    lib.kda_decode_step_gates.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, i32, i32, i32,
                                          i32, ctypes.c_int, vp, vp]
    lib.kda_backward_workspace_size.restype = sz
    lib.kda_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.kda_backward.restype = ctypes.c_int
    lib.kda_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                 ctypes.c_int, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_prefill_additive.restype = ctypes.c_int
    lib.kda_prefill_additive.argtypes = prefill_args + [ctypes.c_int, vp]
    lib.kda_decode_step_additive.restype = ctypes.c_int
    lib.kda_decode_step_additive.argtypes = lib.kda_decode_step.argtypes
    lib.kda_backward_gates_workspace_size.restype = sz
    lib.kda_backward_gates_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int]
    lib.kda_backward_gates.restype = ctypes.c_int
    lib.kda_backward_gates.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, vp, i32, i64, i32,
                                       i32, i32, ctypes.c_int, i32, vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, sz, vp]
    lib.attnres_layer.restype = ctypes.c_int
    lib.attnres_layer.argtypes = [vp, i32, vp, vp, vp, vp, vp, ctypes.c_float, i64, i32,
                                  ctypes.c_int, vp, vp]
    lib.linrec_prefill_workspace_size.restype = sz
    lib.linrec_prefill_workspace_size.argtypes = [i32, i64, i32, i32]
    lib.linrec_prefill.restype = ctypes.c_int
    lib.linrec_prefill.argtypes = [vp, vp, ctypes.c_int, vp, vp, i32, i64, i32, i32,
                                   ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, sz, vp]
    lib.linrec_backward_workspace_size.restype = sz
    lib.linrec_backward_workspace_size.argtypes = [i32, i64, i32, i32, ctypes.c_int, i32]
    lib.linrec_backward.restype = ctypes.c_int
    lib.linrec_backward.argtypes = [vp, vp, ctypes.c_int, vp, vp, i32, i64, i32, i32,
                                    ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, sz,
                                    vp]
    lib.linrec_decode_step.restype = ctypes.c_int
    lib.linrec_decode_step.argtypes = [vp, vp, ctypes.c_int, vp, i32, vp, i32, i32, i32,
                                       ctypes.c_int, ctypes.c_int, vp, vp, vp]
    lib.beam_select_workspace_size.restype = sz
    lib.beam_select_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.beam_select.restype = ctypes.c_int
    lib.beam_select.argtypes = [vp, i64, vp, vp, i32, i32, i32, i32, i32, ctypes.c_int, vp, vp,
                                vp, vp, sz, vp]
    lib.beam_reorder.restype = ctypes.c_int
    lib.beam_reorder.argtypes = [vp, i32, vp, i32, i32, vp]
    lib.kda_decode_step_parents.restype = ctypes.c_int
    lib.kda_decode_step_parents.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, i32, vp, vp,
                                            i32, i32, i32, i32, ctypes.c_int, vp, vp]
    flt, rows = ctypes.c_float, ctypes.POINTER(_ScanRows)
    lib.causalconv_prefill_workspace_size.restype = sz
    lib.causalconv_prefill_workspace_size.argtypes = [i32, i64, i32, i32, ctypes.c_int]
    lib.causalconv_prefill.restype = ctypes.c_int
    lib.causalconv_prefill.argtypes = [vp, i64, vp, vp, vp, vp, i32, i64, i32, i32, ctypes.c_int,
                                       ctypes.c_int, vp, vp, vp, sz, vp]
    lib.causalconv_backward_workspace_size.restype = sz
    lib.causalconv_backward_workspace_size.argtypes = [i32, i64, i32, i32]
    lib.causalconv_backward.restype = ctypes.c_int
    lib.causalconv_backward.argtypes = [vp, i64, vp, vp, vp, vp, i32, i64, i32, i32, ctypes.c_int,
                                        ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.causalconv_decode_step.restype = ctypes.c_int
    lib.causalconv_decode_step.argtypes = [vp, i64, vp, vp, vp, i32, vp, i32, i32, i32,
                                           ctypes.c_int, ctypes.c_int, vp, vp, vp]
    lib.selscan_prefill_workspace_size.restype = sz
    lib.selscan_prefill_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    scan_args = [rows, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, ctypes.c_int, ctypes.c_int]
    lib.selscan_prefill.restype = ctypes.c_int
    lib.selscan_prefill.argtypes = scan_args + [vp, vp, vp, vp, sz, vp]
    lib.selscan_backward_workspace_size.restype = sz
    lib.selscan_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.selscan_backward.restype = ctypes.c_int
    lib.selscan_backward.argtypes = scan_args + [vp, vp, vp, ctypes.POINTER(_ScanGrads), vp, sz,
                                                 vp]
    lib.selscan_decode_step.restype = ctypes.c_int
    lib.selscan_decode_step.argtypes = [rows, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                        ctypes.c_int, ctypes.c_int, vp, vp, vp]
    norm_args = [vp, i64, vp, vp, i32, vp, i64, i64, i32, i32, ctypes.c_int, ctypes.c_int,
                 ctypes.c_int, flt]
    lib.groupnorm_forward.restype = ctypes.c_int
    lib.groupnorm_forward.argtypes = norm_args + [vp, vp]
    lib.groupnorm_backward_workspace_size.restype = sz
    lib.groupnorm_backward_workspace_size.argtypes = [i64, i32, i32]
    lib.groupnorm_backward.restype = ctypes.c_int
    lib.groupnorm_backward.argtypes = norm_args + [vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_version.restype = i32
    lib.kda_version.argtypes = []
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"the storage dtype must be bfloat16 or float32, got {t.dtype}")


# Types are checked before placement, for every entry point: the C ABI reads
# alpha, beta, states and gradients as fp32 and cu_seqlens as int32, so a
# tensor of another type would be misread rather than rejected.
def _check_qkv(q, *others):
    """q and the tensors stored like it (k, v, o, dO) share one dtype, bf16 or fp32."""
    _dtype_code(q)
    for t in others:
        if t is not None and t.dtype != q.dtype:
            raise TypeError("q, k, v and the tensors stored like them must share one dtype")


def _check_f32(what: str, *ts):
    for t in ts:
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{what} must be float32")


def _check_int32(cu_seqlens):
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")


def _check_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")


def supported(kernel: str, H: int, d_k: int, d_v: int, dtype: torch.dtype, chunk: int) -> bool:
    """Whether kda_prefill_ex with this kernel choice accepts the shape (host-only query)."""
    code = BF16 if dtype == torch.bfloat16 else FP32
    return load().kda_prefill_supported(_KERNELS[kernel], H, d_k, d_v, code, chunk) == OK


def workspace_size(num_seqs: int, H: int = 1, d_k: int = 128, d_v: int = 128,
                   chunk: int = 64, total_tokens: int | None = None) -> int:
    """Prefill workspace bytes: kda_prefill_workspace_size_tokens when the
    token count is given (room for the sequence-axis split where it applies),
    else kda_prefill_workspace_size (no split)."""
    if total_tokens is None:
        return int(load().kda_prefill_workspace_size(num_seqs, H, d_k, d_v, chunk))
    return int(load().kda_prefill_workspace_size_tokens(num_seqs, total_tokens, H, d_k, d_v,
                                                        chunk))


def prefill_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace, *, chunk: int = 64,
                 kernel: str = "auto", stream=None) -> None:
    """Enqueue kda_prefill_ex on `stream` (default: current stream) into preallocated outputs.

    q, k: [T, H, d_k]; v, o: [T, H, d_v] (bf16 or fp32, all the same); alpha:
    [T, H, d_v] fp32; beta: [T, H] fp32; S0: [N, H, d_v, d_k] fp32 or None;
    cu_seqlens: int32 [N+1] on the device; S_T: [N, H, d_v, d_k] fp32 (may be S0);
    workspace: a uint8 device tensor of at least ``workspace_size(N)`` bytes.
    """
    _check_int32(cu_seqlens)
    _check_f32("alpha, beta and the states", alpha, beta, S0, S_T)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    st = load().kda_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                               _ptr(cu_seqlens), N, T, H, d_k, d_v, dt, chunk, _ptr(o),
                               _ptr(S_T), _ptr(workspace), workspace.numel(), _KERNELS[kernel],
                               _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_prefill")


def prefill_gates_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace, *,
                       gate: str = "channel", chunk: int = 64, kernel: str = "auto",
                       stream=None) -> None:
    """Enqueue kda_prefill_gates: as prefill_into with the forget gate in layout `gate`:
    "channel" alpha [T, H, d_v] fp32, "head" alpha [T, H] fp32 (one gate per head),
    "log_bf16" log alpha [T, H, d_v] bf16."""
    code, adt, arank = _GATES[gate]
    if alpha.dtype != adt or alpha.dim() != arank:
        raise TypeError(f"gate layout {gate!r} wants a rank-{arank} {adt} tensor")
    _check_int32(cu_seqlens)
    _check_f32("beta and the states", beta, S0, S_T)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    st = load().kda_prefill_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), code, _ptr(beta),
                                  _ptr(S0), _ptr(cu_seqlens), N, T, H, d_k, d_v, dt, chunk,
                                  _ptr(o), _ptr(S_T), _ptr(workspace), workspace.numel(),
                                  _KERNELS[kernel], _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_prefill_gates")


def prefill_gates(q, k, v, alpha, beta, S0, cu_seqlens, *, gate: str = "channel",
                  chunk: int = 64, kernel: str = "auto", stream=None,
                  check_device_status: bool = False):
    """Allocate outputs with PyTorch and run kda_prefill_gates; returns (o, S_T)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    o = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    S_T = torch.empty((N, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws = torch.empty(workspace_size(N, H, d_k, d_v, chunk, T), dtype=torch.uint8,
                     device=q.device)
    prefill_gates_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, ws, gate=gate, chunk=chunk,
                       kernel=kernel, stream=stream)
    if check_device_status:
        device_status(ws, stream=stream)
    return o, S_T


def prefill(q, k, v, alpha, beta, S0, cu_seqlens, *, chunk: int = 64, kernel: str = "auto",
            stream=None, check_device_status: bool = False):
    """Allocate outputs with PyTorch and run kda_prefill; returns (o, S_T)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    o = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    S_T = torch.empty((N, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws = torch.empty(workspace_size(N, H, d_k, d_v, chunk, T), dtype=torch.uint8,
                     device=q.device)
    prefill_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, ws, chunk=chunk, kernel=kernel,
                 stream=stream)
    if check_device_status:
        device_status(ws, stream=stream)
    return o, S_T


NOALLOC_MAX_SEQS = 65536


def prefill_noalloc_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, *, chunk: int = 64,
                         stream=None) -> None:
    """Enqueue kda_prefill_noalloc: like ``prefill_into`` but the scratch lives in
    the library (for callers that cannot allocate).  Calls must not overlap on
    the GPU; at most NOALLOC_MAX_SEQS sequences."""
    _check_int32(cu_seqlens)
    _check_f32("alpha, beta and the states", alpha, beta, S0, S_T)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    if N > NOALLOC_MAX_SEQS:
        raise ValueError(f"kda_prefill_noalloc takes at most {NOALLOC_MAX_SEQS} sequences, "
                         f"got {N}")
    st = load().kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                    _ptr(S0), _ptr(cu_seqlens), N, T, H, d_k, d_v,
                                    _dtype_code(q), chunk, _ptr(o), _ptr(S_T),
                                    _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_prefill_noalloc")


def segment_combine(S_in, g, P, R, S_out=None, *, stream=None):
    """Enqueue kda_segment_combine: S_out = diag(g) S_in P + R per (sequence, head);
    S_in, R [N, H, d_v, d_k], g [N, H, d_v], P [N, H, d_k, d_k], fp32.  Returns S_out."""
    _check_f32("segment maps", S_in, g, P, R)
    _check_cuda(S_in, g, P, R)
    N, H, d_v, d_k = S_in.shape
    if S_out is None:
        S_out = torch.empty_like(S_in)
    st = load().kda_segment_combine(_ptr(S_in), _ptr(g), _ptr(P), _ptr(R), N, H, d_k, d_v,
                                    _ptr(S_out), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_segment_combine")
    return S_out


def check_wait_timeout(workspace, timeout_ns: int, *, stream=None) -> None:
    """Enqueue kda_check_wait_timeout: the prefill's device-side timeout path
    run on purpose; afterwards the workspace's status reads
    ERR_DEVICE_TIMEOUT."""
    _check_cuda(workspace)
    st = load().kda_check_wait_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                       int(timeout_ns), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_check_wait_timeout")


def check_scan_timeout(workspace, timeout_ns: int, *, stream=None) -> None:
    """Enqueue kda_check_scan_timeout: the same for the time-axis scan of the ``linrec_*``
    calls; workspace: at least SCAN_CHECK_BYTES bytes, overwritten."""
    _check_cuda(workspace)
    st = load().kda_check_scan_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                       int(timeout_ns), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_check_scan_timeout")


def device_status(workspace, stream=None) -> None:
    """Synchronise `stream` and raise KdaError if the device rejected the last prefill's input."""
    st = load().kda_prefill_device_status(_ptr(workspace), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_prefill (device check)")


def decode_step(q, k, v, alpha, beta, S, o=None, *, stream=None):
    """Enqueue kda_decode_step: S [B, H, d_v, d_k] fp32 updated in place; returns o [B, H, d_v]."""
    B, H, d_k = q.shape
    d_v = v.shape[2]
    if o is None:
        o = torch.empty((B, H, d_v), dtype=q.dtype, device=q.device)
    _check_f32("S, alpha and beta", S, alpha, beta)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S, o)
    dt = _dtype_code(q)
    st = load().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                B, H, d_k, d_v, dt, _ptr(o), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_decode_step")
    return o


def decode_step_gates(q, k, v, alpha, beta, S, o=None, *, gate: str = "channel", stream=None):
    """kda_decode_step_gates: decode_step with the forget gate in layout `gate`
    ("channel" alpha [B, H, d_v] fp32, "head" alpha [B, H] fp32, "log_bf16" log
    alpha [B, H, d_v] bf16); S updated in place; returns o [B, H, d_v]."""
    code, adt, arank = _GATES[gate]
    B, H, d_k = q.shape
    d_v = v.shape[2]
    if o is None:
        o = torch.empty((B, H, d_v), dtype=q.dtype, device=q.device)
    if alpha.dtype != adt or alpha.dim() != arank:
        raise TypeError(f"gate layout {gate!r} wants a rank-{arank} {adt} tensor")
    _check_f32("S and beta", S, beta)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S, o)
    dt = _dtype_code(q)
    st = load().kda_decode_step_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), code, _ptr(beta),
                                      _ptr(S), B, H, d_k, d_v, dt, _ptr(o), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_decode_step_gates")
    return o


def prefill_additive_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace, *,
                          chunk: int = 64, kernel: str = "auto", stream=None) -> None:
    """Enqueue kda_prefill_additive into preallocated outputs (as prefill_into)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    _check_int32(cu_seqlens)
    _check_f32("alpha, beta and the states", alpha, beta, S0, S_T)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, workspace)
    st = load().kda_prefill_additive(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                     _ptr(S0), _ptr(cu_seqlens), N, T, H, d_k, d_v,
                                     _dtype_code(q), chunk, _ptr(o), _ptr(S_T), _ptr(workspace),
                                     workspace.numel(), _KERNELS[kernel], _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_prefill_additive")


def prefill_additive(q, k, v, alpha, beta, S0, cu_seqlens, *, chunk: int = 64,
                     kernel: str = "auto", stream=None, check_device_status: bool = False):
    """kda_prefill_additive: the additive update of linear attention (no predict
    step; naive linear attention when alpha = beta = 1).  Returns (o, S_T)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    o = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    S_T = torch.empty((N, H, d_v, d_k), dtype=torch.float32, device=q.device)
    ws = torch.empty(workspace_size(N, H, d_k, d_v, chunk, T), dtype=torch.uint8,
                     device=q.device)
    prefill_additive_into(q, k, v, alpha, beta, S0, cu_seqlens, o, S_T, ws, chunk=chunk,
                          kernel=kernel, stream=stream)
    if check_device_status:
        device_status(ws, stream=stream)
    return o, S_T


def decode_step_additive(q, k, v, alpha, beta, S, o=None, *, stream=None):
    """kda_decode_step_additive: one step of the additive update, S in place; returns o."""
    B, H, d_k = q.shape
    d_v = v.shape[2]
    if o is None:
        o = torch.empty((B, H, d_v), dtype=q.dtype, device=q.device)
    _check_f32("S, alpha and beta", S, alpha, beta)
    _check_qkv(q, k, v, o)
    _check_cuda(q, k, v, alpha, beta, S, o)
    st = load().kda_decode_step_additive(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                         _ptr(S), B, H, d_k, d_v, _dtype_code(q), _ptr(o),
                                         _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_decode_step_additive")
    return o


def backward_workspace_size(num_seqs: int, total_tokens: int, H: int, d_k: int = 128,
                            d_v: int = 128, chunk: int = 64) -> int:
    """kda_backward_workspace_size: bytes of workspace (0: shape not supported)."""
    return int(load().kda_backward_workspace_size(num_seqs, total_tokens, H, d_k, d_v, chunk))


def backward_into(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T, grads, workspace, *,
                  chunk: int = 64, stream=None) -> None:
    """Enqueue kda_backward into preallocated fp32 gradients.

    Inputs as ``prefill_into`` (bf16 q, k, v); dO: [T, H, d_v] bf16; dS_T:
    [N, H, d_v, d_k] fp32 or None; grads: dict with "dq", "dk" [T, H, d_k],
    "dv", "dalpha" [T, H, d_v], "dbeta" [T, H] and optionally "dS0"
    [N, H, d_v, d_k], all fp32; workspace: uint8 device tensor of at least
    ``backward_workspace_size`` bytes.
    """
    dS0 = grads.get("dS0")
    _check_int32(cu_seqlens)
    _check_qkv(q, k, v, dO)
    _check_f32("alpha, beta, states and gradients", alpha, beta, S0, dS_T, grads["dq"],
               grads["dk"], grads["dv"], grads["dalpha"], grads["dbeta"], dS0)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T, grads["dq"], grads["dk"],
                grads["dv"], grads["dalpha"], grads["dbeta"], dS0, workspace)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    st = load().kda_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                             _ptr(cu_seqlens), N, T, H, d_k, d_v, _dtype_code(q), chunk,
                             _ptr(dO), _ptr(dS_T), _ptr(grads["dq"]), _ptr(grads["dk"]),
                             _ptr(grads["dv"]), _ptr(grads["dalpha"]), _ptr(grads["dbeta"]),
                             _ptr(dS0), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_backward")


def backward(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T=None, *, chunk: int = 64,
             stream=None, check_device_status: bool = False):
    """Allocate fp32 gradients with PyTorch and run kda_backward; returns a dict
    with dq, dk, dv, dalpha, dbeta and dS0 (tokens past cu_seqlens[-1] zero)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dev = q.device
    grads = {"dq": torch.zeros((T, H, d_k), dtype=torch.float32, device=dev),
             "dk": torch.zeros((T, H, d_k), dtype=torch.float32, device=dev),
             "dv": torch.zeros((T, H, d_v), dtype=torch.float32, device=dev),
             "dalpha": torch.zeros((T, H, d_v), dtype=torch.float32, device=dev),
             "dbeta": torch.zeros((T, H), dtype=torch.float32, device=dev),
             "dS0": torch.zeros((N, H, d_v, d_k), dtype=torch.float32, device=dev)}
    nbytes = backward_workspace_size(N, T, H, d_k, d_v, chunk)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "kda_backward")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    backward_into(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T, grads, ws, chunk=chunk,
                  stream=stream)
    if check_device_status:
        device_status(ws, stream=stream)
    return grads


def backward_gates(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T=None, *, gate: str = "channel",
                   chunk: int = 64, stream=None, check_device_status: bool = False):
    """kda_backward_gates: ``backward`` with the forget gate in layout `gate`
    ("channel", "head" [T, H] fp32, "log_bf16" log alpha [T, H, d_v] bf16).
    Returns the gradients; "dgate" is the gradient with respect to the gate in
    its own layout ([T, H] for "head", d/d log alpha for "log_bf16")."""
    code, adt, arank = _GATES[gate]
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    if alpha.dtype != adt or alpha.dim() != arank:
        raise TypeError(f"gate layout {gate!r} wants a rank-{arank} {adt} tensor")
    _check_int32(cu_seqlens)
    _check_f32("beta and the states", beta, S0, dS_T)
    _check_qkv(q, k, v, dO)
    _check_cuda(q, k, v, alpha, beta, S0, cu_seqlens, dO, dS_T)
    dev = q.device
    gshape = (T, H) if gate == "head" else (T, H, d_v)
    grads = {"dq": torch.zeros((T, H, d_k), dtype=torch.float32, device=dev),
             "dk": torch.zeros((T, H, d_k), dtype=torch.float32, device=dev),
             "dv": torch.zeros((T, H, d_v), dtype=torch.float32, device=dev),
             "dgate": torch.zeros(gshape, dtype=torch.float32, device=dev),
             "dbeta": torch.zeros((T, H), dtype=torch.float32, device=dev),
             "dS0": torch.zeros((N, H, d_v, d_k), dtype=torch.float32, device=dev)}
    lib = load()
    nbytes = int(lib.kda_backward_gates_workspace_size(N, T, H, d_k, d_v, chunk, code))
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "kda_backward_gates")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib.kda_backward_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), code, _ptr(beta),
                                _ptr(S0), _ptr(cu_seqlens), N, T, H, d_k, d_v, _dtype_code(q),
                                chunk, _ptr(dO), _ptr(dS_T), _ptr(grads["dq"]), _ptr(grads["dk"]),
                                _ptr(grads["dv"]), _ptr(grads["dgate"]), _ptr(grads["dbeta"]),
                                _ptr(grads["dS0"]), _ptr(ws), ws.numel(), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "kda_backward_gates")
    if check_device_status:
        device_status(ws, stream=stream)
    return grads


def attnres_layer(blocks, q, *, partial=None, h_last=None, partial_out=None, block_out=None,
                  scale=None, h=None, stream=None):
    """Enqueue attnres_layer: one layer's input under Blocked Attention Residuals.

    blocks: [nb, T, d] (bf16 or fp32; nb may be 0 when partial or h_last is
    given); q: [d] fp32; partial: [T, d] fp32 or None; h_last: [T, d] like
    blocks or None; partial_out: [T, d] fp32 or None (may be partial);
    block_out: [T, d] like blocks or None; scale: default 1/sqrt(d).
    Returns h [T, d] (allocated when not given)."""
    nb, T, d = blocks.shape
    if h is None:
        h = torch.empty((T, d), dtype=blocks.dtype, device=blocks.device)
    _dtype_code(blocks)
    _check_f32("q", q)
    _check_f32("the running sum", partial, partial_out)
    for t in (h_last, block_out, h):
        if t is not None and t.dtype != blocks.dtype:
            raise TypeError("h_last, block_out and h share the dtype of blocks")
    _check_cuda(blocks, q, partial, h_last, partial_out, block_out, h)
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    st = load().attnres_layer(_ptr(blocks) if nb > 0 else None, nb, _ptr(partial), _ptr(h_last),
                              _ptr(partial_out), _ptr(block_out), _ptr(q), float(scale), T, d,
                              _dtype_code(blocks), _ptr(h), _stream_ptr(stream))
    if st != OK:
        raise KdaError(st, "attnres_layer")
    return h


# ---- gated linear recurrence (include/linrec.h) and beam search (include/beam.h)

_DTYPE_CODES = {torch.bfloat16: BF16, torch.float32: FP32}
LINREC_CHUNK = 128
SCAN_CHECK_BYTES = 16384
BEAM_MAX_BEAMS, BEAM_MAX_SELECT = 32, 64


class _BeamState(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


def _check(what: str, t, dtype, shape) -> None:
    """One tensor argument: its type (TypeError), then its shape (ValueError)."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _place(stream, *ts) -> int:
    """Raw stream to launch on; every tensor must be contiguous on the current device."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or dev < 0 or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors on one device")
    return _stream_on(dev, stream)


def _stream_on(dev: int, stream) -> int:
    """Raw handle of `stream`, or of the current one, which must be the current device's.
    (The small calls are bound by this module: torch.cuda.current_stream() alone would
    take as long as the launch.)"""
    if dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current CUDA device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("the stream must belong to the current CUDA device")
    return stream.cuda_stream


def _empty(stream, shape, dtype, device):
    """torch.empty for work on `stream`: the caching allocator hands a block that is freed
    again only to later work of the stream it was allocated on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _p(t):
    return None if t is None else t.data_ptr()


def _linrec_args(x, a, gate: str, rows: str):
    """(H, d, dtype code, gate code) of x [rows, H, d] and its gate."""
    code = _DTYPE_CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"the storage dtype must be bfloat16 or float32, got {x.dtype}")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be [{rows}, H, d], got {tuple(shape)}")
    gcode, adt, arank = _GATES[gate]
    _check("the gate", a, adt, shape[:arank])
    return shape[1], shape[2], code, gcode


def linrec_workspace_size(num_seqs: int, total_tokens: int, H: int, d: int) -> int:
    """linrec_prefill_workspace_size: bytes of workspace (0: size not supported)."""
    return load().linrec_prefill_workspace_size(num_seqs, total_tokens, H, d)


def _linrec_inputs(x, a, S0, cu_seqlens, gate: str):
    """Checked sizes (T, N, H, d, dtype code, gate code) of a packed batch."""
    H, d, code, gcode = _linrec_args(x, a, gate, "T")
    N = cu_seqlens.numel() - 1
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,))
    if S0 is not None:
        _check("S0", S0, torch.float32, (N, H, d))
    return x.shape[0], N, H, d, code, gcode


def linrec_prefill_into(x, a, S0, cu_seqlens, y, S_T, workspace, *, states=None,
                        gate: str = "channel", complement: bool = False, stream=None) -> None:
    """Enqueue linrec_prefill into preallocated outputs: h_t = a_t h_{t-1} + u_t per
    channel, u = x or, with `complement`, (1 - a) x.

    x, y: [T, H, d] (bf16 or fp32); a: the forget gate in layout `gate` as for
    ``prefill_gates_into`` ("channel" [T, H, d] fp32, "head" [T, H] fp32,
    "log_bf16" log a [T, H, d] bf16); S0: [N, H, d] fp32 or None; cu_seqlens:
    int32 [N+1] on the device; S_T: [N, H, d] fp32 (may be S0); states:
    [ceil(T / LINREC_CHUNK), H, d] fp32 or None, kept for ``linrec_backward``;
    workspace: uint8, at least ``linrec_workspace_size`` bytes.
    """
    T, N, H, d, code, gcode = _linrec_inputs(x, a, S0, cu_seqlens, gate)
    _check("y", y, x.dtype, x.shape)
    _check("S_T", S_T, torch.float32, (N, H, d))
    if states is not None:
        _check("states", states, torch.float32, (-(-T // LINREC_CHUNK), H, d))
    raw = _place(stream, x, a, S0, cu_seqlens, y, S_T, states, workspace)
    st = load().linrec_prefill(_p(x), _p(a), gcode, _p(S0), _p(cu_seqlens), N, T, H, d, code,
                               int(complement), _p(y), _p(S_T), _p(states), _p(workspace),
                               workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "linrec_prefill")


def linrec_prefill(x, a, S0, cu_seqlens, *, gate: str = "channel", complement: bool = False,
                   save_states: bool = False, stream=None, check_device_status: bool = False):
    """Allocate outputs with PyTorch and run linrec_prefill; returns (y, S_T), or with
    `save_states` (y, S_T, states) for ``linrec_backward``.  y of tokens past
    cu_seqlens[-1] is not written."""
    T, N, H, d, code, gcode = _linrec_inputs(x, a, S0, cu_seqlens, gate)
    raw = _place(stream, x, a, S0, cu_seqlens)
    lib, dev = load(), x.device
    nbytes = lib.linrec_prefill_workspace_size(N, T, H, d)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "linrec_prefill")
    y = _empty(stream, x.shape, x.dtype, dev)
    S_T = _empty(stream, (N, H, d), torch.float32, dev)
    states = _empty(stream, (-(-T // LINREC_CHUNK), H, d), torch.float32, dev) \
        if save_states else None
    ws = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.linrec_prefill(x.data_ptr(), a.data_ptr(), gcode, _p(S0), cu_seqlens.data_ptr(), N,
                            T, H, d, code, int(complement), y.data_ptr(), S_T.data_ptr(),
                            _p(states), ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "linrec_prefill")
    if check_device_status:
        device_status(ws, stream=stream)
    return (y, S_T, states) if save_states else (y, S_T)


def linrec_backward_workspace_size(num_seqs: int, total_tokens: int, H: int, d: int, *,
                                   gate: str = "channel", with_states: bool = True) -> int:
    """linrec_backward_workspace_size: bytes of workspace (0: size not supported)."""
    return load().linrec_backward_workspace_size(num_seqs, total_tokens, H, d, _GATES[gate][0],
                                                 int(with_states))


def _check_cotangents(x, dy, dS_T, states, T, N, H, d):
    _check("dy", dy, x.dtype, x.shape)
    if dS_T is not None:
        _check("dS_T", dS_T, torch.float32, (N, H, d))
    if states is not None:
        _check("states", states, torch.float32, (-(-T // LINREC_CHUNK), H, d))


def linrec_backward_into(x, a, S0, cu_seqlens, dy, dS_T, grads, workspace, *, states=None,
                         gate: str = "channel", complement: bool = False, stream=None) -> None:
    """Enqueue linrec_backward into preallocated fp32 gradients.

    Inputs as ``linrec_prefill_into``; dy: like x; dS_T: [N, H, d] fp32 or None;
    states: what linrec_prefill saved, or None (the forward scan runs again);
    grads: dict with "dx" [T, H, d], "dgate" (shaped like the gate; with respect
    to log a for "log_bf16") and optionally "dS0" [N, H, d]; workspace: uint8, at
    least ``linrec_backward_workspace_size`` bytes.
    """
    T, N, H, d, code, gcode = _linrec_inputs(x, a, S0, cu_seqlens, gate)
    dx, dgate, dS0 = grads["dx"], grads["dgate"], grads.get("dS0")
    _check_cotangents(x, dy, dS_T, states, T, N, H, d)
    if dS0 is not None:
        _check("dS0", dS0, torch.float32, (N, H, d))
    _check("dx", dx, torch.float32, x.shape)
    _check("dgate", dgate, torch.float32, a.shape)
    raw = _place(stream, x, a, S0, cu_seqlens, dy, dS_T, states, dx, dgate, dS0, workspace)
    st = load().linrec_backward(_p(x), _p(a), gcode, _p(S0), _p(cu_seqlens), N, T, H, d, code,
                                int(complement), _p(dy), _p(dS_T), _p(states), _p(dx),
                                _p(dgate), _p(dS0), _p(workspace),
                                workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "linrec_backward")


def linrec_backward(x, a, S0, cu_seqlens, dy, dS_T=None, *, states=None, gate: str = "channel",
                    complement: bool = False, stream=None, check_device_status: bool = False):
    """Allocate fp32 gradients with PyTorch and run linrec_backward; returns a dict with
    dx, dgate and dS0.  Rows of tokens past cu_seqlens[-1] are not written."""
    T, N, H, d, code, gcode = _linrec_inputs(x, a, S0, cu_seqlens, gate)
    _check_cotangents(x, dy, dS_T, states, T, N, H, d)
    raw = _place(stream, x, a, S0, cu_seqlens, dy, dS_T, states)
    lib, dev = load(), x.device
    nbytes = lib.linrec_backward_workspace_size(N, T, H, d, gcode, int(states is not None))
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "linrec_backward")
    grads = {"dx": _empty(stream, x.shape, torch.float32, dev),
             "dgate": _empty(stream, a.shape, torch.float32, dev),
             "dS0": _empty(stream, (N, H, d), torch.float32, dev)}
    ws = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.linrec_backward(x.data_ptr(), a.data_ptr(), gcode, _p(S0), cu_seqlens.data_ptr(), N,
                             T, H, d, code, int(complement), dy.data_ptr(), _p(dS_T), _p(states),
                             grads["dx"].data_ptr(), grads["dgate"].data_ptr(),
                             grads["dS0"].data_ptr(), ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "linrec_backward")
    if check_device_status:
        device_status(ws, stream=stream)
    return grads


def linrec_decode_step(x, a, S, y=None, *, parents=None, S_out=None, gate: str = "channel",
                       complement: bool = False, stream=None):
    """Enqueue linrec_decode_step: one token for each of B sequences; returns y [B, H, d].

    x: [B, H, d]; a: as for ``linrec_prefill_into`` with B in T's place; S: fp32
    [B, H, d], updated in place unless S_out is given.  parents: int32 [B] or None:
    sequence b continues row parents[b] of S [rows, H, d] (a zero state for an entry
    outside it) and S_out [B, H, d] must be given."""
    H, d, code, gcode = _linrec_args(x, a, gate, "B")
    B = x.shape[0]
    if parents is None:
        _check("S", S, torch.float32, (B, H, d))
    else:
        _check("parents", parents, torch.int32, (B,))
        _check("S", S, torch.float32, (S.shape[0], H, d))
        if S_out is None:
            raise ValueError("parents need S_out: the states cannot move in place")
    if S_out is None:
        S_out = S
    else:
        _check("S_out", S_out, torch.float32, (B, H, d))
    raw = _place(stream, x, a, S, parents, S_out, y)
    if y is None:
        y = _empty(stream, x.shape, x.dtype, x.device)
    else:
        _check("y", y, x.dtype, x.shape)
    st = load().linrec_decode_step(_p(x), _p(a), gcode, _p(S), S.shape[0], _p(parents), B, H, d,
                                   code, int(complement), _p(y), _p(S_out), raw)
    if st != OK:
        raise KdaError(st, "linrec_decode_step")
    return y


def decode_step_parents(q, k, v, alpha, beta, S_in, parents, S_out, o=None, *,
                        gate: str = "channel", stream=None):
    """Enqueue kda_decode_step_parents: ``decode_step_gates`` with sequence b's state read
    from row parents[b] of S_in [rows, H, d_v, d_k] (a zero state for an entry outside it)
    and written to row b of S_out [B, H, d_v, d_k]; returns o [B, H, d_v]."""
    B, H, d_k = q.shape
    d_v = v.shape[2]
    code = _DTYPE_CODES.get(q.dtype)
    if code is None:
        raise TypeError(f"the storage dtype must be bfloat16 or float32, got {q.dtype}")
    gcode, adt, arank = _GATES[gate]
    _check("k", k, q.dtype, q.shape)
    _check("v", v, q.dtype, (B, H, d_v))
    _check(f"alpha (layout {gate!r})", alpha, adt, v.shape[:arank])
    _check("beta", beta, torch.float32, (B, H))
    _check("S_in", S_in, torch.float32, (S_in.shape[0], H, d_v, d_k))
    _check("S_out", S_out, torch.float32, (B, H, d_v, d_k))
    _check("parents", parents, torch.int32, (B,))
    raw = _place(stream, q, k, v, alpha, beta, S_in, parents, S_out, o)
    if o is None:
        o = _empty(stream, v.shape, v.dtype, v.device)
    else:
        _check("o", o, q.dtype, v.shape)
    st = load().kda_decode_step_parents(_p(q), _p(k), _p(v), _p(alpha), gcode, _p(beta),
                                        _p(S_in), S_in.shape[0], _p(parents), _p(S_out), B, H,
                                        d_k, d_v, code, _p(o), raw)
    if st != OK:
        raise KdaError(st, "kda_decode_step_parents")
    return o


def beam_select(logits, scores, num_out: int, *, finished=None, eos: int = 0, out=None,
                workspace=None, stream=None):
    """Enqueue beam_select: the num_out best continuations of each request over its beams
    and the vocabulary; returns (scores fp32, parents int32, tokens int32), each
    [B, num_out], best first.  parents are rows of `logits`.

    logits: [B K, V] (bf16 or fp32; rows may be strided: a padded vocabulary); scores:
    [B, K] fp32; finished: uint8 or bool [B, K] or None: a finished beam's one candidate
    is token `eos` at its score; out: the three outputs to write to; workspace: uint8, at
    least ``beam_select_workspace_size`` bytes (allocated when not given)."""
    code = _DTYPE_CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"the storage dtype must be bfloat16 or float32, got {logits.dtype}")
    if scores.dim() != 2 or logits.dim() != 2:
        raise ValueError("logits must be [B K, V] and scores [B, K]")
    B, K = scores.shape
    V = logits.shape[1]
    _check("scores", scores, torch.float32, (B, K))
    if logits.shape[0] != B * K:
        raise ValueError(f"logits must have {B * K} rows, got {tuple(logits.shape)}")
    if finished is not None:
        if finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
        _check("finished", finished, torch.uint8, (B, K))
    ld = logits.stride(0) if B * K > 1 else V
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("each row of logits must be contiguous")
    lib, dev = load(), scores.device
    nbytes = lib.beam_select_workspace_size(B, K, V, num_out)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED if 1 <= num_out <= K * V else ERR_INVALID_ARG,
                       "beam_select")
    if logits.get_device() != scores.get_device():
        raise ValueError("all tensors must be CUDA tensors on one device")
    raw = _place(stream, scores, finished, workspace, *(out or ()))
    if out is None:
        out = (_empty(stream, (B, num_out), torch.float32, dev),
               _empty(stream, (B, num_out), torch.int32, dev),
               _empty(stream, (B, num_out), torch.int32, dev))
    else:
        for what, t, dt in zip(("out scores", "out parents", "out tokens"), out,
                               (torch.float32, torch.int32, torch.int32)):
            _check(what, t, dt, (B, num_out))
    if workspace is None:
        workspace = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.beam_select(_p(logits), ld, _p(scores), _p(finished), B, K, V, num_out, eos, code,
                         _p(out[0]), _p(out[1]), _p(out[2]), _p(workspace),
                         workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "beam_select")
    return out


def beam_select_workspace_size(B: int, K: int, V: int, num_out: int) -> int:
    """beam_select_workspace_size: bytes of workspace (0: size not supported)."""
    return load().beam_select_workspace_size(B, K, V, num_out)


def beam_reorder(states, parents, beams: int, *, stream=None) -> None:
    """Enqueue beam_reorder: row i of each tensor becomes its old row parents[i], in place.

    states: tensors whose first axis is the B x beams rows (any type, contiguous);
    parents: int32, B x beams entries, each a row of the same request (an entry that is
    not leaves its row as it is)."""
    if parents.dtype != torch.int32:
        raise TypeError("parents must be int32")
    rows = parents.numel()
    if beams < 1 or rows % beams:
        raise ValueError(f"parents must have a multiple of {beams} entries, got {rows}")
    descr = (_BeamState * len(states))()
    for s, t in zip(descr, states):
        if t.dim() < 1 or t.shape[0] != rows:
            raise ValueError(f"every state must have {rows} rows, got {tuple(t.shape)}")
        s.data = t.data_ptr()
        s.row_bytes = t.numel() * t.element_size() // rows if rows else 0
    raw = _place(stream, parents, *states)
    st = load().beam_reorder(ctypes.byref(descr), len(states), _p(parents), rows // beams, beams,
                             raw)
    if st != OK:
        raise KdaError(st, "beam_reorder")


# ---- around a layer's recurrence: the short causal convolution (include/causalconv.h), the
# ---- selective scan (include/selscan.h) and the gated group norm (include/groupnorm.h)

SELSCAN_CHUNK = 16
_ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}


def _storage(x) -> int:
    code = _DTYPE_CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"the storage dtype must be bfloat16 or float32, got {x.dtype}")
    return code


def _row_stride(what: str, t) -> int:
    """Distance in elements between the rows of t, each of which must be dense."""
    if t.is_contiguous():
        return t.numel() // t.shape[0] if t.shape[0] else _width(t)
    width = 1
    for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and step != width:
            raise ValueError(f"each row of {what} must be contiguous")
        width *= size
    if t.shape[0] < 2:
        return width
    if t.stride(0) < width:
        raise ValueError(f"the rows of {what} must not overlap")
    return t.stride(0)


def _width(t) -> int:
    n = 1
    for size in t.shape[1:]:
        n *= size
    return n


def _place_rows(stream, rows, *ts) -> int:
    """``_place`` for `ts`; `rows` may be strided but must be on the same device."""
    dev = rows[0].get_device()
    for t in rows:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError("all tensors must be CUDA tensors on one device")
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors on one device")
    return _stream_on(dev, stream)


def _conv_args(x, w, b):
    """(channels' shape, D, W, dtype code) of x [rows, ...] and its filter."""
    code = _storage(x)
    ch = x.shape[1:]
    if x.dim() < 2 or w.dim() != x.dim():
        raise ValueError(f"x must be [T, ...] and w [..., W], got {tuple(x.shape)} and "
                         f"{tuple(w.shape)}")
    W = w.shape[-1]
    _check("w", w, torch.float32, (*ch, W))
    if b is not None:
        _check("b", b, torch.float32, ch)
    return ch, _width(x), W, code


def _conv_inputs(x, w, b, S0, cu_seqlens):
    ch, D, W, code = _conv_args(x, w, b)
    N = cu_seqlens.numel() - 1
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,))
    if S0 is not None:
        _check("S0", S0, x.dtype, (N, W - 1, *ch))
    return ch, D, W, code, N


def causalconv_workspace_size(num_seqs: int, total_tokens: int, D: int, W: int,
                              dtype=torch.bfloat16) -> int:
    """causalconv_prefill_workspace_size: bytes of workspace (0: size not supported)."""
    return load().causalconv_prefill_workspace_size(num_seqs, total_tokens, D, W,
                                                    _DTYPE_CODES[dtype])


def causalconv_prefill_into(x, w, b, S0, cu_seqlens, y, S_T, workspace, *, silu: bool = True,
                            stream=None) -> None:
    """Enqueue causalconv_prefill into preallocated outputs: the depthwise filter over each
    channel's last W inputs, then silu.

    x: [T, ...] (bf16 or fp32; any channel shape; rows may be strided: a slice of a wider
    projection); w: [..., W] fp32, the token itself last, 2 <= W <= 4; b: [...] fp32 or None;
    S0: [N, W-1, ...] like x or None, the inputs before each sequence; cu_seqlens: int32
    [N+1] on the device; y: like x; S_T: like S0 (may be S0); workspace: uint8, at least
    ``causalconv_workspace_size`` bytes."""
    ch, D, W, code, N = _conv_inputs(x, w, b, S0, cu_seqlens)
    _check("y", y, x.dtype, x.shape)
    _check("S_T", S_T, x.dtype, (N, W - 1, *ch))
    ld = _row_stride("x", x)
    raw = _place_rows(stream, (x,), w, b, S0, cu_seqlens, y, S_T, workspace)
    st = load().causalconv_prefill(_p(x), ld, _p(w), _p(b), _p(S0), _p(cu_seqlens), N, x.shape[0],
                                   D, W, code, int(silu), _p(y), _p(S_T), _p(workspace),
                                   workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "causalconv_prefill")


def causalconv_prefill(x, w, b, S0, cu_seqlens, *, silu: bool = True, stream=None,
                       check_device_status: bool = False):
    """Allocate outputs with PyTorch and run causalconv_prefill; returns (y, S_T).  y of
    tokens past cu_seqlens[-1] is not written."""
    ch, D, W, code, N = _conv_inputs(x, w, b, S0, cu_seqlens)
    ld = _row_stride("x", x)
    raw = _place_rows(stream, (x,), w, b, S0, cu_seqlens)
    lib, dev, T = load(), x.device, x.shape[0]
    nbytes = lib.causalconv_prefill_workspace_size(N, T, D, W, code)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "causalconv_prefill")
    y = _empty(stream, x.shape, x.dtype, dev)
    S_T = _empty(stream, (N, W - 1, *ch), x.dtype, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.causalconv_prefill(x.data_ptr(), ld, w.data_ptr(), _p(b), _p(S0),
                                cu_seqlens.data_ptr(), N, T, D, W, code, int(silu), y.data_ptr(),
                                S_T.data_ptr(), ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "causalconv_prefill")
    if check_device_status:
        device_status(ws, stream=stream)
    return y, S_T


def causalconv_backward_workspace_size(num_seqs: int, total_tokens: int, D: int, W: int) -> int:
    """causalconv_backward_workspace_size: bytes of workspace (0: size not supported)."""
    return load().causalconv_backward_workspace_size(num_seqs, total_tokens, D, W)


def _conv_cotangents(x, dy, dS_T, N, W, ch):
    _check("dy", dy, x.dtype, x.shape)
    if dS_T is not None:
        _check("dS_T", dS_T, torch.float32, (N, W - 1, *ch))


def causalconv_backward_into(x, w, b, S0, cu_seqlens, dy, dS_T, grads, workspace, *,
                             silu: bool = True, stream=None) -> None:
    """Enqueue causalconv_backward into preallocated fp32 gradients.

    Inputs as ``causalconv_prefill_into``; dy: like x; dS_T: [N, W-1, ...] fp32 or None;
    grads: dict with "dx" [T, ...], "dw" [..., W] and optionally "db" [...] and "dS0"
    [N, W-1, ...]; workspace: uint8, at least ``causalconv_backward_workspace_size`` bytes."""
    ch, D, W, code, N = _conv_inputs(x, w, b, S0, cu_seqlens)
    dx, dw, db, dS0 = grads["dx"], grads["dw"], grads.get("db"), grads.get("dS0")
    _conv_cotangents(x, dy, dS_T, N, W, ch)
    _check("dx", dx, torch.float32, x.shape)
    _check("dw", dw, torch.float32, w.shape)
    if db is not None:
        _check("db", db, torch.float32, ch)
    if dS0 is not None:
        _check("dS0", dS0, torch.float32, (N, W - 1, *ch))
    ld = _row_stride("x", x)
    raw = _place_rows(stream, (x,), w, b, S0, cu_seqlens, dy, dS_T, dx, dw, db, dS0, workspace)
    st = load().causalconv_backward(_p(x), ld, _p(w), _p(b), _p(S0), _p(cu_seqlens), N,
                                    x.shape[0], D, W, code, int(silu), _p(dy), _p(dS_T), _p(dx),
                                    _p(dw), _p(db), _p(dS0), _p(workspace),
                                    workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "causalconv_backward")


def causalconv_backward(x, w, b, S0, cu_seqlens, dy, dS_T=None, *, silu: bool = True, stream=None,
                        check_device_status: bool = False):
    """Allocate fp32 gradients with PyTorch and run causalconv_backward; returns a dict with
    dx, dw, dS0 and, with a bias, db.  Rows of tokens past cu_seqlens[-1] are not written."""
    ch, D, W, code, N = _conv_inputs(x, w, b, S0, cu_seqlens)
    _conv_cotangents(x, dy, dS_T, N, W, ch)
    ld = _row_stride("x", x)
    raw = _place_rows(stream, (x,), w, b, S0, cu_seqlens, dy, dS_T)
    lib, dev, T = load(), x.device, x.shape[0]
    nbytes = lib.causalconv_backward_workspace_size(N, T, D, W)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "causalconv_backward")
    grads = {"dx": _empty(stream, x.shape, torch.float32, dev),
             "dw": _empty(stream, w.shape, torch.float32, dev),
             "dS0": _empty(stream, (N, W - 1, *ch), torch.float32, dev)}
    if b is not None:
        grads["db"] = _empty(stream, ch, torch.float32, dev)
    ws = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.causalconv_backward(x.data_ptr(), ld, w.data_ptr(), _p(b), _p(S0),
                                 cu_seqlens.data_ptr(), N, T, D, W, code, int(silu),
                                 dy.data_ptr(), _p(dS_T), grads["dx"].data_ptr(),
                                 grads["dw"].data_ptr(), _p(grads.get("db")),
                                 grads["dS0"].data_ptr(), ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "causalconv_backward")
    if check_device_status:
        device_status(ws, stream=stream)
    return grads


def causalconv_decode_step(x, w, b, S, y=None, *, parents=None, S_out=None, silu: bool = True,
                           stream=None):
    """Enqueue causalconv_decode_step: one token for each of B sequences; returns y [B, ...].

    x: [B, ...] (rows may be strided); w, b: as for ``causalconv_prefill_into``; S: like x
    [B, W-1, ...], the inputs before, moved on in place unless S_out is given.  parents:
    int32 [B] or None: sequence b continues row parents[b] of S [rows, W-1, ...] (zeros for an
    entry outside it) and S_out [B, W-1, ...] must be given."""
    ch, D, W, code = _conv_args(x, w, b)
    B = x.shape[0]
    if parents is None:
        _check("S", S, x.dtype, (B, W - 1, *ch))
    else:
        _check("parents", parents, torch.int32, (B,))
        _check("S", S, x.dtype, (S.shape[0], W - 1, *ch))
        if S_out is None:
            raise ValueError("parents need S_out: the states cannot move in place")
    if S_out is None:
        S_out = S
    else:
        _check("S_out", S_out, x.dtype, (B, W - 1, *ch))
    ld = _row_stride("x", x)
    raw = _place_rows(stream, (x,), w, b, S, parents, S_out, y)
    if y is None:
        y = _empty(stream, x.shape, x.dtype, x.device)
    else:
        _check("y", y, x.dtype, x.shape)
    st = load().causalconv_decode_step(x.data_ptr(), ld, w.data_ptr(), _p(b), S.data_ptr(),
                                       S.shape[0], _p(parents), B, D, W, code, int(silu),
                                       y.data_ptr(), S_out.data_ptr(), raw)
    if st != OK:
        raise KdaError(st, "causalconv_decode_step")
    return y


def _scan_args(x, dt, A, B, C, D, z, dt_bias, rows: str):
    """(H, d, n, dtype code, row descriptor) of the scan's inputs."""
    code = _storage(x)
    if x.dim() != 3 or A.dim() != 3:
        raise ValueError(f"x must be [{rows}, H, d] and A [H, d, n], got {tuple(x.shape)} and "
                         f"{tuple(A.shape)}")
    T, H, d = x.shape
    n = A.shape[2]
    _check("A", A, torch.float32, (H, d, n))
    _check("dt", dt, x.dtype, x.shape)
    _check("B", B, x.dtype, (T, H, n))
    _check("C", C, x.dtype, (T, H, n))
    if z is not None:
        _check("z", z, x.dtype, x.shape)
    if D is not None:
        _check("D", D, torch.float32, (H, d))
    if dt_bias is not None:
        _check("dt_bias", dt_bias, torch.float32, (H, d))
    r = _ScanRows(_p(x), _p(dt), _p(B), _p(C), _p(z), _row_stride("x", x), _row_stride("dt", dt),
                  _row_stride("B", B), _row_stride("C", C),
                  0 if z is None else _row_stride("z", z))
    return H, d, n, code, r


def _scan_inputs(x, dt, A, B, C, S0, cu_seqlens, D, z, dt_bias):
    H, d, n, code, r = _scan_args(x, dt, A, B, C, D, z, dt_bias, "T")
    N = cu_seqlens.numel() - 1
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,))
    if S0 is not None:
        _check("S0", S0, torch.float32, (N, H, d, n))
    return x.shape[0], N, H, d, n, code, r


def selscan_workspace_size(num_seqs: int, total_tokens: int, H: int, d: int, n: int) -> int:
    """selscan_prefill_workspace_size on the current device: bytes of workspace (0: size not
    supported)."""
    return load().selscan_prefill_workspace_size(num_seqs, total_tokens, H, d, n)


def _scan_chunks(T: int) -> int:
    return -(-T // SELSCAN_CHUNK)


def selscan_prefill_into(x, dt, A, B, C, S0, cu_seqlens, y, S_T, workspace, *, D=None, z=None,
                         dt_bias=None, softplus: bool = True, states=None, stream=None) -> None:
    """Enqueue selscan_prefill into preallocated outputs: h_t = exp(step_t A) h_{t-1} + step_t
    x_t B_t per channel over n values, y_t = (C_t . h_t + D x_t) silu(z_t), step = softplus(dt
    + dt_bias) (without `softplus` dt + dt_bias).

    x, dt, z: [T, H, d] (bf16 or fp32; z may be None); B, C: [T, H, n] like x, one for the d
    channels of a group; all five may have strided rows (slices of a wider projection); A:
    [H, d, n] fp32; D, dt_bias: [H, d] fp32 or None; S0: [N, H, d, n] fp32 or None; cu_seqlens:
    int32 [N+1] on the device; y: like x; S_T: like S0 (may be S0); states: [ceil(T /
    SELSCAN_CHUNK), H, d, n] fp32 or None, kept for ``selscan_backward``; workspace: uint8, at
    least ``selscan_workspace_size`` bytes.  One sequence far longer than many others of its
    batch is done sooner by a call of its own."""
    T, N, H, d, n, code, r = _scan_inputs(x, dt, A, B, C, S0, cu_seqlens, D, z, dt_bias)
    _check("y", y, x.dtype, x.shape)
    _check("S_T", S_T, torch.float32, (N, H, d, n))
    if states is not None:
        _check("states", states, torch.float32, (_scan_chunks(T), H, d, n))
    raw = _place_rows(stream, (x, dt, B, C, z), A, D, dt_bias, S0, cu_seqlens, y, S_T, states,
                      workspace)
    st = load().selscan_prefill(ctypes.byref(r), _p(A), _p(D), _p(dt_bias), _p(S0),
                                _p(cu_seqlens), N, T, H, d, n, code, int(softplus), _p(y),
                                _p(S_T), _p(states), _p(workspace),
                                workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "selscan_prefill")


def selscan_prefill(x, dt, A, B, C, S0, cu_seqlens, *, D=None, z=None, dt_bias=None,
                    softplus: bool = True, save_states: bool = False, stream=None,
                    check_device_status: bool = False):
    """Allocate outputs with PyTorch and run selscan_prefill; returns (y, S_T), or with
    `save_states` (y, S_T, states) for ``selscan_backward``.  y of tokens past cu_seqlens[-1]
    is not written."""
    T, N, H, d, n, code, r = _scan_inputs(x, dt, A, B, C, S0, cu_seqlens, D, z, dt_bias)
    raw = _place_rows(stream, (x, dt, B, C, z), A, D, dt_bias, S0, cu_seqlens)
    lib, dev = load(), x.device
    nbytes = lib.selscan_prefill_workspace_size(N, T, H, d, n)
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "selscan_prefill")
    y = _empty(stream, x.shape, x.dtype, dev)
    S_T = _empty(stream, (N, H, d, n), torch.float32, dev)
    states = _empty(stream, (_scan_chunks(T), H, d, n), torch.float32, dev) if save_states \
        else None
    ws = _empty(stream, nbytes, torch.uint8, dev)
    st = lib.selscan_prefill(ctypes.byref(r), A.data_ptr(), _p(D), _p(dt_bias), _p(S0),
                             cu_seqlens.data_ptr(), N, T, H, d, n, code, int(softplus),
                             y.data_ptr(), S_T.data_ptr(), _p(states), ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "selscan_prefill")
    if check_device_status:
        device_status(ws, stream=stream)
    return (y, S_T, states) if save_states else (y, S_T)


def selscan_backward_workspace_size(num_seqs: int, total_tokens: int, H: int, d: int, n: int, *,
                                    with_states: bool = True) -> int:
    """selscan_backward_workspace_size on the current device: bytes of workspace (0: size not
    supported)."""
    return load().selscan_backward_workspace_size(num_seqs, total_tokens, H, d, n,
                                                  int(with_states))


def _scan_cotangents(x, dy, dS_T, states, T, N, H, d, n):
    _check("dy", dy, x.dtype, x.shape)
    if dS_T is not None:
        _check("dS_T", dS_T, torch.float32, (N, H, d, n))
    if states is not None:
        _check("states", states, torch.float32, (_scan_chunks(T), H, d, n))


def _scan_grad_shapes(T, N, H, d, n, z, D, dt_bias):
    shapes = {"dx": (T, H, d), "ddt": (T, H, d), "dB": (T, H, n), "dC": (T, H, n),
              "dA": (H, d, n), "dS0": (N, H, d, n)}
    if z is not None:
        shapes["dz"] = (T, H, d)
    if D is not None:
        shapes["dD"] = (H, d)
    if dt_bias is not None:
        shapes["ddt_bias"] = (H, d)
    return shapes


def selscan_backward_into(x, dt, A, B, C, S0, cu_seqlens, dy, dS_T, grads, workspace, *, D=None,
                          z=None, dt_bias=None, softplus: bool = True, states=None,
                          stream=None) -> None:
    """Enqueue selscan_backward into preallocated fp32 gradients.

    Inputs as ``selscan_prefill_into``; dy: like x (the fp32 dx of an operator behind is cast
    for bf16, as for the other backward passes); dS_T: [N, H, d, n] fp32 or None; states:
    what selscan_prefill saved, or None (the forward scan runs again); grads: dict with "dx",
    "ddt" [T, H, d], "dB", "dC" [T, H, n], "dA" [H, d, n], with a gate "dz" [T, H, d], and
    optionally "dD", "ddt_bias" [H, d] and "dS0" [N, H, d, n]; workspace: uint8, at least
    ``selscan_backward_workspace_size`` bytes."""
    T, N, H, d, n, code, r = _scan_inputs(x, dt, A, B, C, S0, cu_seqlens, D, z, dt_bias)
    _scan_cotangents(x, dy, dS_T, states, T, N, H, d, n)
    shapes = _scan_grad_shapes(T, N, H, d, n, True, True, True)
    for name in ("dx", "ddt", "dB", "dC", "dA") + (("dz",) if z is not None else ()):
        _check(name, grads[name], torch.float32, shapes[name])
    for name in ("dD", "ddt_bias", "dS0"):
        if grads.get(name) is not None:
            _check(name, grads[name], torch.float32, shapes[name])
    outs = [grads.get(f) if f != "dz" or z is not None else None for f, _ in _ScanGrads._fields_]
    raw = _place_rows(stream, (x, dt, B, C, z), A, D, dt_bias, S0, cu_seqlens, dy, dS_T, states,
                      workspace, *outs)
    g = _ScanGrads(*(_p(t) for t in outs))
    st = load().selscan_backward(ctypes.byref(r), _p(A), _p(D), _p(dt_bias), _p(S0),
                                 _p(cu_seqlens), N, T, H, d, n, code, int(softplus), _p(dy),
                                 _p(dS_T), _p(states), ctypes.byref(g), _p(workspace),
                                 workspace.numel() * workspace.element_size(), raw)
    if st != OK:
        raise KdaError(st, "selscan_backward")


def selscan_backward(x, dt, A, B, C, S0, cu_seqlens, dy, dS_T=None, *, D=None, z=None,
                     dt_bias=None, softplus: bool = True, states=None, stream=None,
                     check_device_status: bool = False):
    """Allocate fp32 gradients with PyTorch and run selscan_backward; returns a dict with dx,
    ddt, dB, dC, dA, dS0 and, for each that is given, dz, dD and ddt_bias.  Rows of tokens past
    cu_seqlens[-1] are not written."""
    T, N, H, d, n, code, r = _scan_inputs(x, dt, A, B, C, S0, cu_seqlens, D, z, dt_bias)
    _scan_cotangents(x, dy, dS_T, states, T, N, H, d, n)
    raw = _place_rows(stream, (x, dt, B, C, z), A, D, dt_bias, S0, cu_seqlens, dy, dS_T, states)
    lib, dev = load(), x.device
    nbytes = lib.selscan_backward_workspace_size(N, T, H, d, n, int(states is not None))
    if nbytes == 0:
        raise KdaError(ERR_UNSUPPORTED, "selscan_backward")
    grads = {name: _empty(stream, shape, torch.float32, dev)
             for name, shape in _scan_grad_shapes(T, N, H, d, n, z, D, dt_bias).items()}
    ws = _empty(stream, nbytes, torch.uint8, dev)
    g = _ScanGrads(*(_p(grads.get(f)) for f, _ in _ScanGrads._fields_))
    st = lib.selscan_backward(ctypes.byref(r), A.data_ptr(), _p(D), _p(dt_bias), _p(S0),
                              cu_seqlens.data_ptr(), N, T, H, d, n, code, int(softplus),
                              dy.data_ptr(), _p(dS_T), _p(states), ctypes.byref(g),
                              ws.data_ptr(), nbytes, raw)
    if st != OK:
        raise KdaError(st, "selscan_backward")
    if check_device_status:
        device_status(ws, stream=stream)
    return grads


def selscan_decode_step(x, dt, A, B, C, S, y=None, *, D=None, z=None, dt_bias=None,
                        softplus: bool = True, parents=None, S_out=None, stream=None):
    """Enqueue selscan_decode_step: one token for each of R sequences; returns y [R, H, d].

    Inputs as ``selscan_prefill_into`` with R in T's place; S: fp32 [R, H, d, n], updated in
    place unless S_out is given.  parents: int32 [R] or None: sequence b continues row
    parents[b] of S [rows, H, d, n] (a zero state for an entry outside it) and S_out [R, H, d,
    n] must be given."""
    H, d, n, code, r = _scan_args(x, dt, A, B, C, D, z, dt_bias, "R")
    R = x.shape[0]
    if parents is None:
        _check("S", S, torch.float32, (R, H, d, n))
    else:
        _check("parents", parents, torch.int32, (R,))
        _check("S", S, torch.float32, (S.shape[0], H, d, n))
        if S_out is None:
            raise ValueError("parents need S_out: the states cannot move in place")
    if S_out is None:
        S_out = S
    else:
        _check("S_out", S_out, torch.float32, (R, H, d, n))
    raw = _place_rows(stream, (x, dt, B, C, z), A, D, dt_bias, S, parents, S_out, y)
    if y is None:
        y = _empty(stream, x.shape, x.dtype, x.device)
    else:
        _check("y", y, x.dtype, x.shape)
    st = load().selscan_decode_step(ctypes.byref(r), A.data_ptr(), _p(D), _p(dt_bias),
                                    S.data_ptr(), S.shape[0], _p(parents), R, H, d, n, code,
                                    int(softplus), y.data_ptr(), S_out.data_ptr(), raw)
    if st != OK:
        raise KdaError(st, "selscan_decode_step")
    return y


def _norm_args(x, w, b, z, act: str):
    """(T, H, d, heads of the parameters, dtype code, activation) of the norm's inputs."""
    code = _storage(x)
    if x.dim() != 3:
        raise ValueError(f"x must be [T, H, d], got {tuple(x.shape)}")
    T, H, d = x.shape
    if act not in _ACTIVATIONS:
        raise ValueError(f"the activation must be one of {sorted(_ACTIVATIONS)}, got {act!r}")
    heads = 1
    for what, t in (("w", w), ("b", b)):
        if t is None:
            continue
        if t.dim() not in (1, 2):
            raise ValueError(f"{what} must be [d] or [H, d], got {tuple(t.shape)}")
        _check(what, t, torch.float32, (H, d) if t.dim() == 2 else (d,))
    if w is not None and b is not None and w.dim() != b.dim():
        raise ValueError("w and b must have one shape")
    for t in (w, b):
        if t is not None and t.dim() == 2:
            heads = H
    if z is not None:
        _check("z", z, x.dtype, x.shape)
    return T, H, d, heads, code, _ACTIVATIONS[act]


def groupnorm_forward(x, w=None, b=None, y=None, *, z=None, act: str = "silu", eps: float = 1e-5,
                      center: bool = False, stream=None):
    """Enqueue groupnorm_forward: the norm of each head's d channels, then its gate; returns y.

    x: [T, H, d] (bf16 or fp32); w, b: [d] or [H, d] fp32 or None; z: the gate like x or None;
    rows of x and z may be strided.  y = v act(z) with a gate and act(v) without, v = w (x - m)
    / sqrt(mean((x - m)^2) + eps) + b, m the mean with `center` and else 0; act "silu",
    "sigmoid" or "none".  y: like x, allocated when not given (may be x, or z)."""
    T, H, d, heads, code, acode = _norm_args(x, w, b, z, act)
    ldx, ldz = _row_stride("x", x), 0 if z is None else _row_stride("z", z)
    raw = _place_rows(stream, (x, z), w, b, y)
    if y is None:
        y = _empty(stream, x.shape, x.dtype, x.device)
    else:
        _check("y", y, x.dtype, x.shape)
    st = load().groupnorm_forward(x.data_ptr(), ldx, _p(w), _p(b), heads, _p(z), ldz, T, H, d,
                                  code, int(center), acode, eps, y.data_ptr(), raw)
    if st != OK:
        raise KdaError(st, "groupnorm_forward")
    return y


def groupnorm_backward_workspace_size(T: int, H: int, d: int) -> int:
    """groupnorm_backward_workspace_size: bytes of workspace (0: size not supported)."""
    return load().groupnorm_backward_workspace_size(T, H, d)


def groupnorm_backward_into(x, w, b, dy, grads, workspace, *, z=None, act: str = "silu",
                            eps: float = 1e-5, center: bool = False, stream=None) -> None:
    """Enqueue groupnorm_backward into preallocated fp32 gradients.

    Inputs as ``groupnorm_forward``; dy: like x; grads: dict with "dx" [T, H, d] and optionally
    "dz" (with a gate), "dw" and "db" ([d], or [H, d] when w or b are); workspace: uint8, at
    least ``groupnorm_backward_workspace_size`` bytes (may be None without dw and db)."""
    T, H, d, heads, code, acode = _norm_args(x, w, b, z, act)
    _check("dy", dy, x.dtype, x.shape)
    dx, dz, dw, db = grads["dx"], grads.get("dz"), grads.get("dw"), grads.get("db")
    _check("dx", dx, torch.float32, x.shape)
    if dz is not None:
        _check("dz", dz, torch.float32, x.shape)
    for what, t in (("dw", dw), ("db", db)):
        if t is not None:
            _check(what, t, torch.float32, (H, d) if heads > 1 else (d,) if t.dim() == 1 else (1, d))
    ldx, ldz = _row_stride("x", x), 0 if z is None else _row_stride("z", z)
    raw = _place_rows(stream, (x, z), w, b, dy, dx, dz, dw, db, workspace)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().groupnorm_backward(_p(x), ldx, _p(w), _p(b), heads, _p(z), ldz, T, H, d, code,
                                   int(center), acode, eps, _p(dy), _p(dx), _p(dz), _p(dw),
                                   _p(db), _p(workspace), nbytes, raw)
    if st != OK:
        raise KdaError(st, "groupnorm_backward")


def groupnorm_backward(x, w, b, dy, *, z=None, act: str = "silu", eps: float = 1e-5,
                       center: bool = False, stream=None):
    """Allocate fp32 gradients with PyTorch and run groupnorm_backward; returns a dict with dx
    and, for each that is given, dz, dw and db."""
    T, H, d, heads, code, acode = _norm_args(x, w, b, z, act)
    _check("dy", dy, x.dtype, x.shape)
    ldx, ldz = _row_stride("x", x), 0 if z is None else _row_stride("z", z)
    raw = _place_rows(stream, (x, z), w, b, dy)
    lib, dev = load(), x.device
    grads = {"dx": _empty(stream, x.shape, torch.float32, dev)}
    if z is not None:
        grads["dz"] = _empty(stream, x.shape, torch.float32, dev)
    ws, nbytes = None, 0
    if w is not None or b is not None:
        nbytes = lib.groupnorm_backward_workspace_size(T, H, d)
        if nbytes == 0:
            raise KdaError(ERR_UNSUPPORTED, "groupnorm_backward")
        ws = _empty(stream, nbytes, torch.uint8, dev)
        if w is not None:
            grads["dw"] = _empty(stream, w.shape, torch.float32, dev)
        if b is not None:
            grads["db"] = _empty(stream, b.shape, torch.float32, dev)
    st = lib.groupnorm_backward(_p(x), ldx, _p(w), _p(b), heads, _p(z), ldz, T, H, d, code,
                                int(center), acode, eps, _p(dy), _p(grads["dx"]),
                                _p(grads.get("dz")), _p(grads.get("dw")), _p(grads.get("db")),
                                _p(ws), nbytes, raw)
    if st != OK:
        raise KdaError(st, "groupnorm_backward")
    return grads
