"""Thin Python binding of the C ABI in ``include/kla.h`` (ctypes; the mixer
operators through the CPython extension ``_mixer``).

Argument marshalling only: every step of the filter runs in the CUDA kernels
of ``libkla.so``.  PyTorch is used for device memory and streams.  There is no
CPU fallback: without the built library, or without a CUDA device, every call
raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libkla.so")

KLA_F32 = 0
KLA_BF16 = 1
STATUS = {0: "KLA_OK", 1: "KLA_ERR_INVALID_ARG", 2: "KLA_ERR_UNSUPPORTED_DTYPE",
          3: "KLA_ERR_WORKSPACE_TOO_SMALL", 4: "KLA_ERR_CUDA", 5: "KLA_ERR_TIMEOUT",
          6: "KLA_ERR_MISALIGNED", 7: "KLA_ERR_TOO_LARGE"}
KLA_OK, KLA_ERR_INVALID_ARG, KLA_ERR_UNSUPPORTED_DTYPE = 0, 1, 2
KLA_ERR_WORKSPACE_TOO_SMALL, KLA_ERR_CUDA, KLA_ERR_TIMEOUT, KLA_ERR_MISALIGNED = 3, 4, 5, 6
KLA_ERR_TOO_LARGE = 7
KLA_GATE_CHANNEL, KLA_GATE_HEAD = 0, 1
STATIC_SCRATCH_BYTES = 32 << 20  # KLA_STATIC_SCRATCH_BYTES

# Every exported symbol of include/kla.h, with (restype, argtypes).
_VP, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "kla_abi_version": (ctypes.c_int, []),
    "kla_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "kla_scan_forward_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int,
                                                       ctypes.POINTER(_SZ)]),
    "kla_scan_forward": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                        _VP, _I64, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_scan_step": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP,
                                     _I64, _I64, _I64, _VP]),
    "kla_get_error": (ctypes.c_int, [_VP]),
    "kla_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "kla_debug_unset_flag_wait": (ctypes.c_int, [_VP]),
    "kla_forward_chunk_tokens": (ctypes.c_int, []),
    "kla_debug_stall_chunk": (ctypes.c_int, [_I64]),
    "kla_debug_force_forward_kernel": (ctypes.c_int, [ctypes.c_int]),
    "kla_scan_forward_plan": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP, _VP,
                                             ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "kla_scan_forward_static": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP,
                                               _VP, _VP, _I64, _I64, _I64, _I64, _VP]),
    "kla_scan_forward_host_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, _I64,
                                                            ctypes.POINTER(_SZ)]),
    "kla_scan_forward_host": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP,
                                             _I64, _I64, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_scan_backward_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int,
                                                        ctypes.POINTER(_SZ)]),
    "kla_scan_backward": (ctypes.c_int, [_VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                         _VP, _VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_scan_backward_plan": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP,
                                              ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "kla_debug_force_backward_kernel": (ctypes.c_int, [ctypes.c_int]),
    "kla_layer_forward_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, _I64, ctypes.c_int,
                                                        ctypes.POINTER(_SZ)]),
    "kla_layer_forward": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                         _VP, _I64, _I64, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_layer_step": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP,
                                      _I64, _I64, _I64, _I64, _VP]),
    "kla_attention_weights": (ctypes.c_int, [_VP, _VP, ctypes.c_int, _VP, _VP, _I64, _I64, _I64, _I64,
                                             _I64, _I64, _I64, _VP]),
    "kla_scan_forward_lti_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int,
                                                           ctypes.POINTER(_SZ)]),
    "kla_scan_forward_lti": (ctypes.c_int, [_VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP,
                                            _I64, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_scan_forward_lti_plan": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP,
                                                 ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "kla_gated_scan_forward": (ctypes.c_int, [_VP, _VP, ctypes.c_int, ctypes.c_int, _VP, _VP, _I64, _I64, _I64,
                                              _I64, _VP]),
    "kla_gated_scan_plan": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _VP]),
    "kla_gated_scan_step": (ctypes.c_int, [_VP, _VP, ctypes.c_int, ctypes.c_int, _VP, _VP, _I64, _I64, _I64, _VP]),
    "kla_gated_scan_backward_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int,
                                                              ctypes.POINTER(_SZ)]),
    "kla_gated_scan_backward": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP, _I64,
                                               _I64, _I64, _I64, _VP, _SZ, _VP]),
    "kla_rotary_forward": (ctypes.c_int, [_VP, _VP, ctypes.c_int, _VP, _I64, ctypes.c_int, ctypes.c_float,
                                          ctypes.c_int, _VP, _I64, _I64, _VP, _I64, _I64, _I64, _I64, _VP]),
    "kla_qk_norm_rotary_forward": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, ctypes.c_float, _VP,
                                                  _I64, ctypes.c_int, ctypes.c_float, _VP, _I64, _I64, _VP, _VP,
                                                  _I64, _I64, _I64, _I64, _I64, _VP]),
    "kla_qk_norm_rotary_backward_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    "kla_qk_norm_rotary_backward": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, ctypes.c_float, _VP,
                                                   _I64, ctypes.c_int, ctypes.c_float, _VP, _I64, _I64, _VP, _VP,
                                                   _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _I64, _VP, _SZ,
                                                   _VP]),
}
ATTENTION_MAX_WINDOW = 64  # KLA_ATTENTION_MAX_WINDOW
ROTARY_MAX_D = 1024  # KLA_ROTARY_MAX_D

_lib: Optional[ctypes.CDLL] = None


class KlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


def load_library(path: str = LIBRARY) -> ctypes.CDLL:
    """Load ``libkla.so`` and declare the C signatures (raises if it is missing)."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; build it with "
            "`python -m kalman_linear_attention_b200._build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def _check(status: int, what: str) -> None:
    if status != KLA_OK:
        raise KlaError(status, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KLA_F32
    if t.dtype == torch.bfloat16:
        return KLA_BF16
    raise TypeError(f"inputs must be float32 or bfloat16, got {t.dtype}")


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _require_cuda(*ts: torch.Tensor) -> None:
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensor must be on a CUDA device")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensor must be contiguous")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def workspace_size(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_scan_forward_workspace_size(B, T, H, N, code, ctypes.byref(out)),
           "kla_scan_forward_workspace_size")
    return int(out.value)


def forward_plan(a: torch.Tensor, p: torch.Tensor, phi: torch.Tensor, b: torch.Tensor) -> Tuple[int, int]:
    """(kernel, launches) that scan_forward would use for these inputs:
    kernel 1 = chunked (workspace carries), 2 = channel-owning streaming."""
    B, T, H, N = a.shape
    k, n = ctypes.c_int(0), ctypes.c_int(0)
    with torch.cuda.device(a.device):
        _check(lib().kla_scan_forward_plan(B, T, H, N, _dtype_code(a), _ptr(a), _ptr(p), _ptr(phi),
                                           _ptr(b), ctypes.byref(k), ctypes.byref(n)),
               "kla_scan_forward_plan")
    return int(k.value), int(n.value)


def chunk_tokens() -> int:
    return int(lib().kla_forward_chunk_tokens())


def new_workspace(B: int, T: int, H: int, N: int, dtype: torch.dtype, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(workspace_size(B, T, H, N, dtype), 1), dtype=torch.uint8, device=device)


def scan_forward(a: torch.Tensor, p: torch.Tensor, phi: torch.Tensor, b: torch.Tensor,
                 lam0: torch.Tensor, eta0: torch.Tensor, *,
                 want_mu: bool = True, want_var: bool = True,
                 out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None,
                 ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Filter [B, T, H, N] inputs from the [B, H, N] prior.

    Returns (lambda, eta, mu, var) as fp32 [B, T, H, N] tensors (mu / var are
    None when not wanted).  CUDA inputs give CUDA outputs, enqueued on
    ``stream`` (default: the current stream) without synchronising.  CPU
    inputs (ideally pinned) are copied to the current CUDA device, filtered
    there, and copied back; the call then returns CPU tensors after a
    synchronise.  ``out`` may supply the four output tensors (None entries
    for skipped outputs) on the side the results are returned on.
    """
    if not (a.shape == p.shape == phi.shape == b.shape) or a.dim() != 4:
        raise ValueError("a, p, phi, b must share one [B, T, H, N] shape")
    if not (a.dtype == p.dtype == phi.dtype == b.dtype):
        raise TypeError("a, p, phi, b must share one dtype")
    B, T, H, N = a.shape
    if lam0.shape != (B, H, N) or eta0.shape != (B, H, N):
        raise ValueError("lam0 and eta0 must be [B, H, N]")
    if lam0.dtype != torch.float32 or eta0.dtype != torch.float32:
        raise TypeError("lam0 and eta0 must be float32")
    host = not a.is_cuda
    if host:
        return _scan_forward_host(a, p, phi, b, lam0, eta0, want_mu=want_mu, want_var=want_var, out=out,
                                  workspace=workspace, stream=stream)

    _require_cuda(a, p, phi, b, lam0, eta0)
    code = _dtype_code(a)
    dev = a.device
    if out is None:
        outs = [torch.empty((B, T, H, N), dtype=torch.float32, device=dev),
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev),
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev) if want_mu else None,
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev) if want_var else None]
    else:
        outs = list(out)
        _require_cuda(*[o for o in outs if o is not None])
    if workspace is None:
        workspace = new_workspace(B, T, H, N, a.dtype, dev)
    with torch.cuda.device(dev):
        st = kla_scan_forward_raw(a, p, phi, b, code, lam0, eta0, outs, B, T, H, N, workspace,
                                  _stream_handle(stream))
    _check(st, "kla_scan_forward")
    return tuple(outs)


def host_workspace_size(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32,
                        t_block: int = 0) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_scan_forward_host_workspace_size(B, T, H, N, code, t_block, ctypes.byref(out)),
           "kla_scan_forward_host_workspace_size")
    return int(out.value)


def _scan_forward_host(a, p, phi, b, lam0, eta0, *, want_mu, want_var, out, workspace, stream,
                       t_block: int = 0):
    """kla_scan_forward_host: host tensors in and out, copies pipelined with
    the scan on the current CUDA device; returns after the outputs are in
    host memory."""
    for t in (a, p, phi, b, lam0, eta0):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host path: every tensor must be a contiguous CPU tensor")
    B, T, H, N = a.shape
    pinned = a.is_pinned()
    if out is None:
        outs = [torch.empty((B, T, H, N), dtype=torch.float32, pin_memory=pinned),
                torch.empty((B, T, H, N), dtype=torch.float32, pin_memory=pinned),
                torch.empty((B, T, H, N), dtype=torch.float32, pin_memory=pinned) if want_mu else None,
                torch.empty((B, T, H, N), dtype=torch.float32, pin_memory=pinned) if want_var else None]
    else:
        outs = list(out)
    dev = torch.device("cuda", torch.cuda.current_device())
    if workspace is None:
        workspace = torch.empty(max(host_workspace_size(B, T, H, N, a.dtype, t_block), 1), dtype=torch.uint8,
                                device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        st = lib().kla_scan_forward_host(
            _ptr(a), _ptr(p), _ptr(phi), _ptr(b), _dtype_code(a), _ptr(lam0), _ptr(eta0),
            _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(outs[3]), B, T, H, N, t_block,
            _ptr(workspace), workspace.numel(), s.cuda_stream)
    _check(st, "kla_scan_forward_host")
    s.synchronize()
    return tuple(outs)


def kla_scan_forward_raw(a, p, phi, b, code, lam0, eta0, outs, B, T, H, N, workspace, stream) -> int:
    """Direct C-ABI call; returns the status code."""
    return lib().kla_scan_forward(
        _ptr(a), _ptr(p), _ptr(phi), _ptr(b), code, _ptr(lam0), _ptr(eta0),
        _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(outs[3]), B, T, H, N,
        _ptr(workspace), workspace.numel() if workspace is not None else 0, stream)


def scan_step(a: torch.Tensor, p: torch.Tensor, phi: torch.Tensor, b: torch.Tensor,
              lam_state: torch.Tensor, eta_state: torch.Tensor, *,
              mu_out: Optional[torch.Tensor] = None, var_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> None:
    """One decode token for every channel of [B, H, N] inputs; updates
    ``lam_state`` / ``eta_state`` in place and writes ``mu_out`` / ``var_out``
    when given.  Enqueued on ``stream`` (default: the current stream)."""
    if not (a.shape == p.shape == phi.shape == b.shape == lam_state.shape == eta_state.shape):
        raise ValueError("step inputs and state must share one [B, H, N] shape")
    if a.dim() != 3:
        raise ValueError("step tensors are [B, H, N]")
    if lam_state.dtype != torch.float32 or eta_state.dtype != torch.float32:
        raise TypeError("state must be float32")
    _require_cuda(a, p, phi, b, lam_state, eta_state, mu_out, var_out)
    B, H, N = a.shape
    with torch.cuda.device(a.device):
        st = lib().kla_scan_step(_ptr(a), _ptr(p), _ptr(phi), _ptr(b), _dtype_code(a),
                                 _ptr(lam_state), _ptr(eta_state), _ptr(mu_out), _ptr(var_out),
                                 B, H, N, _stream_handle(stream))
    _check(st, "kla_scan_step")


def get_error(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise and return the device-side status (KLA_OK, KLA_ERR_TIMEOUT, ...)."""
    return int(lib().kla_get_error(_stream_handle(stream)))


def set_wait_limit_ns(ns: int) -> None:
    _check(lib().kla_set_wait_limit_ns(int(ns)), "kla_set_wait_limit_ns")


def debug_unset_flag_wait(stream: Optional[torch.cuda.Stream] = None) -> None:
    _check(lib().kla_debug_unset_flag_wait(_stream_handle(stream)), "kla_debug_unset_flag_wait")


def debug_force_forward_kernel(which: int) -> None:
    """0: choose by shape; 1: chunked kernel (workspace carries); 2: streaming kernel."""
    _check(lib().kla_debug_force_forward_kernel(int(which)), "kla_debug_force_forward_kernel")


def debug_stall_chunk(chunk: int) -> None:
    _check(lib().kla_debug_stall_chunk(int(chunk)), "kla_debug_stall_chunk")


def scan_forward_static(a: torch.Tensor, p: torch.Tensor, phi: torch.Tensor, b: torch.Tensor,
                        lam0: torch.Tensor, eta0: torch.Tensor,
                        out: Sequence[Optional[torch.Tensor]],
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """kla_scan_forward_static: the forward scan for callers that cannot
    allocate device memory.  The caller passes every tensor, outputs
    included (``out`` = lambda, eta, mu, var; mu / var may be None); the
    library uses its own fixed static device scratch (KLA_STATIC_SCRATCH_BYTES),
    so nothing is allocated.  Calls that overlap on the GPU share that scratch
    and must be serialised.  Raises KlaError(KLA_ERR_TOO_LARGE) when the
    problem does not fit."""
    if not (a.shape == p.shape == phi.shape == b.shape) or a.dim() != 4:
        raise ValueError("a, p, phi, b must share one [B, T, H, N] shape")
    B, T, H, N = a.shape
    outs = list(out)
    _require_cuda(a, p, phi, b, lam0, eta0, *outs)
    with torch.cuda.device(a.device):
        st = lib().kla_scan_forward_static(
            _ptr(a), _ptr(p), _ptr(phi), _ptr(b), _dtype_code(a), _ptr(lam0), _ptr(eta0),
            _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(outs[3]), B, T, H, N,
            _stream_handle(stream))
    _check(st, "kla_scan_forward_static")


# ---------------------------------------------------------------- gradients
def backward_workspace_size(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_scan_backward_workspace_size(B, T, H, N, code, ctypes.byref(out)),
           "kla_scan_backward_workspace_size")
    return int(out.value)


def backward_plan(a: torch.Tensor, p: torch.Tensor) -> Tuple[int, int]:
    """(kernel, launches) that scan_backward would use: kernel 1 = one thread
    per channel, 2 = channel-owning streaming kernel."""
    B, T, H, N = a.shape
    k, n = ctypes.c_int(0), ctypes.c_int(0)
    with torch.cuda.device(a.device):
        _check(lib().kla_scan_backward_plan(B, T, H, N, _dtype_code(a), _ptr(a), _ptr(p), ctypes.byref(k),
                                            ctypes.byref(n)), "kla_scan_backward_plan")
    return int(k.value), int(n.value)


def debug_force_backward_kernel(which: int) -> None:
    """0: choose by shape; 1: one thread per channel; 2: streaming kernel."""
    _check(lib().kla_debug_force_backward_kernel(int(which)), "kla_debug_force_backward_kernel")


def scan_backward(a: torch.Tensor, p: torch.Tensor, lam0: torch.Tensor, eta0: torch.Tensor,
                  lam: torch.Tensor, eta: torch.Tensor,
                  g_lam: Optional[torch.Tensor] = None, g_eta: Optional[torch.Tensor] = None,
                  g_mu: Optional[torch.Tensor] = None, g_var: Optional[torch.Tensor] = None, *,
                  want: Sequence[bool] = (True,) * 6,
                  out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                  workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[Optional[torch.Tensor], ...]:
    """Gradients through scan_forward (kla_scan_backward).

    ``a``, ``p`` are the forward inputs, ``lam0``, ``eta0`` its prior and
    ``lam``, ``eta`` its outputs; ``g_*`` are the loss gradients with respect
    to the four outputs (None = zero).  Returns the gradients with respect to
    (a, p, phi, b, lam0, eta0): the first four in the inputs' dtype, the prior
    ones fp32, None where ``want`` is False.  Enqueued on ``stream`` without
    synchronising.
    """
    if a.dim() != 4 or a.shape != p.shape or a.dtype != p.dtype:
        raise ValueError("a and p must share one [B, T, H, N] shape and dtype")
    B, T, H, N = a.shape
    if lam.shape != a.shape or eta.shape != a.shape:
        raise ValueError("lam and eta must be the forward outputs, [B, T, H, N]")
    if lam0.shape != (B, H, N) or eta0.shape != (B, H, N):
        raise ValueError("lam0 and eta0 must be [B, H, N]")
    grads_in = [g_lam, g_eta, g_mu, g_var]
    for t in [lam, eta, lam0, eta0] + [g for g in grads_in if g is not None]:
        if t.dtype != torch.float32:
            raise TypeError("states, prior and output gradients must be float32")
    for g in grads_in:
        if g is not None and g.shape != a.shape:
            raise ValueError("output gradients must be [B, T, H, N]")
    _require_cuda(a, p, lam0, eta0, lam, eta, *grads_in)
    code = _dtype_code(a)
    dev = a.device
    if out is None:
        outs = [torch.empty((B, T, H, N), dtype=a.dtype, device=dev) if w else None for w in want[:4]]
        outs += [torch.empty((B, H, N), dtype=torch.float32, device=dev) if w else None for w in want[4:6]]
    else:
        outs = list(out)
        _require_cuda(*outs)
    if workspace is None:
        n = backward_workspace_size(B, T, H, N, a.dtype)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    with torch.cuda.device(dev):
        st = lib().kla_scan_backward(
            _ptr(a), _ptr(p), code, _ptr(lam0), _ptr(eta0), _ptr(lam), _ptr(eta),
            *[_ptr(g) for g in grads_in], *[_ptr(o) for o in outs], B, T, H, N,
            _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream_handle(stream))
    _check(st, "kla_scan_backward")
    return tuple(outs)


class KalmanFilterScan(torch.autograd.Function):
    """Differentiable filter scan: forward = kla_scan_forward, backward =
    kla_scan_backward.  Inputs (a, p, phi, b, lam0, eta0) as in scan_forward
    (CUDA tensors); returns (lambda, eta, mu, var)."""

    @staticmethod
    def forward(ctx, a, p, phi, b, lam0, eta0):
        ctx.set_materialize_grads(False)
        lam, eta, mu, var = scan_forward(a, p, phi, b, lam0, eta0)
        ctx.save_for_backward(a, p, lam0, eta0, lam, eta)
        return lam, eta, mu, var

    @staticmethod
    def backward(ctx, g_lam, g_eta, g_mu, g_var):
        a, p, lam0, eta0, lam, eta = ctx.saved_tensors
        grads = [None if g is None else g.contiguous() for g in (g_lam, g_eta, g_mu, g_var)]
        if all(g is None for g in grads):
            return (None,) * 6
        return scan_backward(a, p, lam0, eta0, lam, eta, *grads, want=ctx.needs_input_grad)


def kalman_filter(a: torch.Tensor, p: torch.Tensor, phi: torch.Tensor, b: torch.Tensor,
                  lam0: torch.Tensor, eta0: torch.Tensor):
    """(lambda, eta, mu, var) of the filter, differentiable with respect to
    every input through the CUDA backward scan."""
    return KalmanFilterScan.apply(a, p, phi, b, lam0, eta0)


# ------------------------------------------------------------ fused layer
class QKNorm(NamedTuple):
    """What layer_forward and layer_step do to k and q first
    (qk_norm_rotary_forward with D = Ns): weights [Ns] fp32 or None, and the
    rotation (none without inv_freq)."""
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6
    inv_freq: Optional[torch.Tensor] = None
    interleaved: bool = False
    scale: float = 1.0


def _normed(norm: QKNorm, k, q, positions, position0, stream):
    q, k = qk_norm_rotary_forward(q, k, norm.q_weight, norm.k_weight, norm.inv_freq, positions,
                                  position0=position0, eps=norm.eps, interleaved=norm.interleaved,
                                  scale=norm.scale, stream=stream)
    return k, q


def layer_workspace_size(B: int, T: int, H: int, D: int, Ns: int, dtype: torch.dtype = torch.float32) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_layer_forward_workspace_size(B, T, H, D, Ns, code, ctypes.byref(out)),
           "kla_layer_forward_workspace_size")
    return int(out.value)


def layer_forward(k: torch.Tensor, q: torch.Tensor, v: torch.Tensor, w: torch.Tensor,
                  a: torch.Tensor, p: torch.Tensor, lam0: torch.Tensor, eta0: torch.Tensor, *,
                  want_s: bool = True, want_state: bool = True,
                  qk_norm: Optional[QKNorm] = None, positions: Optional[torch.Tensor] = None, position0: int = 0,
                  out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                  workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None):
    """The KLA layer's filter with evidence formation and readout fused
    (kla_layer_forward): k, q [B, T, H, Ns]; v, w [B, T, H, D] (one dtype,
    fp32 or bf16); a, p [H, D, Ns] fp32; lam0, eta0 [B, H, D, Ns] fp32.
    Returns (y, s, lam_T, eta_T): y, s fp32 [B, T, H, D], the final state fp32
    [B, H, D, Ns]; s / the state are None when not wanted.  With ``qk_norm``, k
    and q are normalised (and rotated by ``positions``, or position0 + t) first
    and may be strided."""
    if k.dim() != 4 or q.shape != k.shape or v.dim() != 4 or w.shape != v.shape:
        raise ValueError("k, q must be [B, T, H, Ns] and v, w [B, T, H, D]")
    if not (k.dtype == q.dtype == v.dtype == w.dtype):
        raise TypeError("k, q, v, w must share one dtype")
    B, T, H, Ns = k.shape
    D = v.shape[3]
    if tuple(v.shape[:3]) != (B, T, H) or a.shape != (H, D, Ns) or p.shape != (H, D, Ns):
        raise ValueError("v, w must be [B, T, H, D] and a, p [H, D, Ns]")
    if lam0.shape != (B, H, D, Ns) or eta0.shape != (B, H, D, Ns):
        raise ValueError("lam0 and eta0 must be [B, H, D, Ns]")
    for t in (a, p, lam0, eta0):
        if t.dtype != torch.float32:
            raise TypeError("a, p, lam0, eta0 must be float32")
    if qk_norm is not None:
        k, q = _normed(qk_norm, k, q, positions, position0, stream)
    elif positions is not None or position0:
        raise ValueError("positions need qk_norm")
    _require_cuda(k, q, v, w, a, p, lam0, eta0)
    dev = k.device
    if out is None:
        outs = [torch.empty((B, T, H, D), dtype=torch.float32, device=dev),
                torch.empty((B, T, H, D), dtype=torch.float32, device=dev) if want_s else None,
                torch.empty((B, H, D, Ns), dtype=torch.float32, device=dev) if want_state else None,
                torch.empty((B, H, D, Ns), dtype=torch.float32, device=dev) if want_state else None]
    else:
        outs = list(out)
        _require_cuda(*outs)
    if workspace is None:
        n = layer_workspace_size(B, T, H, D, Ns, k.dtype)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    with torch.cuda.device(dev):
        st = lib().kla_layer_forward(
            _ptr(k), _ptr(q), _ptr(v), _ptr(w), _dtype_code(k), _ptr(a), _ptr(p), _ptr(lam0), _ptr(eta0),
            *[_ptr(o) for o in outs], B, T, H, D, Ns,
            _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream_handle(stream))
    _check(st, "kla_layer_forward")
    return tuple(outs)


def layer_step(k: torch.Tensor, q: torch.Tensor, v: torch.Tensor, w: torch.Tensor,
               a: torch.Tensor, p: torch.Tensor, lam_state: torch.Tensor, eta_state: torch.Tensor, *,
               y: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None, want_s: bool = True,
               qk_norm: Optional[QKNorm] = None, positions: Optional[torch.Tensor] = None, position0: int = 0,
               stream: Optional[torch.cuda.Stream] = None):
    """One decode token of the fused layer (kla_layer_step): k, q [B, H, Ns];
    v, w [B, H, D]; a, p [H, D, Ns]; the state [B, H, D, Ns] is updated in
    place.  Returns (y, s), fp32 [B, H, D] (s None when not wanted).  With
    ``qk_norm``, k and q are normalised (and rotated by the positions [B], or
    position0) first."""
    if k.dim() != 3 or q.shape != k.shape or v.dim() != 3 or w.shape != v.shape:
        raise ValueError("k, q must be [B, H, Ns] and v, w [B, H, D]")
    if not (k.dtype == q.dtype == v.dtype == w.dtype):
        raise TypeError("k, q, v, w must share one dtype")
    B, H, Ns = k.shape
    D = v.shape[2]
    if tuple(v.shape[:2]) != (B, H) or lam_state.shape != (B, H, D, Ns) or eta_state.shape != (B, H, D, Ns):
        raise ValueError("v, w must be [B, H, D] and the state [B, H, D, Ns]")
    if qk_norm is not None:
        at = None if positions is None else positions.unsqueeze(-1)
        k, q = (t.squeeze(1) for t in _normed(qk_norm, k.unsqueeze(1), q.unsqueeze(1), at, position0, stream))
    elif positions is not None or position0:
        raise ValueError("positions need qk_norm")
    _require_cuda(k, q, v, w, a, p, lam_state, eta_state, y, s)
    if y is None:
        y = torch.empty((B, H, D), dtype=torch.float32, device=k.device)
    if s is None and want_s:
        s = torch.empty((B, H, D), dtype=torch.float32, device=k.device)
    with torch.cuda.device(k.device):
        st = lib().kla_layer_step(_ptr(k), _ptr(q), _ptr(v), _ptr(w), _dtype_code(k), _ptr(a), _ptr(p),
                                  _ptr(lam_state), _ptr(eta_state), _ptr(y), _ptr(s), B, H, D, Ns,
                                  _stream_handle(stream))
    _check(st, "kla_layer_step")
    return y, s


def attention_weights(a: torch.Tensor, p: torch.Tensor, lam: torch.Tensor, *, t0: int = 0,
                      span: Optional[int] = None, W: int = ATTENTION_MAX_WINDOW,
                      out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The Kalman attention weights F(t, s) = prod_{k=s+1..t} f_k of the
    windows of W tokens of [t0, t0 + span), from the forward inputs a, p and
    the forward scan's lambda ([B, T, H, N]).  Returns fp32
    [B, ceil(span / W), W, W, H, N] (kla_attention_weights)."""
    if a.dim() != 4 or p.shape != a.shape or lam.shape != a.shape:
        raise ValueError("a, p, lam must share one [B, T, H, N] shape")
    if p.dtype != a.dtype or lam.dtype != torch.float32:
        raise TypeError("a and p share one dtype; lam is float32")
    B, T, H, N = a.shape
    span = T - t0 if span is None else span
    nwin = -(-span // W) if W > 0 else 0
    _require_cuda(a, p, lam)
    if out is None:
        out = torch.empty((B, nwin, W, W, H, N), dtype=torch.float32, device=a.device)
    else:
        _require_cuda(out)
        if out.shape != (B, nwin, W, W, H, N) or out.dtype != torch.float32:
            raise ValueError("out must be float32 [B, nwin, W, W, H, N]")
    with torch.cuda.device(a.device):
        _check(lib().kla_attention_weights(_ptr(a), _ptr(p), _dtype_code(a), _ptr(lam), _ptr(out), B, T, H, N,
                                           t0, span, W, _stream_handle(stream)), "kla_attention_weights")
    return out


def lti_workspace_size(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_scan_forward_lti_workspace_size(B, T, H, N, code, ctypes.byref(out)),
           "kla_scan_forward_lti_workspace_size")
    return int(out.value)


def lti_plan(phi: torch.Tensor, b: torch.Tensor) -> Tuple[int, int]:
    """(kernel, launches) of scan_forward_lti: 1 = one thread per channel,
    2 = channel-owning streaming."""
    B, T, H, N = phi.shape
    k, n = ctypes.c_int(0), ctypes.c_int(0)
    with torch.cuda.device(phi.device):
        _check(lib().kla_scan_forward_lti_plan(B, T, H, N, _dtype_code(phi), _ptr(phi), _ptr(b), ctypes.byref(k),
                                               ctypes.byref(n)), "kla_scan_forward_lti_plan")
    return int(k.value), int(n.value)


def scan_forward_lti(a: torch.Tensor, phi: torch.Tensor, b: torch.Tensor, lam0: torch.Tensor,
                     eta0: torch.Tensor, *, want_mu: bool = True, want_var: bool = True,
                     out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None,
                     ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The deterministic time-invariant filter (p = 0, decay a [B, H, N]
    constant in time) in its convolutional form (kla_scan_forward_lti):
    phi, b [B, T, H, N]; returns (lambda, eta, mu, var) as scan_forward does."""
    if phi.dim() != 4 or b.shape != phi.shape or b.dtype != phi.dtype:
        raise ValueError("phi, b must share one [B, T, H, N] shape and dtype")
    B, T, H, N = phi.shape
    for t, name in ((a, "a"), (lam0, "lam0"), (eta0, "eta0")):
        if t.shape != (B, H, N) or t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32 [B, H, N]")
    _require_cuda(a, phi, b, lam0, eta0)
    dev = phi.device
    if out is None:
        outs = [torch.empty((B, T, H, N), dtype=torch.float32, device=dev),
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev),
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev) if want_mu else None,
                torch.empty((B, T, H, N), dtype=torch.float32, device=dev) if want_var else None]
    else:
        outs = list(out)
        _require_cuda(*[o for o in outs if o is not None])
    if workspace is None:
        workspace = torch.empty(max(lti_workspace_size(B, T, H, N, phi.dtype), 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = lib().kla_scan_forward_lti(_ptr(a), _ptr(phi), _ptr(b), _dtype_code(phi), _ptr(lam0), _ptr(eta0),
                                        _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(outs[3]), B, T, H, N,
                                        _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check(st, "kla_scan_forward_lti")
    return tuple(outs)


# ------------------------------------------------ gated linear recurrence
# The mixer operators are bound natively (csrc/kla_binding.cpp): their checks,
# allocations and stream take about as long there as one of these calls takes
# the GPU.
_mixer = None


def _native():
    """The extension ``_mixer.so`` (raises if it is missing, or for another torch or Python)."""
    global _mixer
    if _mixer is None:
        lib()  # raises if libkla.so, which it is linked to, is missing
        from . import _build
        build = "build it with `python -m kalman_linear_attention_b200._build`"
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(f"the binding of the mixer operators is not built; {build}")
        try:
            from . import _mixer as module
        except ImportError as e:
            raise RuntimeError(f"the binding of the mixer operators could not be loaded ({e}); {build}") from e
        if module.built_for != _build.built_for():
            raise RuntimeError(f"the binding of the mixer operators is for {module.built_for}, "
                               f"this is {_build.built_for()}; {build}")
        module.set_error(KlaError)
        _mixer = module
    return _mixer


def gated_scan_forward(f: torch.Tensor, x: torch.Tensor, h0: Optional[torch.Tensor] = None, *,
                       out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gated linear recurrence h_t = f_t h_{t-1} + x_t
    (kla_gated_scan_forward): x [B, T, H, N]; f of the same shape, or
    [B, T, H] with one gate for a head's channels (both fp32 or both bf16); h0
    [B, H, N] fp32 (None: zero).  Returns the states, fp32 [B, T, H, N]; the
    last one continues with gated_scan_step.  Enqueued on ``stream`` (default:
    the current stream) without synchronising."""
    return (_mixer or _native()).gated_scan_forward(f, x, h0, out, stream)


class GatedPlan(NamedTuple):
    """How a gated scan runs (kla_gated_plan_t)."""
    tiles: int
    rounds: int
    channels: int
    parts: int
    tokens: int
    warps: int
    cluster: int
    whole_rows: int


class _GatedPlan(ctypes.Structure):
    _fields_ = [("tiles", _I64), ("rounds", _I64)] + [(n, ctypes.c_int) for n in GatedPlan._fields[2:]]


def gated_scan_plan(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32, head_gate: bool = False,
                    backward: bool = False) -> GatedPlan:
    """How gated_scan_forward, or gated_scan_backward, runs on aligned arrays of
    these sizes (kla_gated_scan_plan)."""
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = _GatedPlan()
    _check(lib().kla_gated_scan_plan(B, T, H, N, code, int(head_gate), int(backward), ctypes.byref(out)),
           "kla_gated_scan_plan")
    return GatedPlan(*(getattr(out, n) for n in GatedPlan._fields))


def gated_scan_step(f: torch.Tensor, x: torch.Tensor, h_state: torch.Tensor, *,
                    out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode token of the gated recurrence (kla_gated_scan_step): x
    [B, H, N], f of that shape or [B, H], h_state [B, H, N] fp32.  The new state
    goes to ``out``, or in place to h_state without it; returns where it went."""
    return (_mixer or _native()).gated_scan_step(f, x, h_state, out, stream)


def gated_scan_backward_workspace_size(B: int, T: int, H: int, N: int, dtype: torch.dtype = torch.float32,
                                       head_gate: bool = False) -> int:
    code = KLA_BF16 if dtype == torch.bfloat16 else KLA_F32
    out = ctypes.c_size_t(0)
    _check(lib().kla_gated_scan_backward_workspace_size(B, T, H, N, code, int(head_gate), ctypes.byref(out)),
           "kla_gated_scan_backward_workspace_size")
    return int(out.value)


def gated_scan_backward(f: torch.Tensor, h: torch.Tensor, g_h: torch.Tensor, h0: Optional[torch.Tensor] = None, *,
                        want: Sequence[bool] = (True, True, True),
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> Tuple[Optional[torch.Tensor], ...]:
    """Gradients through gated_scan_forward (kla_gated_scan_backward): f and
    h0 as given to it, h the states it returned, g_h the loss gradient with
    respect to them (fp32).  Returns the gradients with respect to (f, x, h0):
    the first two in f's dtype, the last fp32; None where ``want`` is False."""
    return (_mixer or _native()).gated_scan_backward(f, h, g_h, h0, *want, workspace, stream)


class GatedScan(torch.autograd.Function):
    """Differentiable gated recurrence: forward = kla_gated_scan_forward,
    backward = kla_gated_scan_backward.  Inputs (f, x, h0) as in
    gated_scan_forward; returns the states.  (To capture a backward pass into a
    CUDA graph, let go of every eager graph over the same leaves first: torch
    would join the stream that they were made on to the capture.)"""

    @staticmethod
    def forward(ctx, f, x, h0):
        h = gated_scan_forward(f, x, h0)
        ctx.save_for_backward(f, h, h0)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, g_h):
        f, h, h0 = ctx.saved_tensors
        need = ctx.needs_input_grad
        return gated_scan_backward(f, h, g_h.contiguous(), h0, want=(need[0], need[1], need[2] and h0 is not None))


def gated_scan(f: torch.Tensor, x: torch.Tensor, h0: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The states of the gated recurrence, differentiable with respect to
    f, x and h0 through the CUDA backward scan."""
    return GatedScan.apply(f, x, h0)


# ---------------------------------------- QK norm and rotary positions
def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                       length: int = 4096, fast: float = 32.0, slow: float = 1.0,
                       device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, scale) for rotary and qk_norm_rotary: inv_freq [rot_dim / 2]
    fp64, base^(-2 i / rot_dim) radians per position, made for contexts
    ``factor`` times as long as the ``length`` a model was trained on:

    * ``"none"``: as it is;
    * ``"linear"``: every position divided by ``factor``;
    * ``"ntk"``: the base raised, so that the slowest pair turns ``factor``
      times slower and the fastest keeps its angle;
    * ``"yarn"``: pairs that make more than ``fast`` turns over ``length`` keep
      their angle, those with fewer than ``slow`` are divided by ``factor``,
      with a ramp between that is linear in the turns, as published; scale = 0.1
      ln(factor) + 1.  A checkpoint whose ramp is linear in the pair's index
      instead needs frequencies of its own.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if not base > 0.0:
        raise ValueError("base must be positive")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    inv_freq = base ** (-i / max(rot_dim, 1))
    if scaling == "linear":
        inv_freq = inv_freq / factor
    elif scaling == "yarn":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        keep = ((length * inv_freq / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        inv_freq = inv_freq / factor * (1 - keep) + inv_freq * keep
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be none, linear, ntk or yarn, got {scaling!r}")
    return inv_freq.to(device) if device is not None else inv_freq, scale


def rotary_forward(x: torch.Tensor, inv_freq: torch.Tensor, positions: Optional[torch.Tensor] = None, *,
                   position0: int = 0, interleaved: bool = False, scale: float = 1.0, inverse: bool = False,
                   out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rotary positions (kla_rotary_forward): the first 2 len(inv_freq)
    elements of every row of x [B, T, H, D] (fp32 or bf16; any strides of B, T,
    H) turned by position times frequency.  inv_freq fp64
    (rotary_frequencies); positions int64 [B, T] or [T], or None for position0
    + t; ``interleaved``: neighbours form a pair, else the two halves do;
    ``inverse``: the other way round.  Returns a dense tensor of x's type."""
    return (_mixer or _native()).rotary_forward(x, inv_freq, positions, position0, interleaved, scale, inverse, out,
                                                stream)


def _not_formed(ctx, first, *names):
    """Refuse a backward pass that wants the gradient of an input from ``first`` on."""
    for name, wanted in zip(names, ctx.needs_input_grad[first:]):
        if wanted:
            raise RuntimeError(f"the gradient of {name} is not formed; pass it without requires_grad")


class Rotary(torch.autograd.Function):
    """Differentiable rotary_forward: the gradient is the inverse rotation.
    Frequencies that want a gradient are refused in the backward pass."""

    @staticmethod
    def forward(ctx, x, inv_freq, positions, position0, interleaved, scale):
        ctx.rotation = dict(position0=position0, interleaved=interleaved, scale=scale)
        ctx.save_for_backward(inv_freq, positions)
        return rotary_forward(x, inv_freq, positions, **ctx.rotation)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        _not_formed(ctx, 1, "inv_freq", "positions", "position0", "interleaved", "scale")
        inv_freq, positions = ctx.saved_tensors
        return (rotary_forward(g.contiguous(), inv_freq, positions, inverse=True, **ctx.rotation),
                None, None, None, None, None)


def rotary(x: torch.Tensor, inv_freq: torch.Tensor, positions: Optional[torch.Tensor] = None, *,
           position0: int = 0, interleaved: bool = False, scale: float = 1.0) -> torch.Tensor:
    """rotary_forward, differentiable with respect to x alone."""
    return Rotary.apply(x, inv_freq, positions, position0, interleaved, scale)


def qk_norm_rotary_forward(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                           positions: Optional[torch.Tensor] = None, *, position0: int = 0, eps: float = 1e-6,
                           interleaved: bool = False, scale: float = 1.0,
                           out: Optional[Sequence[torch.Tensor]] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """QK-Norm with the position rotation in the same pass
    (kla_qk_norm_rotary_forward): q [B, T, Hq, D], k [B, T, Hk, D] (one of fp32
    and bf16; any strides of B, T, H, so slices of a packed projection); the
    RMS norm of each head, times the weight ([D] fp32 or None), rotated as in
    rotary_forward (not at all without inv_freq).  Returns dense (q, k) of the
    inputs' type."""
    q_out, k_out = (None, None) if out is None else out
    return (_mixer or _native()).qk_norm_rotary_forward(q, k, q_weight, k_weight, inv_freq, positions, position0, eps,
                                                        interleaved, scale, q_out, k_out, stream)


def qk_norm_rotary_backward_workspace_size(Hq: int, Hk: int, D: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kla_qk_norm_rotary_backward_workspace_size(Hq, Hk, D, ctypes.byref(out)),
           "kla_qk_norm_rotary_backward_workspace_size")
    return int(out.value)


def qk_norm_rotary_backward(q: torch.Tensor, k: torch.Tensor, g_q: Optional[torch.Tensor],
                            g_k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                            k_weight: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                            positions: Optional[torch.Tensor] = None, *, position0: int = 0, eps: float = 1e-6,
                            interleaved: bool = False, scale: float = 1.0, want: Sequence[bool] = (True,) * 4,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> Tuple[Optional[torch.Tensor], ...]:
    """Gradients through qk_norm_rotary_forward (kla_qk_norm_rotary_backward):
    its inputs and the gradients g_q, g_k of its outputs (dense, the inputs'
    type; None = zero).  Returns the gradients with respect to (q, k, q_weight,
    k_weight): the first two dense in the inputs' type, the weights' fp32;
    None where ``want`` is False, where there is no weight, or where the
    output's gradient is None."""
    return (_mixer or _native()).qk_norm_rotary_backward(q, k, q_weight, k_weight, inv_freq, positions, position0, eps,
                                                         interleaved, scale, g_q, g_k, *want, workspace, stream)


class QKNormRotary(torch.autograd.Function):
    """Differentiable QK-Norm with rotation: forward =
    kla_qk_norm_rotary_forward, backward = kla_qk_norm_rotary_backward.
    Frequencies that want a gradient are refused in the backward pass."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, position0, eps, interleaved, scale):
        ctx.set_materialize_grads(False)
        ctx.options = dict(position0=position0, eps=eps, interleaved=interleaved, scale=scale)
        ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions)
        return qk_norm_rotary_forward(q, k, q_weight, k_weight, inv_freq, positions, **ctx.options)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_q, g_k):
        _not_formed(ctx, 4, "inv_freq", "positions", "position0", "eps", "interleaved", "scale")
        q, k, *rest = ctx.saved_tensors
        grads = [None if g is None else g.contiguous() for g in (g_q, g_k)]
        got = qk_norm_rotary_backward(q, k, *grads, *rest, **ctx.options, want=ctx.needs_input_grad[:4])
        return (*got, None, None, None, None, None, None)


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                   positions: Optional[torch.Tensor] = None, *, position0: int = 0, eps: float = 1e-6,
                   interleaved: bool = False, scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """qk_norm_rotary_forward, differentiable with respect to q, k and the
    weights alone."""
    return QKNormRotary.apply(q, k, q_weight, k_weight, inv_freq, positions, position0, eps, interleaved, scale)
