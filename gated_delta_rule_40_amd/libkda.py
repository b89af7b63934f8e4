"""ctypes binding over libkda.so (C ABI declared in include/kda.h).

Argument marshalling only: shapes and dtypes are read off torch tensors,
device pointers and the current HIP stream are passed to the C entry points,
and every step of the computation runs in libkda's HIP kernels.  There is no
fallback: if the library is missing the calls raise.

    kda_prefill(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    kda_prefill_ex(..., chunk=0, dv_block=0)
    kda_prefill_snapshots(..., snapshots, snap_every)
    kda_prefill_cp(..., seg_len=0, workspace=None)
    kda_prefill_cp_workspace_size(num_seqs, total_tokens, num_heads, dk, dv, seg_len)
    kda_prefill_cp_noalloc(..., seg_len=0)
    kda_decode_step(q, k, v, g, beta, state_inout, out)
    kda_decode_tokens(q, k, v, g, beta, cu_seqlens, state_in, state_out=None, out=None, num_tokens=None)
    kda_backward(q, k, v, g, beta, initial_state, cu_seqlens, dout, dfinal=None, ...) -> gradients

The operators around the recurrence in a layer:

    kda_scan_prefill(x, g, initial_state, cu_seqlens, out, final_state, checkpoints=None, workspace=None)
    kda_scan_decode_step(x, g, state_inout, out)
    kda_scan_backward(x, g, initial_state, cu_seqlens, dout, dfinal=None, checkpoints=None, ...) -> gradients
    kda_conv_prefill(x, weight, bias, initial_state, cu_seqlens, out, final_state, silu=True)
    kda_conv_decode_step(x, weight, bias, state_inout, out, silu=True)
    kda_conv_backward(x, weight, bias, initial_state, cu_seqlens, dout, dfinal=None, silu=True, ...) -> gradients
    kda_rmsnorm(x, weight, out=None, residual=None, residual_out=None, out_mx=None, scales=None, eps=1e-6)
    kda_rmsnorm_backward(x, weight, dout, dresidual=None, eps=1e-6, ...) -> gradients
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_LAUNCH, KDA_ERR_SCRATCH = 0, 1, 2, 3, 4
KDA_STATIC_SCRATCH_BYTES = 256 * 1024 * 1024      # include/kda.h
KDA_F32, KDA_BF16 = 0, 1
KDA_SCAN_TILE, KDA_MX_BLOCK = 128, 32              # include/kda.h

EXPORTS = ("kda_prefill", "kda_prefill_ex", "kda_prefill_snapshots", "kda_prefill_cp",
           "kda_prefill_cp_workspace_size", "kda_prefill_cp_noalloc", "kda_decode_step", "kda_decode_tokens", "kda_backward",
           "kda_backward_workspace_size", "kda_scan_prefill", "kda_scan_workspace_size", "kda_scan_decode_step",
           "kda_scan_backward", "kda_scan_backward_workspace_size", "kda_conv_prefill", "kda_conv_decode_step",
           "kda_conv_backward", "kda_conv_backward_workspace_size", "kda_rmsnorm", "kda_rmsnorm_backward",
           "kda_rmsnorm_backward_workspace_size", "kda_status_string", "kda_version")

_lib = None


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libkda.so (built by ``python -m gated_delta_rule_40_amd.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError("libkda.so not built at %s; run python -m gated_delta_rule_40_amd.build" % p)
    lib = ctypes.CDLL(p)
    vp, fp, ip, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32
    lib.kda_prefill.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp, fp, vp]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill_ex.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp, fp,
                                   i32, i32, vp]
    lib.kda_prefill_ex.restype = ctypes.c_int
    lib.kda_prefill_snapshots.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp,
                                          fp, i32, i32, fp, vp]
    lib.kda_prefill_snapshots.restype = ctypes.c_int
    lib.kda_prefill_cp.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp, fp,
                                   i32, vp, ctypes.c_size_t, vp]
    lib.kda_prefill_cp.restype = ctypes.c_int
    lib.kda_prefill_cp_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp,
                                           fp, i32, vp]
    lib.kda_prefill_cp_noalloc.restype = ctypes.c_int
    lib.kda_prefill_cp_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int, i32]
    lib.kda_prefill_cp_workspace_size.restype = ctypes.c_size_t
    lib.kda_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, i32, i32, i32, i32, ctypes.c_int, vp, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_tokens.argtypes = [vp, vp, vp, fp, fp, ip, ip, fp, fp, i32, i32, i32, i32, i32, ctypes.c_int,
                                      vp, vp]
    lib.kda_decode_tokens.restype = ctypes.c_int
    lib.kda_backward.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i32, i32, i32, i32, ctypes.c_int, vp, fp,
                                 fp, fp, fp, fp, fp, fp, vp, ctypes.c_size_t, vp]
    lib.kda_backward.restype = ctypes.c_int
    lib.kda_backward_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int]
    lib.kda_backward_workspace_size.restype = ctypes.c_size_t
    size = ctypes.c_size_t
    for name, restype, args in (
            ("kda_scan_prefill", ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, ctypes.c_int, vp, vp, vp, vp, size, vp]),
            ("kda_scan_workspace_size", size, [i32, i32, i32, ctypes.c_int]),
            ("kda_scan_decode_step", ctypes.c_int, [vp, vp, vp, i32, i32, ctypes.c_int, vp, vp]),
            ("kda_scan_backward", ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                                 vp, size, vp]),
            ("kda_scan_backward_workspace_size", size, [i32, i32, i32, ctypes.c_int, i32]),
            ("kda_conv_prefill", ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_int, vp, vp, vp]),
            ("kda_conv_decode_step", ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_int, vp, vp]),
            ("kda_conv_backward", ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_int, vp, vp, vp,
                                                 vp, vp, vp, vp, size, vp]),
            ("kda_conv_backward_workspace_size", size, [i32, i32, i32, i32, ctypes.c_int]),
            ("kda_rmsnorm", ctypes.c_int, [vp, vp, vp, i32, i32, ctypes.c_float, ctypes.c_int, vp, vp, vp, vp, vp]),
            ("kda_rmsnorm_backward", ctypes.c_int, [vp, vp, vp, vp, i32, i32, ctypes.c_float, ctypes.c_int, vp, vp, vp,
                                                    size, vp]),
            ("kda_rmsnorm_backward_workspace_size", size, [i32, i32, ctypes.c_int])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = restype, args
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = ctypes.c_int32
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(status).decode()


def _check(status: int) -> None:
    if status != KDA_OK:
        raise KdaError(status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _on_device(ref: torch.Tensor, **tensors) -> None:
    """Every given tensor (None entries skipped) must be a device tensor on
    ref's device: the library dereferences the pointers on the GPU, so a host
    pointer or another device's memory would fault there."""
    _require(torch.is_tensor(ref) and ref.is_cuda, "q must be a device tensor")
    for name, t in tensors.items():
        if t is None:
            continue
        _require(torch.is_tensor(t) and t.is_cuda and t.device == ref.device,
                 "%s must be a tensor on %s" % (name, ref.device))


def _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state):
    _on_device(q, k=k, v=v, g=g, beta=beta, initial_state=initial_state, cu_seqlens=cu_seqlens, out=out,
               final_state=final_state)
    _require(q.dim() == 3 and v.dim() == 3 and cu_seqlens.dim() == 1 and cu_seqlens.shape[0] >= 1,
             "q, k, g, v, out must be [T, H, d] and cu_seqlens [N + 1]")
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("out", out),
                    ("cu_seqlens", cu_seqlens)):
        _require(t.is_contiguous(), "%s must be contiguous" % name)
    _require(cu_seqlens.dtype == torch.int32, "cu_seqlens must be int32")
    _require(g.dtype == torch.float32 and beta.dtype == torch.float32, "g and beta must be float32")
    _require(k.shape == q.shape and g.shape == q.shape and v.shape[:2] == (T, H) and out.shape == v.shape,
             "shape mismatch")
    _require(tuple(beta.shape) == (T, H), "beta must be [T, H]")
    _require(k.dtype == q.dtype and v.dtype == q.dtype and out.dtype == q.dtype, "q/k/v/out dtypes differ")
    for name, s in (("initial_state", initial_state), ("final_state", final_state)):
        if s is not None:
            _require(s.dtype == torch.float32 and s.is_contiguous() and tuple(s.shape) == (N, H, dk, dv),
                     "%s must be contiguous float32 [N, H, dk, dv]" % name)
    return N, T, H, dk, dv


def kda_prefill_ex(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state,
                   chunk: int = 0, dv_block: int = 0, stream=None) -> None:
    """Packed varlen prefill.  q, k, g: [T, H, dk]; v, out: [T, H, dv];
    beta: [T, H] fp32; initial_state/final_state: [N, H, dk, dv] fp32 or None;
    cu_seqlens: [N+1] int32 on the device."""
    N, T, H, dk, dv = _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    lib = load()
    _check(lib.kda_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                              _ptr(cu_seqlens), N, T, H, dk, dv, _dtype_code(q), _ptr(out),
                              _ptr(final_state), int(chunk), int(dv_block), _stream(stream)))


def kda_prefill_snapshots(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, snapshots,
                          snap_every: int, stream=None) -> None:
    """kda_prefill plus the state after every snap_every tokens of each
    sequence: snapshots [N, max_snaps, H, dk, dv] fp32 (max_snaps from its shape)."""
    N, T, H, dk, dv = _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    _on_device(q, snapshots=snapshots)
    _require(snapshots.dtype == torch.float32 and snapshots.is_contiguous() and snapshots.dim() == 5 and
             snapshots.shape[0] == N and tuple(snapshots.shape[2:]) == (H, dk, dv),
             "snapshots must be contiguous float32 [N, max_snaps, H, dk, dv]")
    lib = load()
    _check(lib.kda_prefill_snapshots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                     _ptr(cu_seqlens), N, T, H, dk, dv, _dtype_code(q), _ptr(out),
                                     _ptr(final_state), int(snap_every), int(snapshots.shape[1]),
                                     _ptr(snapshots), _stream(stream)))


def kda_prefill_cp_workspace_size(num_seqs: int, total_tokens: int, num_heads: int, dk: int, dv: int,
                                  dtype=torch.bfloat16, seg_len: int = 0) -> int:
    """Bytes of device workspace kda_prefill_cp needs (0 = unsupported sizes);
    dtype is that of q/k/v (torch.bfloat16 or torch.float32)."""
    code = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}.get(dtype)
    if code is None:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32, got %s" % dtype)
    return int(load().kda_prefill_cp_workspace_size(num_seqs, total_tokens, num_heads, dk, dv, code, seg_len))


def kda_prefill_cp(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state,
                   seg_len: int = 0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Context-parallel prefill (same arguments and result as kda_prefill):
    sequences are split into seg_len-token segments that run side by side
    (seg_len < 0: pieces of -seg_len tokens over the packed chunk order;
    0: automatic, see include/kda.h).
    ``workspace`` is a uint8 device tensor of at least
    kda_prefill_cp_workspace_size(...) bytes; if None, one is allocated."""
    N, T, H, dk, dv = _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    need = kda_prefill_cp_workspace_size(N, T, H, dk, dv, q.dtype, seg_len)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _on_device(q, workspace=workspace)
    _require(workspace.is_contiguous(), "workspace must be contiguous")
    nbytes = workspace.numel() * workspace.element_size()
    lib = load()
    _check(lib.kda_prefill_cp(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                              _ptr(cu_seqlens), N, T, H, dk, dv, _dtype_code(q), _ptr(out),
                              _ptr(final_state), int(seg_len), _ptr(workspace), nbytes, _stream(stream)))


def kda_prefill_cp_noalloc(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state,
                           seg_len: int = 0, stream=None) -> None:
    """kda_prefill_cp in the library's static device scratch: no workspace
    argument and no allocation.  Raises KdaError(KDA_ERR_SCRATCH) when the
    problem needs more than KDA_STATIC_SCRATCH_BYTES; calls overlapping in
    time on one GPU race on the shared scratch."""
    N, T, H, dk, dv = _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    lib = load()
    _check(lib.kda_prefill_cp_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                      _ptr(cu_seqlens), N, T, H, dk, dv, _dtype_code(q), _ptr(out),
                                      _ptr(final_state), int(seg_len), _stream(stream)))


def kda_prefill(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, stream=None) -> None:
    """kda_prefill with the library's default tiling."""
    kda_prefill_ex(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, 0, 0, stream)


def kda_decode_step(q, k, v, g, beta, state_inout, out, stream=None) -> None:
    """One decode step, state updated in place.  q, k, g: [N, H, dk];
    v, out: [N, H, dv]; beta: [N, H]; state_inout: [N, H, dk, dv] fp32."""
    _on_device(q, k=k, v=v, g=g, beta=beta, state_inout=state_inout, out=out)
    _require(q.dim() == 3 and v.dim() == 3, "q, k, g, v, out must be [N, H, d]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state_inout),
                    ("out", out)):
        _require(t.is_contiguous(), "%s must be contiguous" % name)
    _require(k.dtype == q.dtype and v.dtype == q.dtype and out.dtype == q.dtype, "q/k/v/out dtypes differ")
    _require(k.shape == q.shape and g.shape == q.shape and v.shape[:2] == (N, H) and out.shape == v.shape,
             "shape mismatch")
    _require(tuple(beta.shape) == (N, H) and tuple(state_inout.shape) == (N, H, dk, dv), "shape mismatch")
    _require(state_inout.dtype == torch.float32 and g.dtype == torch.float32 and beta.dtype == torch.float32,
             "g, beta and state must be float32")
    lib = load()
    _check(lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_inout), N, H, dk,
                               dv, _dtype_code(q), _ptr(out), _stream(stream)))


def kda_decode_tokens(q, k, v, g, beta, cu_seqlens, state_in, state_out=None, out=None, num_tokens=None,
                      stream=None) -> None:
    """A few consecutive tokens per (sequence, head), state kept on chip.
    q, k, g: [T, H, dk]; v, out: [T, H, dv]; beta: [T, H]; cu_seqlens: [N+1]
    int32 on the device; num_tokens: [N] int32 on the device or None;
    state_in / state_out: [N, H, dk, dv] fp32 (state_out None: not written)."""
    _on_device(q, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, state_in=state_in, state_out=state_out,
               out=out, num_tokens=num_tokens)
    _require(q.dim() == 3 and v.dim() == 3 and cu_seqlens.dim() == 1 and cu_seqlens.shape[0] >= 1,
             "q, k, g, v, out must be [T, H, d] and cu_seqlens [N + 1]")
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state_in", state_in),
                    ("cu_seqlens", cu_seqlens)):
        _require(t.is_contiguous(), "%s must be contiguous" % name)
    _require(cu_seqlens.dtype == torch.int32, "cu_seqlens must be int32")
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q/k/v dtypes differ")
    _require(k.shape == q.shape and g.shape == q.shape and v.shape[:2] == (T, H) and tuple(beta.shape) == (T, H),
             "shape mismatch")
    _require(g.dtype == torch.float32 and beta.dtype == torch.float32, "g and beta must be float32")
    for name, st in (("state_in", state_in), ("state_out", state_out)):
        if st is not None:
            _require(st.dtype == torch.float32 and st.is_contiguous() and tuple(st.shape) == (N, H, dk, dv),
                     "%s must be contiguous float32 [N, H, dk, dv]" % name)
    if out is not None:
        _require(out.is_contiguous() and out.shape == v.shape and out.dtype == q.dtype, "out must match v")
    if num_tokens is not None:
        _require(num_tokens.dtype == torch.int32 and num_tokens.is_contiguous() and tuple(num_tokens.shape) == (N,),
                 "num_tokens must be int32 [N] on the device")
    lib = load()
    _check(lib.kda_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                 _ptr(num_tokens), _ptr(state_in), _ptr(state_out), N, T, H, dk, dv,
                                 _dtype_code(q), _ptr(out), _stream(stream)))


def kda_backward_workspace_size(num_seqs: int, total_tokens: int, num_heads: int, dk: int, dv: int,
                                dtype=torch.bfloat16) -> int:
    code = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}.get(dtype)
    if code is None:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32, got %s" % dtype)
    return int(load().kda_backward_workspace_size(num_seqs, total_tokens, num_heads, dk, dv, code))


def kda_backward(q, k, v, g, beta, initial_state, cu_seqlens, dout, dfinal=None, grads=None, want_dinit=True,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of a scalar loss given dout = dL/d(out) [T, H, dv] (q's dtype)
    and dfinal = dL/d(final_state) [N, H, dk, dv] fp32 or None.  Returns a dict
    of fp32 tensors dq, dk, dv, dg [T, H, *], dbeta [T, H] and dinit
    [N, H, dk, dv] (None unless want_dinit); ``grads`` may supply them."""
    N, T, H, dk, dv = _check_prefill_args(q, k, v, g, beta, initial_state, cu_seqlens, dout, None)
    _on_device(q, dfinal=dfinal, workspace=workspace)
    if dfinal is not None:
        _require(dfinal.dtype == torch.float32 and dfinal.is_contiguous() and tuple(dfinal.shape) == (N, H, dk, dv),
                 "dfinal must be contiguous float32 [N, H, dk, dv]")
    dev = q.device
    shapes = {"dq": (T, H, dk), "dk": (T, H, dk), "dv": (T, H, dv), "dg": (T, H, dk), "dbeta": (T, H),
              "dinit": (N, H, dk, dv)}
    if grads is None:
        f = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)
        grads = {key: f(*shape) for key, shape in shapes.items() if key != "dinit"}
        grads["dinit"] = f(*shapes["dinit"]) if want_dinit else None
    for key, shape in shapes.items():
        t = grads.get(key)
        if t is None and key == "dinit":
            continue
        _require(t is not None, "grads[%r] is missing" % key)
        _on_device(q, **{key: t})
        _require(t.dtype == torch.float32 and t.is_contiguous() and tuple(t.shape) == shape,
                 "grads[%r] must be contiguous float32 %s" % (key, list(shape)))
    need = kda_backward_workspace_size(N, T, H, dk, dv, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _require(workspace.is_contiguous(), "workspace must be contiguous")
    nbytes = workspace.numel() * workspace.element_size()
    lib = load()
    _check(lib.kda_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
                            N, T, H, dk, dv, _dtype_code(q), _ptr(dout), _ptr(dfinal), _ptr(grads["dq"]),
                            _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dg"]), _ptr(grads["dbeta"]),
                            _ptr(grads.get("dinit")), _ptr(workspace), nbytes, _stream(stream)))
    return grads


# ---------------------------------------------------------------- layer operators
# One call of these is a few microseconds of GPU time at decode sizes, so the
# checks of a tensor are one expression each (a host tensor's device number is
# -1), the reasons are worked out only when it fails, and pointers and the
# stream go to the library as plain ints.
#
# A call given a `stream` runs there, and tensors that it makes (gradients,
# a workspace) come from that stream's memory: who uses them on another stream
# waits for this one and records the use (Tensor.record_stream), or supplies
# tensors of their own.
_MOST = 2 ** 31 - 1                                # int32 sizes in the C ABI
_DTYPE_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_F32 = torch.float32


def _bad(name, t, dev, dtype, shape) -> None:
    _require(torch.is_tensor(t) and t.is_cuda and t.get_device() == dev, "%s must be a tensor on cuda:%d" % (name, dev))
    _require(t.dtype == dtype, "%s must be %s, got %s" % (name, dtype, t.dtype))
    _require(tuple(t.shape) == tuple(shape), "%s must have shape %s, got %s" % (name, list(shape), list(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _addr(name, t, dev, dtype, shape) -> int:
    """The address of a contiguous tensor of this type and shape on device `dev`, after checking that it is one."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:   # no tensor
        pass
    _bad(name, t, dev, dtype, shape)


def _addr_if(name, t, dev, dtype, shape) -> Optional[int]:
    """As _addr, for an argument that may be None."""
    return None if t is None else _addr(name, t, dev, dtype, shape)


def _rows(name, x):
    """A contiguous device tensor of rows in a supported type: its address, device, type code, shape, rows and row
    length."""
    _require(isinstance(x, torch.Tensor) and x.is_cuda, "%s must be a device tensor" % name)
    code = _DTYPE_CODE.get(x.dtype)
    if code is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, x.dtype))
    shape = x.shape
    if len(shape) == 2:
        rows, D = shape
    else:
        _require(len(shape) > 2, "%s must be [rows, ...channels]" % name)
        rows, D = shape[0], shape[1:].numel()
    if rows > _MOST or D > _MOST or not x.is_contiguous():
        _require(x.is_contiguous(), "%s must be contiguous" % name)
        raise ValueError("%s has too many rows or channels" % name)
    return x.data_ptr(), x.get_device(), code, shape, rows, D


def _cu(cu_seqlens, dev):
    """cu_seqlens' address and the number of sequences."""
    _require(isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.get_device() == dev,
             "cu_seqlens must be a tensor on the inputs' device")
    n = cu_seqlens.numel()
    _require(cu_seqlens.dtype is torch.int32 and cu_seqlens.dim() == 1 and 1 <= n <= _MOST and cu_seqlens.is_contiguous(),
             "cu_seqlens must be contiguous int32 [N + 1]")
    return cu_seqlens.data_ptr(), n - 1


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """A new tensor on device `dev`.  Given another stream than the current one it comes from that stream's pool: what
    the current stream still does with memory freed there is not ordered before the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        # (ExternalStream(0) would be a new stream, not the null stream)
        stream = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


@functools.lru_cache(maxsize=1024)
def _need(query: str, *sizes) -> int:
    """Bytes of workspace, as the library's function `query` says: it goes by the sizes alone."""
    return getattr(load(), query)(*sizes)


def _workspace(workspace, dev, stream, query, *sizes):
    """The given workspace, or a new one of the size that `query` says: (tensor, address, bytes)."""
    if workspace is None:
        need = _need(query, *sizes)
        if need == 0:
            return None, None, 0
        workspace = _empty(need, torch.uint8, dev, stream)
        return workspace, workspace.data_ptr(), need
    _require(isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and workspace.is_contiguous(),
             "workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _call(fn, dev, stream, *args) -> None:
    """fn(*args, stream) with device `dev` current; stream None: that device's current stream."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, *args)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    status = fn(*args, raw)
    if status != KDA_OK:
        _check(status)


def kda_scan_workspace_size(num_seqs: int, total_tokens: int, channels: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace kda_scan_prefill needs."""
    return int(load().kda_scan_workspace_size(num_seqs, total_tokens, channels, _code(dtype)))


def _code(dtype) -> int:
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32, got %s" % dtype)
    return code


def kda_scan_prefill(x, g, initial_state, cu_seqlens, out, final_state, checkpoints=None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over packed
    sequences.  x, out: [T, ...channels]; g: the same shape, fp32;
    initial_state / final_state: [N, ...channels] fp32 or None; checkpoints:
    [ceil(T / 128), ...channels] fp32 or None, the states kda_scan_backward
    starts from; workspace: kda_scan_workspace_size(...) bytes, allocated if
    None."""
    px, dev, code, shape, T, D = _rows("x", x)
    pcu, N = _cu(cu_seqlens, dev)
    state = (N, *shape[1:])
    lib = _lib or load()
    args = (px, _addr("g", g, dev, _F32, shape), _addr_if("initial_state", initial_state, dev, _F32, state), pcu, N, T, D,
            code, _addr("out", out, dev, x.dtype, shape), _addr_if("final_state", final_state, dev, _F32, state),
            _addr_if("checkpoints", checkpoints, dev, _F32, (-(-T // KDA_SCAN_TILE), *shape[1:])))
    ws, pws, nbytes = _workspace(workspace, dev, stream, "kda_scan_workspace_size", N, T, D, code)
    _call(lib.kda_scan_prefill, dev, stream, *args, pws, nbytes)


def kda_scan_decode_step(x, g, state_inout, out, stream=None) -> None:
    """One token per sequence, state updated in place.  x, out: [N, ...channels];
    g, state_inout: the same shape, fp32."""
    px, dev, code, shape, N, D = _rows("x", x)
    _call((_lib or load()).kda_scan_decode_step, dev, stream, px, _addr("g", g, dev, _F32, shape),
          _addr("state_inout", state_inout, dev, _F32, shape), N, D, code, _addr("out", out, dev, x.dtype, shape))


def kda_scan_backward_workspace_size(num_seqs: int, total_tokens: int, channels: int, dtype=torch.bfloat16,
                                     has_checkpoints: bool = False) -> int:
    """Bytes of workspace kda_scan_backward needs."""
    return int(load().kda_scan_backward_workspace_size(num_seqs, total_tokens, channels, _code(dtype),
                                                       int(has_checkpoints)))


def _grads(given, dev, want, stream) -> dict:
    """The gradients' tensors: those given, or new ones.  want: name -> (dtype, shape), or None (left out)."""
    if given is None:
        return {name: None if w is None else _empty(w[1], w[0], dev, stream) for name, w in want.items()}
    return given


def kda_scan_backward(x, g, initial_state, cu_seqlens, dout, dfinal=None, checkpoints=None, grads=None,
                      want_dinit: bool = True, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of kda_scan_prefill given dout [T, ...channels] (x's type) and
    dfinal [N, ...channels] fp32 or None.  ``checkpoints`` are those
    kda_scan_prefill wrote for the same inputs; without them the states are
    computed again.  Returns a dict of dx (x's type), dg (fp32) and dinit (fp32;
    None unless want_dinit); ``grads`` may supply the tensors, which otherwise
    belong to ``stream`` (record_stream them for use on another)."""
    px, dev, code, shape, T, D = _rows("x", x)
    pcu, N = _cu(cu_seqlens, dev)
    dt, state = x.dtype, (N, *shape[1:])
    lib = _lib or load()
    grads = _grads(grads, dev, {"dx": (dt, shape), "dg": (_F32, shape), "dinit": (_F32, state) if want_dinit else None},
                   stream)
    args = (px, _addr("g", g, dev, _F32, shape), _addr_if("initial_state", initial_state, dev, _F32, state), pcu, N, T, D,
            code, _addr("dout", dout, dev, dt, shape), _addr_if("dfinal", dfinal, dev, _F32, state),
            _addr_if("checkpoints", checkpoints, dev, _F32, (-(-T // KDA_SCAN_TILE), *shape[1:])),
            _addr("grads['dx']", grads.get("dx"), dev, dt, shape), _addr("grads['dg']", grads.get("dg"), dev, _F32, shape),
            _addr_if("grads['dinit']", grads.get("dinit"), dev, _F32, state))
    ws, pws, nbytes = _workspace(workspace, dev, stream, "kda_scan_backward_workspace_size", N, T, D, code,
                                 int(checkpoints is not None))
    _call(lib.kda_scan_backward, dev, stream, *args, pws, nbytes)
    return grads


def _conv_weight(weight, dev, shape):
    """The weight's address and width: [...channels, width] fp32 for rows of this shape."""
    _require(isinstance(weight, torch.Tensor) and weight.dim() == len(shape), "weight must be [...channels, width]")
    W = weight.shape[-1]
    return _addr("weight", weight, dev, _F32, (*shape[1:], W)), W


def kda_conv_prefill(x, weight, bias, initial_state, cu_seqlens, out, final_state, silu: bool = True,
                     stream=None) -> None:
    """Short causal convolution over packed sequences, with SiLU unless silu is
    False.  x, out: [T, ...channels]; weight: [...channels, width] fp32, width 2
    to 4; bias: [...channels] fp32 or None; initial_state / final_state:
    [N, width - 1, ...channels] of x's type or None."""
    px, dev, code, shape, T, D = _rows("x", x)
    pcu, N = _cu(cu_seqlens, dev)
    pw, W = _conv_weight(weight, dev, shape)
    dt, state = x.dtype, (N, W - 1, *shape[1:])
    _call((_lib or load()).kda_conv_prefill, dev, stream, px, pw, _addr_if("bias", bias, dev, _F32, shape[1:]),
          _addr_if("initial_state", initial_state, dev, dt, state), pcu, N, T, D, W, int(silu), code,
          _addr("out", out, dev, dt, shape), _addr_if("final_state", final_state, dev, dt, state))


def kda_conv_decode_step(x, weight, bias, state_inout, out, silu: bool = True, stream=None) -> None:
    """One token per sequence, state shifted in place.  x, out: [N, ...channels];
    state_inout: [N, width - 1, ...channels] of x's type."""
    px, dev, code, shape, N, D = _rows("x", x)
    pw, W = _conv_weight(weight, dev, shape)
    _call((_lib or load()).kda_conv_decode_step, dev, stream, px, pw, _addr_if("bias", bias, dev, _F32, shape[1:]),
          _addr("state_inout", state_inout, dev, x.dtype, (N, W - 1, *shape[1:])), N, D, W, int(silu), code,
          _addr("out", out, dev, x.dtype, shape))


def kda_conv_backward_workspace_size(num_seqs: int, total_tokens: int, channels: int, width: int,
                                     dtype=torch.bfloat16) -> int:
    """Bytes of workspace kda_conv_backward needs."""
    return int(load().kda_conv_backward_workspace_size(num_seqs, total_tokens, channels, width, _code(dtype)))


def kda_conv_backward(x, weight, bias, initial_state, cu_seqlens, dout, dfinal=None, silu: bool = True, grads=None,
                      want_dinit: bool = True, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of kda_conv_prefill given dout [T, ...channels] and dfinal
    [N, width - 1, ...channels] (x's type) or None.  Returns a dict of dx and
    dinit (x's type; dinit None unless want_dinit), dweight and dbias (fp32;
    dbias None without a bias); ``grads`` may supply the tensors, which otherwise
    belong to ``stream`` (record_stream them for use on another)."""
    px, dev, code, shape, T, D = _rows("x", x)
    pcu, N = _cu(cu_seqlens, dev)
    pw, W = _conv_weight(weight, dev, shape)
    dt, row, state = x.dtype, shape[1:], (N, W - 1, *shape[1:])
    lib = _lib or load()
    grads = _grads(grads, dev, {"dx": (dt, shape), "dweight": (_F32, (*row, W)),
                              "dbias": None if bias is None else (_F32, row),
                              "dinit": (dt, state) if want_dinit else None}, stream)
    args = (px, pw, _addr_if("bias", bias, dev, _F32, row), _addr_if("initial_state", initial_state, dev, dt, state), pcu,
            N, T, D, W, int(silu), code, _addr("dout", dout, dev, dt, shape), _addr_if("dfinal", dfinal, dev, dt, state),
            _addr("grads['dx']", grads.get("dx"), dev, dt, shape),
            _addr("grads['dweight']", grads.get("dweight"), dev, _F32, (*row, W)),
            _addr_if("grads['dbias']", grads.get("dbias"), dev, _F32, row),
            _addr_if("grads['dinit']", grads.get("dinit"), dev, dt, state))
    ws, pws, nbytes = _workspace(workspace, dev, stream, "kda_conv_backward_workspace_size", N, T, D, W, code)
    _call(lib.kda_conv_backward, dev, stream, *args, pws, nbytes)
    return grads


def _norm_rows(name, x):
    """As _rows, for tensors whose rows are their last dimension."""
    _require(isinstance(x, torch.Tensor) and x.is_cuda, "%s must be a device tensor" % name)
    code = _DTYPE_CODE.get(x.dtype)
    if code is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, x.dtype))
    shape = x.shape
    D = shape[-1] if shape else 0
    _require(D > 0 and x.is_contiguous(), "%s must be contiguous, [..., channels]" % name)
    rows = shape[0] if len(shape) == 2 else x.numel() // D
    _require(rows <= _MOST and D <= _MOST, "%s has too many rows or channels" % name)
    return x.data_ptr(), x.get_device(), code, shape, rows, D


def kda_rmsnorm(x, weight, out=None, residual=None, residual_out=None, out_mx=None, scales=None, eps: float = 1e-6,
                stream=None) -> None:
    """r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight over the last
    dimension.  x, residual, residual_out (r), out (y): [..., channels] of one
    type; weight: [channels] fp32 or None.  out_mx: [..., channels] uint8 or
    float8_e4m3fn and scales: [..., ceil(channels / 32)] uint8 or
    float8_e8m0fnu, y in 8 bits with a power-of-two scale for every 32
    channels."""
    px, dev, code, shape, rows, D = _norm_rows("x", x)
    dt = x.dtype
    mx = sc = None
    if out_mx is not None or scales is not None:
        _require(isinstance(out_mx, torch.Tensor) and isinstance(scales, torch.Tensor),
                 "out_mx and scales go together")
        mx = _addr("out_mx", out_mx, dev, torch.uint8 if out_mx.dtype is torch.uint8 else torch.float8_e4m3fn, shape)
        sc = _addr("scales", scales, dev, torch.uint8 if scales.dtype is torch.uint8 else torch.float8_e8m0fnu,
                   (*shape[:-1], -(-D // KDA_MX_BLOCK)))
    _call((_lib or load()).kda_rmsnorm, dev, stream, px, _addr_if("residual", residual, dev, dt, shape),
          _addr_if("weight", weight, dev, _F32, (D,)), rows, D, eps, code,
          _addr_if("residual_out", residual_out, dev, dt, shape), _addr_if("out", out, dev, dt, shape), mx, sc)


def kda_rmsnorm_backward_workspace_size(rows: int, channels: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace kda_rmsnorm_backward needs."""
    return int(load().kda_rmsnorm_backward_workspace_size(rows, channels, _code(dtype)))


def kda_rmsnorm_backward(x, weight, dout, dresidual=None, eps: float = 1e-6, grads=None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of kda_rmsnorm's y given the normed rows x (its residual_out,
    where it added one) and dout; dresidual, a gradient of x from elsewhere, is
    added.  Returns a dict of dx (x's type) and dweight (fp32; None without a
    weight); ``grads`` may supply the tensors, which otherwise belong to
    ``stream`` (record_stream them for use on another)."""
    px, dev, code, shape, rows, D = _norm_rows("x", x)
    dt = x.dtype
    lib = _lib or load()
    grads = _grads(grads, dev, {"dx": (dt, shape), "dweight": None if weight is None else (_F32, (D,))}, stream)
    pdw = _addr_if("grads['dweight']", grads.get("dweight"), dev, _F32, (D,))
    args = (px, _addr_if("weight", weight, dev, _F32, (D,)), _addr("dout", dout, dev, dt, shape),
            _addr_if("dresidual", dresidual, dev, dt, shape), rows, D, eps, code,
            _addr("grads['dx']", grads.get("dx"), dev, dt, shape), pdw)
    ws = pws = None
    nbytes = 0
    if pdw is not None:
        ws, pws, nbytes = _workspace(workspace, dev, stream, "kda_rmsnorm_backward_workspace_size", rows, D, code)
    _call(lib.kda_rmsnorm_backward, dev, stream, *args, pws, nbytes)
    return grads
