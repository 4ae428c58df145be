"""Thin ctypes binding of ``libkda.so`` (the C ABI in ``include/kda.h``).

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream, and every step of the computation runs in the library's
kernels.  Importing this module loads the library and raises ``ImportError``
when it has not been built (``python -m gated_delta_rule_kda_gb300.build``):
there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional

import torch

from .build import LIB as _LIB_PATH

KDA_OK = 0
KDA_BF16 = 0
KDA_FP32 = 1
HEAD_DIM = 128
DEFAULT_SCALE = 1.0 / math.sqrt(128.0)

STATUS_NAMES = {
    0: "KDA_OK",
    1: "KDA_ERR_INVALID_ARGUMENT",
    2: "KDA_ERR_UNSUPPORTED",
    3: "KDA_ERR_WORKSPACE",
    4: "KDA_ERR_CUDA",
    5: "KDA_ERR_DEVICE_TIMEOUT",
    6: "KDA_ERR_DEVICE_CHECK",
}

# Every entry point include/kda.h declares (checked by tests on CPU).
EXPORTED = (
    "kda_status_string",
    "kda_version",
    "kda_prefill_workspace_size",
    "kda_prefill",
    "kda_prefill_with_checkpoints",
    "kda_prefill_head_decay",
    "kda_prefill_unbounded_decay",
    "kda_decode_step",
    "kda_decode_step_head_decay",
    "kda_frontend",
    "kda_frontend_unbounded_decay",
    "kda_output_gate",
    "kda_layer_core_workspace_size",
    "kda_layer_core",
    "kda_layer_core_unbounded_decay",
    "kda_layer_core_noalloc",
    "kda_layer_core_fused",
    "kda_layer_core_fused_unbounded_decay",
    "kda_layer_core_fused_with_checkpoints",
    "kda_decode_layer",
    "kda_decode_tokens",
    "kda_decode_layer_tokens",
    "kda_qk_norm_rope",
    "kda_qk_norm_rope_append",
    "kda_window_attention",
    "kda_pages_copy",
    "kda_pages_workspace_size",
    "kda_pages_fork",
    "kda_pages_release",
    "kda_pages_compact",
    "kda_check_prefill_inputs",
    "kda_get_device_status",
    "kda_debug_inject_handoff_timeout",
    "kda_debug_inject_attention_timeout",
)

# Capacity of the fixed scratch array behind kda_layer_core_noalloc (include/kda.h).
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


class KdaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libkda.so is not built ({_LIB_PATH}); run "
                          "`python -m gated_delta_rule_kda_gb300.build` first")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I32, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                          ctypes.c_size_t)
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = I32
    lib.kda_prefill_workspace_size.argtypes = [I32, I32, I32, ctypes.c_int]
    lib.kda_prefill_workspace_size.restype = SZ
    lib.kda_prefill.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, I32, P, P, P, P, P, P, P,
                                F, P, P, P, SZ, P]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill_with_checkpoints.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, I32, P, P,
                                                 P, P, P, P, P, F, P, P, P, SZ, I32, P, P, P]
    lib.kda_prefill_with_checkpoints.restype = ctypes.c_int
    lib.kda_prefill_head_decay.argtypes = lib.kda_prefill_with_checkpoints.argtypes
    lib.kda_prefill_head_decay.restype = ctypes.c_int
    lib.kda_prefill_unbounded_decay.argtypes = lib.kda_prefill.argtypes
    lib.kda_prefill_unbounded_decay.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, P, P, P, P, P, P, F,
                                    P, P]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step_head_decay.argtypes = lib.kda_decode_step.argtypes
    lib.kda_decode_step_head_decay.restype = ctypes.c_int
    lib.kda_frontend.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, P, F, ctypes.c_int,
                                 P, P, P, P, P, P]
    lib.kda_frontend.restype = ctypes.c_int
    lib.kda_frontend_unbounded_decay.argtypes = lib.kda_frontend.argtypes
    lib.kda_frontend_unbounded_decay.restype = ctypes.c_int
    lib.kda_output_gate.argtypes = [I64, ctypes.c_int, P, P, F, ctypes.c_int, P, P]
    lib.kda_output_gate.restype = ctypes.c_int
    lib.kda_layer_core_workspace_size.argtypes = [I32, I32, I32]
    lib.kda_layer_core_workspace_size.restype = SZ
    lib.kda_layer_core.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, F, F, F,
                                   ctypes.c_int, P, P, P, SZ, P]
    lib.kda_layer_core.restype = ctypes.c_int
    lib.kda_layer_core_unbounded_decay.argtypes = lib.kda_layer_core.argtypes
    lib.kda_layer_core_unbounded_decay.restype = ctypes.c_int
    lib.kda_layer_core_noalloc.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, F, F,
                                           F, ctypes.c_int, P, P, P]
    lib.kda_layer_core_noalloc.restype = ctypes.c_int
    lib.kda_layer_core_fused.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, F, F,
                                         F, ctypes.c_int, P, P, P]
    lib.kda_layer_core_fused.restype = ctypes.c_int
    lib.kda_layer_core_fused_unbounded_decay.argtypes = lib.kda_layer_core_fused.argtypes
    lib.kda_layer_core_fused_unbounded_decay.restype = ctypes.c_int
    lib.kda_layer_core_fused_with_checkpoints.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P,
                                                          P, P, P, F, F, F, ctypes.c_int, P, P,
                                                          I32, P, P, P]
    lib.kda_layer_core_fused_with_checkpoints.restype = ctypes.c_int
    lib.kda_decode_layer.argtypes = [I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, P, F, F, F,
                                     ctypes.c_int, P, P]
    lib.kda_decode_layer.restype = ctypes.c_int
    lib.kda_decode_tokens.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, I32, I32, P, P, P, P,
                                      P, P, P, P, I32, P, F, P, P]
    lib.kda_decode_tokens.restype = ctypes.c_int
    lib.kda_decode_layer_tokens.argtypes = [I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P,
                                            P, P, I32, F, F, F, ctypes.c_int, P, P]
    lib.kda_decode_layer_tokens.restype = ctypes.c_int
    lib.kda_qk_norm_rope.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, I32, P, I64, P, I64, P, P,
                                     F, I32, P, I32, I32, I32, P, P, P, P]
    lib.kda_qk_norm_rope.restype = ctypes.c_int
    lib.kda_qk_norm_rope_append.argtypes = [ctypes.c_int, ctypes.c_int, I32, I32, I32, I32, P, I64,
                                            P, I64, P, I64, P, P, F, I32, P, I32, I32, I32, P, I32,
                                            I32, I32, I32, P, P, P, P, P, P, P]
    lib.kda_qk_norm_rope_append.restype = ctypes.c_int
    lib.kda_window_attention.argtypes = [ctypes.c_int] + [I32] * 11 + [P] * 6 + [F, P, P]
    lib.kda_window_attention.restype = ctypes.c_int
    lib.kda_pages_copy.argtypes = [I32, I32, I64, I32, P, P, P, P]
    lib.kda_pages_copy.restype = ctypes.c_int
    lib.kda_pages_workspace_size.argtypes = [I32, I32]
    lib.kda_pages_workspace_size.restype = SZ
    lib.kda_pages_fork.argtypes = [I32, I32, I64, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P]
    lib.kda_pages_fork.restype = ctypes.c_int
    lib.kda_pages_release.argtypes = [I32, I32, I32, I32, P, I32, I32, P, P, P]
    lib.kda_pages_release.restype = ctypes.c_int
    lib.kda_pages_compact.argtypes = [I32, I32, I64, I32, I32, P, P, P, P, P, SZ, P]
    lib.kda_pages_compact.restype = ctypes.c_int
    lib.kda_check_prefill_inputs.argtypes = [I32, I32, I32, P, I32, P, P]
    lib.kda_check_prefill_inputs.restype = ctypes.c_int
    lib.kda_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.kda_get_device_status.restype = ctypes.c_int
    lib.kda_debug_inject_handoff_timeout.argtypes = []
    lib.kda_debug_inject_handoff_timeout.restype = ctypes.c_int
    lib.kda_debug_inject_attention_timeout.argtypes = []
    lib.kda_debug_inject_attention_timeout.restype = ctypes.c_int
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def library_path() -> str:
    return _LIB_PATH


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dtype_code(d: torch.dtype) -> int:
    return KDA_BF16 if d == torch.bfloat16 else KDA_FP32


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# What a call allocates belongs to the stream that it launches on: a block of the current stream's would
# be handed out again at once when the caller drops it (a workspace: when the call returns), while the
# other stream's kernels still use it.
def _on(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _kept(t: torch.Tensor, stream) -> torch.Tensor:
    """t, allocated for `stream`, not handed out again before what the caller's stream does with it is done."""
    if stream is not None and t.is_cuda:
        current = torch.cuda.current_stream(t.device)
        if current != stream:
            t.record_stream(current)
    return t


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    return _kept(t, stream)


def _check(fn: str, rc: int):
    if rc != KDA_OK:
        raise KdaError(fn, rc)


def kda_prefill_workspace_size(num_seqs: int, total_tokens: int, num_heads: int,
                               in_dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_lib.kda_prefill_workspace_size(num_seqs, total_tokens, num_heads,
                                               _dtype_code(in_dtype)))


def kda_prefill(q, k, v, log_alpha, beta, cu_seqlens, S0=None, scale=DEFAULT_SCALE, *,
                out_dtype=None, o=None, S_final=None, want_state=True, workspace=None,
                stream=None, _entry="kda_prefill"):
    """Packed-varlen prefill.  Returns (o, S_final or None).

    q, k, v [T, H, 128] (bf16 or fp32); log_alpha [T, H, 128] fp32; beta [T, H] fp32;
    cu_seqlens [N+1] int32 (device); S0 [N, H, 128, 128] fp32 or None.
    S_final may be S0 itself (in-place resume)."""
    T, H, _ = q.shape
    N = cu_seqlens.shape[0] - 1
    out_dtype = out_dtype or q.dtype
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, q.device, stream)
    if S_final is None and want_state:
        S_final = _empty((N, H, HEAD_DIM, HEAD_DIM), torch.float32, q.device, stream)
    need = kda_prefill_workspace_size(N, T, H, q.dtype)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = getattr(_lib, _entry)(_dt(q), _dtype_code(o.dtype), N, T, H, _p(q), _p(k), _p(v),
                          _p(log_alpha), _p(beta), _p(S0), _p(cu_seqlens), float(scale), _p(o),
                          _p(S_final), _p(workspace), wbytes, _stream(stream))
    _check(_entry, rc)
    return o, S_final


def kda_prefill_unbounded_decay(q, k, v, log_alpha, beta, cu_seqlens, S0=None,
                                scale=DEFAULT_SCALE, **kw):
    """kda_prefill for any log_alpha <= 0 (-inf included) on the token-by-token kernel."""
    return kda_prefill(q, k, v, log_alpha, beta, cu_seqlens, S0, scale,
                       _entry="kda_prefill_unbounded_decay", **kw)


def checkpoint_offsets(cu_seqlens, every: int) -> torch.Tensor:
    """Snapshot offsets [N+1] int32 (host) for one snapshot per `every` tokens of each
    sequence: base[n+1] - base[n] = len_n // every."""
    cu = torch.as_tensor(cu_seqlens).to("cpu", torch.int64)
    counts = torch.div(cu[1:] - cu[:-1], every, rounding_mode="floor")
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)


def _checkpoint_args(cu_seqlens, H, every, ckpt_base, ckpt_states, device, stream):
    with _on(stream):  # the offsets are read, and uploaded, in the order of the call's stream
        base = checkpoint_offsets(cu_seqlens, every).to(device) if ckpt_base is None else ckpt_base
        total = int(base[-1]) if ckpt_states is None else 0
    if ckpt_base is None:
        ckpt_base = _kept(base, stream)
    if ckpt_states is None:
        ckpt_states = _empty((total, H, HEAD_DIM, HEAD_DIM), torch.float32, device, stream)
    return ckpt_base, ckpt_states


def kda_prefill_with_checkpoints(q, k, v, log_alpha, beta, cu_seqlens, every, S0=None,
                                 scale=DEFAULT_SCALE, *, ckpt_base=None, ckpt_states=None,
                                 out_dtype=None, o=None, S_final=None, want_state=True,
                                 workspace=None, stream=None, _entry="kda_prefill_with_checkpoints"):
    """kda_prefill that also writes the state after every `every` tokens of each sequence
    (every: a positive multiple of 32).  ckpt_base [N+1] int32 (device) defaults to
    checkpoint_offsets(cu_seqlens, every).  Returns (o, S_final, ckpt_base, ckpt_states)."""
    T, H, _ = q.shape
    N = cu_seqlens.shape[0] - 1
    out_dtype = out_dtype or q.dtype
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, q.device, stream)
    if S_final is None and want_state:
        S_final = _empty((N, H, HEAD_DIM, HEAD_DIM), torch.float32, q.device, stream)
    if every:
        ckpt_base, ckpt_states = _checkpoint_args(cu_seqlens, H, every, ckpt_base, ckpt_states,
                                                  q.device, stream)
    need = kda_prefill_workspace_size(N, T, H, q.dtype)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = getattr(_lib, _entry)(
        _dt(q), _dtype_code(o.dtype), N, T, H, _p(q), _p(k), _p(v), _p(log_alpha), _p(beta),
        _p(S0), _p(cu_seqlens), float(scale), _p(o), _p(S_final), _p(workspace), wbytes,
        int(every), _p(ckpt_base), _p(ckpt_states), _stream(stream))
    _check(_entry, rc)
    return o, S_final, ckpt_base, ckpt_states


def kda_prefill_head_decay(q, k, v, log_alpha, beta, cu_seqlens, S0=None, scale=DEFAULT_SCALE, *,
                           every=0, ckpt_base=None, ckpt_states=None, out_dtype=None, o=None,
                           S_final=None, want_state=True, workspace=None, stream=None):
    """The Gated DeltaNet case: log_alpha [T, H] fp32, one decay per (token, head).
    Returns (o, S_final, ckpt_base, ckpt_states) (the last two None without snapshots)."""
    return kda_prefill_with_checkpoints(q, k, v, log_alpha, beta, cu_seqlens, every, S0, scale,
                                        ckpt_base=ckpt_base, ckpt_states=ckpt_states,
                                        out_dtype=out_dtype, o=o, S_final=S_final,
                                        want_state=want_state, workspace=workspace, stream=stream,
                                        _entry="kda_prefill_head_decay")


def kda_decode_step(q, k, v, log_alpha, beta, S_inout, scale=DEFAULT_SCALE, *, out_dtype=None,
                    o=None, stream=None, _entry="kda_decode_step"):
    """One decode step; S_inout [B, H, 128, 128] fp32 is updated in place.  Returns o."""
    B, H, _ = q.shape
    out_dtype = out_dtype or q.dtype
    if o is None:
        o = _empty((B, H, HEAD_DIM), out_dtype, q.device, stream)
    rc = getattr(_lib, _entry)(_dt(q), _dtype_code(o.dtype), B, H, _p(q), _p(k), _p(v),
                               _p(log_alpha), _p(beta), _p(S_inout), float(scale), _p(o),
                               _stream(stream))
    _check(_entry, rc)
    return o


def kda_decode_step_head_decay(q, k, v, log_alpha, beta, S_inout, scale=DEFAULT_SCALE, *,
                               out_dtype=None, o=None, stream=None):
    """kda_decode_step with log_alpha [B, H] fp32 (one decay per request and head)."""
    return kda_decode_step(q, k, v, log_alpha, beta, S_inout, scale, out_dtype=out_dtype, o=o,
                           stream=stream, _entry="kda_decode_step_head_decay")


def kda_frontend(qp, kp, vp, conv_w, z, A, b, beta_logit, cu_seqlens, l2_eps=1e-6, *,
                 out_dtype=torch.bfloat16, stream=None, _entry="kda_frontend"):
    """Returns (q_hat, k_hat, v, log_alpha, beta)."""
    T, H, _ = qp.shape
    N = cu_seqlens.shape[0] - 1
    dev = qp.device
    q_hat = _empty((T, H, HEAD_DIM), out_dtype, dev, stream)
    k_hat = _empty(q_hat.shape, out_dtype, dev, stream)
    v_out = _empty(q_hat.shape, out_dtype, dev, stream)
    log_alpha = _empty((T, H, HEAD_DIM), torch.float32, dev, stream)
    beta = _empty((T, H), torch.float32, dev, stream)
    rc = getattr(_lib, _entry)(N, T, H, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A), _p(b),
                           _p(beta_logit), _p(cu_seqlens), float(l2_eps),
                           _dtype_code(out_dtype), _p(q_hat), _p(k_hat), _p(v_out),
                           _p(log_alpha), _p(beta), _stream(stream))
    _check(_entry, rc)
    return q_hat, k_hat, v_out, log_alpha, beta


def kda_frontend_unbounded_decay(qp, kp, vp, conv_w, z, A, b, beta_logit, cu_seqlens, l2_eps=1e-6,
                                 **kw):
    """kda_frontend with Kimi Linear's gate log_alpha = -e^A softplus(z + b)."""
    return kda_frontend(qp, kp, vp, conv_w, z, A, b, beta_logit, cu_seqlens, l2_eps,
                        _entry="kda_frontend_unbounded_decay", **kw)


def kda_output_gate(o_tilde, g, eps=1e-6, *, out_dtype=torch.bfloat16, out=None, stream=None):
    rows = o_tilde.numel() // HEAD_DIM
    if out is None:
        out = _empty(o_tilde.shape, out_dtype, o_tilde.device, stream)
    rc = _lib.kda_output_gate(rows, _dt(o_tilde), _p(o_tilde), _p(g), float(eps),
                              _dtype_code(out.dtype), _p(out), _stream(stream))
    _check("kda_output_gate", rc)
    return out


def kda_layer_core_workspace_size(num_seqs: int, total_tokens: int, num_heads: int) -> int:
    return int(_lib.kda_layer_core_workspace_size(num_seqs, total_tokens, num_heads))


def kda_layer_core(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0=None,
                   scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6, *, out_dtype=torch.bfloat16,
                   o=None, S_final=None, want_state=True, workspace=None, stream=None,
                   _entry="kda_layer_core"):
    """Front end -> recurrence -> output gate.  Returns (o_gated, S_final or None)."""
    T, H, _ = qp.shape
    N = cu_seqlens.shape[0] - 1
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, qp.device, stream)
    if S_final is None and want_state:
        S_final = _empty((N, H, HEAD_DIM, HEAD_DIM), torch.float32, qp.device, stream)
    need = kda_layer_core_workspace_size(N, T, H)
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, qp.device, stream)
    wbytes = workspace.numel() * workspace.element_size()
    rc = getattr(_lib, _entry)(N, T, H, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A), _p(b),
                             _p(beta_logit), _p(g), _p(cu_seqlens), _p(S0), float(scale),
                             float(l2_eps), float(rms_eps), _dtype_code(o.dtype), _p(o),
                             _p(S_final), _p(workspace), wbytes, _stream(stream))
    _check(_entry, rc)
    return o, S_final


def kda_layer_core_unbounded_decay(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0=None,
                                   **kw):
    """kda_layer_core with Kimi Linear's unbounded decay gate (staged, fp32 intermediates)."""
    return kda_layer_core(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0,
                          _entry="kda_layer_core_unbounded_decay", **kw)


def kda_layer_core_noalloc(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0=None,
                           scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6, *, o, S_final=None,
                           stream=None):
    """kda_layer_core for callers that cannot allocate device memory: the library
    supplies the scratch from a fixed array of NOALLOC_SCRATCH_BYTES bytes.
    `o` (and `S_final` if wanted) must be provided by the caller; nothing is
    allocated here.  Calls that overlap on the GPU race on the shared scratch."""
    T, H, _ = qp.shape
    N = cu_seqlens.shape[0] - 1
    rc = _lib.kda_layer_core_noalloc(N, T, H, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A),
                                     _p(b), _p(beta_logit), _p(g), _p(cu_seqlens), _p(S0),
                                     float(scale), float(l2_eps), float(rms_eps),
                                     _dtype_code(o.dtype), _p(o), _p(S_final), _stream(stream))
    _check("kda_layer_core_noalloc", rc)
    return o, S_final


def kda_layer_core_fused(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0=None,
                         scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6, *,
                         out_dtype=torch.bfloat16, o=None, S_final=None, want_state=True,
                         stream=None, _entry="kda_layer_core_fused"):
    """The layer core in one tensor-core kernel.  Returns (o_gated, S_final or None)."""
    T, H, _ = qp.shape
    N = cu_seqlens.shape[0] - 1
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, qp.device, stream)
    if S_final is None and want_state:
        S_final = _empty((N, H, HEAD_DIM, HEAD_DIM), torch.float32, qp.device, stream)
    rc = getattr(_lib, _entry)(N, T, H, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A),
                               _p(b), _p(beta_logit), _p(g), _p(cu_seqlens), _p(S0),
                               float(scale), float(l2_eps), float(rms_eps),
                               _dtype_code(o.dtype), _p(o), _p(S_final), _stream(stream))
    _check(_entry, rc)
    return o, S_final


def kda_layer_core_fused_unbounded_decay(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens,
                                         S0=None, scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6,
                                         *, out_dtype=torch.bfloat16, o=None, S_final=None,
                                         want_state=True, stream=None):
    """kda_layer_core_fused with Kimi Linear's decay gate -e^A softplus(z + b) (no floor)."""
    return kda_layer_core_fused(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens, S0,
                                scale, l2_eps, rms_eps, out_dtype=out_dtype, o=o,
                                S_final=S_final, want_state=want_state, stream=stream,
                                _entry="kda_layer_core_fused_unbounded_decay")


def kda_layer_core_fused_with_checkpoints(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_seqlens,
                                          every, S0=None, scale=DEFAULT_SCALE, l2_eps=1e-6,
                                          rms_eps=1e-6, *, ckpt_base=None, ckpt_states=None,
                                          out_dtype=torch.bfloat16, o=None, S_final=None,
                                          want_state=True, stream=None):
    """kda_layer_core_fused that also writes the recurrent state after every `every` tokens
    of each sequence.  Returns (o_gated, S_final, ckpt_base, ckpt_states)."""
    T, H, _ = qp.shape
    N = cu_seqlens.shape[0] - 1
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, qp.device, stream)
    if S_final is None and want_state:
        S_final = _empty((N, H, HEAD_DIM, HEAD_DIM), torch.float32, qp.device, stream)
    ckpt_base, ckpt_states = _checkpoint_args(cu_seqlens, H, every, ckpt_base, ckpt_states,
                                              qp.device, stream)
    rc = _lib.kda_layer_core_fused_with_checkpoints(
        N, T, H, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A), _p(b), _p(beta_logit), _p(g),
        _p(cu_seqlens), _p(S0), float(scale), float(l2_eps), float(rms_eps),
        _dtype_code(o.dtype), _p(o), _p(S_final), int(every), _p(ckpt_base), _p(ckpt_states),
        _stream(stream))
    _check("kda_layer_core_fused_with_checkpoints", rc)
    return o, S_final, ckpt_base, ckpt_states


def kda_decode_layer(qp, kp, vp, conv_w, z, A, b, beta_logit, g, slot, S_pool, conv_pool,
                     scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6, *, out_dtype=torch.bfloat16,
                     o=None, stream=None):
    """One decode step of the layer core for requests whose states sit in pools.

    qp, kp, vp, z, g: [B, H, 128] bf16; beta_logit: [B, H] bf16; slot: [B] int32 (distinct
    pool rows); S_pool: [P, H, 128, 128] fp32 and conv_pool: [P, 3, 3, H, 128] bf16, both
    updated in place.  Returns o [B, H, 128].
    """
    B, H, _ = qp.shape
    P = S_pool.shape[0]
    if o is None:
        o = _empty((B, H, HEAD_DIM), out_dtype, qp.device, stream)
    rc = _lib.kda_decode_layer(B, H, P, _p(qp), _p(kp), _p(vp), _p(conv_w), _p(z), _p(A), _p(b),
                               _p(beta_logit), _p(g), _p(slot), _p(S_pool), _p(conv_pool),
                               float(scale), float(l2_eps), float(rms_eps), _dtype_code(o.dtype),
                               _p(o), _stream(stream))
    _check("kda_decode_layer", rc)
    return o


def kda_decode_tokens(q, k, v, log_alpha, beta, cu_tokens, slot, S_pool, write_back,
                      scale=DEFAULT_SCALE, *, S_final=None, out_dtype=None, o=None, stream=None):
    """A few tokens per request from pool rows (speculative verify: write_back=False;
    replay of accepted tokens: write_back=True).  q, k, v [T, H, 128]; log_alpha
    [T, H, 128] fp32; beta [T, H] fp32; cu_tokens [B+1] int32 and slot [B] int32 (device);
    S_pool [P, H, 128, 128] fp32.  Returns o [T, H, 128]."""
    T, H, _ = q.shape
    B = slot.shape[0]
    P = S_pool.shape[0]
    out_dtype = out_dtype or q.dtype
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, q.device, stream)
    rc = _lib.kda_decode_tokens(_dt(q), _dtype_code(o.dtype), B, H, P, T, _p(cu_tokens),
                                _p(slot), _p(q), _p(k), _p(v), _p(log_alpha), _p(beta),
                                _p(S_pool), int(bool(write_back)), _p(S_final), float(scale),
                                _p(o), _stream(stream))
    _check("kda_decode_tokens", rc)
    return o


DECODE_LAYER_MAX_TOKENS = 16  # KDA_DECODE_LAYER_MAX_TOKENS in include/kda.h


def kda_decode_layer_tokens(qp, kp, vp, conv_w, z, A, b, beta_logit, g, cu_tokens, slot, S_pool,
                            conv_pool, write_back, scale=DEFAULT_SCALE, l2_eps=1e-6, rms_eps=1e-6,
                            *, out_dtype=torch.bfloat16, o=None, stream=None):
    """The layer core for a few tokens per request from pooled states (verify:
    write_back=False; replay: write_back=True).  Returns o_gated [T, H, 128]."""
    T, H, _ = qp.shape
    B = slot.shape[0]
    P = S_pool.shape[0]
    if o is None:
        o = _empty((T, H, HEAD_DIM), out_dtype, qp.device, stream)
    rc = _lib.kda_decode_layer_tokens(B, H, P, T, _p(cu_tokens), _p(slot), _p(qp), _p(kp), _p(vp),
                                      _p(conv_w), _p(z), _p(A), _p(b), _p(beta_logit), _p(g),
                                      _p(S_pool), _p(conv_pool), int(bool(write_back)),
                                      float(scale), float(l2_eps), float(rms_eps),
                                      _dtype_code(o.dtype), _p(o), _stream(stream))
    _check("kda_decode_layer_tokens", rc)
    return o


def rope_table(num_positions: int, rotary_dim: int = HEAD_DIM, base: float = 10000.0, *,
               inv_freq=None, magnitude: float = 1.0, device="cuda") -> torch.Tensor:
    """(cos, sin) of every position and rotated pair, [num_positions, rotary_dim/2, 2] fp32, kept
    by the caller like a weight.  inv_freq [rotary_dim/2] (default base^(-2i/rotary_dim)) and
    magnitude carry a long-context scaling; the angles are formed in 64 bits."""
    if inv_freq is None:
        inv_freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device=device)
    angle = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] * inv_freq
    return torch.stack([angle.cos(), angle.sin()], -1).mul_(magnitude).float().contiguous()


# Marshalling of the calls below: plain integers for pointers, the raw current stream, and few
# Python calls (a decode step's kernels take less time than objects for each argument would).
_F32, _I32 = torch.float32, torch.int32
_ELEM = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}


def _refuse(t: torch.Tensor, dtype, dev: int):
    """Says why a tensor cannot be handed to a call on GPU dev."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    raise ValueError("tensors must be contiguous")


def _ptr(t: torch.Tensor, dev: int):
    if not t.is_contiguous() or t.get_device() != dev:
        _refuse(t, None, dev)
    return t.data_ptr()


def _ptrs(dev: int, dtype: torch.dtype, *tensors):
    """Pointers of dense tensors of one type on GPU dev (None for None)."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
            _refuse(t, dtype, dev)
        out.append(t.data_ptr())
    return out


def _launch(stream, dev: int):
    """The raw stream of a call on tensors of GPU dev.  It must be the current one: the library launches
    there, and its kernels would take a host or another GPU's address for one of that GPU's."""
    if dev < 0:
        raise ValueError("tensors must be on a GPU")
    if dev != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current GPU")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _elem(dtype: torch.dtype) -> int:
    code = _ELEM.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _count(n: int) -> int:
    """n as the int32 that means the same, where more than 2^31 - 1 means no more than that and any negative
    number is refused (ctypes would keep the low 32 bits)."""
    return -1 if n < 0 else n if n <= 0x7fffffff else 0x7fffffff


def _heads(t: torch.Tensor, dev: int):
    """(tokens, heads, elements from token to token) of [T, heads, 128] whose heads lie side by side."""
    T, H, d = t.shape
    s0, s1, s2 = t.stride()
    if d != HEAD_DIM or s2 != 1 or (s1 != HEAD_DIM and H > 1):
        raise ValueError("the heads of a token must lie side by side, 128 channels each")
    if t.get_device() != dev:
        _refuse(t, None, dev)
    return T, H, s0 if T > 1 else H * HEAD_DIM


def _pool_shape(kv_pool):
    """(pages, kv heads, page_size) of a cache pool [P, 2, Hkv, page_size, 128]."""
    shape = kv_pool.shape
    if len(shape) != 5 or shape[1] != 2 or shape[4] != HEAD_DIM:
        raise ValueError("kv_pool must be [pages, 2, kv heads, page_size, 128]")
    return shape[0], shape[2], shape[3]


def _rope_args(rope, positions, T, dev):
    if rope is None:
        return None, 0, 0, None
    if positions.numel() != T:
        raise ValueError("positions must have one entry per token")
    shape = rope.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError("the rotation table must be [positions, rotary_dim / 2, 2]")
    if rope.dtype is not _F32 or positions.dtype is not _I32:
        raise TypeError("the rotation table must be float32, positions int32")
    return _ptr(rope, dev), shape[0], 2 * shape[1], _ptr(positions, dev)


def _weights(dev, *weights):
    for w in weights:
        if w is not None and w.numel() != HEAD_DIM:
            raise ValueError("a weight must be [128]")
    return _ptrs(dev, _F32, *weights)


def _cache_args(dev, page_table, slot, cu_tokens, kv_len):
    """(requests, rows, width, pointers of the table, slots, offsets and lengths)."""
    R, M = page_table.shape
    B = slot.numel()
    if cu_tokens.numel() != B + 1 or kv_len.numel() != R:
        raise ValueError("cu_tokens must have one entry more than slot, kv_len one per table row")
    return B, R, M, _ptrs(dev, _I32, page_table, slot, cu_tokens, kv_len)


def kda_qk_norm_rope(q, k, rope, positions, q_weight=None, k_weight=None, eps=1e-6, *, norm=True,
                     interleaved=False, out_dtype=None, q_out=None, k_out=None, stream=None):
    """q [T, Hq, 128] and k [T, Hkv, 128] (heads dense, any token stride) normed per head and
    rotated by rope_table(...) at positions [T] int32 (rope None: no rotation).
    Returns (q_out, k_out)."""
    dtype, dev = q.dtype, q.get_device()
    out_dtype = q_out.dtype if q_out is not None else out_dtype or dtype
    if q_out is None:
        q_out = _empty(q.shape, out_dtype, q.device, stream)
    if k_out is None:
        k_out = _empty(k.shape, out_dtype, k.device, stream)
    if k.shape[0] != q.shape[0] or q_out.shape != q.shape or k_out.shape != k.shape or k_out.dtype is not out_dtype \
            or k.dtype is not dtype:
        raise ValueError("q, k and their outputs must agree in tokens, heads and type")
    (T, Hq, qs), (_, Hkv, ks) = _heads(q, dev), _heads(k, dev)
    table, P, R, pos = _rope_args(rope, positions, T, dev)
    wq, wk = _weights(dev, q_weight, k_weight)
    rc = _lib.kda_qk_norm_rope(_elem(dtype), _elem(out_dtype), T, Hq, Hkv, q.data_ptr(), qs, k.data_ptr(), ks,
                               wq, wk, eps, norm, table, P, R, interleaved, pos, _ptr(q_out, dev),
                               _ptr(k_out, dev), _launch(stream, dev))
    _check("kda_qk_norm_rope", rc)
    return q_out, k_out


def kda_qk_norm_rope_append(q, k, v, rope, positions, kv_pool, page_table, slot, cu_tokens, kv_len,
                            q_weight=None, k_weight=None, eps=1e-6, *, norm=True, interleaved=False,
                            q_out=None, stream=None):
    """kda_qk_norm_rope with k (normed and rotated) and v written to the cache pages of the tokens:
    kv_pool [P, 2, Hkv, page_size, 128], page_table [R, M], kv_len [R] (these tokens counted),
    slot [B], cu_tokens [B+1].  Outputs have the pool's type.  Returns q_out."""
    dtype, out_dtype, dev = q.dtype, kv_pool.dtype, q.get_device()
    P, pool_heads, page = _pool_shape(kv_pool)
    if q_out is None:
        q_out = _empty(q.shape, out_dtype, q.device, stream)
    (T, Hq, qs), (Tk, Hkv, ks), (Tv, Hv, vs) = _heads(q, dev), _heads(k, dev), _heads(v, dev)
    if Tk != T or Tv != T or Hkv != pool_heads or Hv != Hkv or q_out.shape != q.shape \
            or q_out.dtype is not out_dtype or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k, v, q_out and kv_pool must agree in tokens, heads and type")
    table, npos, R, pos = _rope_args(rope, positions, T, dev)
    B, rows, width, (pt, sl, cu, kl) = _cache_args(dev, page_table, slot, cu_tokens, kv_len)
    wq, wk = _weights(dev, q_weight, k_weight)
    rc = _lib.kda_qk_norm_rope_append(
        _elem(dtype), _elem(out_dtype), B, T, Hq, Hkv, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
        wq, wk, eps, norm, table, npos, R, interleaved, pos, P, page, rows, width, pt, sl, cu, kl,
        _ptr(kv_pool, dev), _ptr(q_out, dev), _launch(stream, dev))
    _check("kda_qk_norm_rope_append", rc)
    return q_out


def kda_window_attention(q, kv_pool, page_table, slot, cu_tokens, kv_len, window, sinks=0,
                         scale=DEFAULT_SCALE, *, max_tokens=None, o=None, stream=None):
    """Attention of q [T, Hq, 128] over the requests' rows of the cache, with a sliding window and
    the first `sinks` tokens always visible (window None: plain causal).  max_tokens: no request
    brings more (default: T); small values let the call split long rows.  Returns o."""
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    T, Hq, d = shape
    P, Hkv, page = _pool_shape(kv_pool)
    if kv_pool.dtype is not dtype:
        raise TypeError("q and kv_pool must have one type")
    if o is None:
        o = _empty(shape, dtype, q.device, stream)
    elif o.shape != shape or o.dtype is not dtype:
        raise ValueError("o must have q's shape and type")
    if d != HEAD_DIM:
        raise ValueError("q must be [tokens, heads, 128]")
    B, rows, width, (pt, sl, cu, kl) = _cache_args(dev, page_table, slot, cu_tokens, kv_len)
    rc = _lib.kda_window_attention(
        _elem(dtype), B, T, max(T, 1) if max_tokens is None else _count(max_tokens), Hq, Hkv, P, page, rows, width,
        0x7fffffff if window is None else _count(window), _count(sinks), _ptr(q, dev), _ptr(kv_pool, dev), pt, sl, cu, kl, scale,
        _ptr(o, dev), _launch(stream, dev))
    _check("kda_window_attention", rc)
    return o


def _layers(pool):
    """(layers, pages, bytes of a page) of [layers, pages, ...]."""
    shape = pool.shape
    if len(shape) < 3:
        raise ValueError("pool must be [layers, pages, ...]")
    L, P = shape[0], shape[1]
    if L > 0x7fffffff or P > 0x7fffffff:
        raise ValueError("a pool has at most 2^31 - 1 layers and pages")
    return L, P, pool.numel() // max(1, L * P) * pool.element_size()


def kda_pages_copy(pool, src, dst, *, stream=None):
    """Pages dst[i] := pages src[i] in every layer of pool [layers, pages, ...] (rows of a
    recurrent-state pool as well); src, dst int32 on the device."""
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have one length")
    L, P, nbytes = _layers(pool)
    dev = pool.get_device()
    s, d = _ptrs(dev, _I32, src, dst)
    _check("kda_pages_copy", _lib.kda_pages_copy(L, P, nbytes, n, s, d, _ptr(pool, dev), _launch(stream, dev)))


def kda_pages_workspace_size(num_pages: int, table_rows: int) -> int:
    return int(_lib.kda_pages_workspace_size(num_pages, table_rows))


def _pages_workspace(workspace, P, rows, device, stream):
    if workspace is None:
        n = kda_pages_workspace_size(P, rows)
        workspace = _empty(n, torch.uint8, device, stream)
        return workspace, n
    return workspace, workspace.numel() * workspace.element_size()


def kda_pages_fork(pool, page_table, kv_len, parent, child, page_size, *, workspace=None, stream=None):
    """Rows child[i] become branches of rows parent[i], in place in page_table and kv_len: whole
    pages shared, a part-filled last page copied to a fresh one in every layer of pool, no entry
    past the parent's tokens."""
    F = parent.numel()
    R, M = page_table.shape
    if child.numel() != F or kv_len.numel() != R:
        raise ValueError("parent and child must have one length, kv_len one entry per table row")
    L, P, nbytes = _layers(pool)
    workspace, wbytes = _pages_workspace(workspace, P, R, pool.device, stream)
    dev = pool.get_device()
    pa, ch, pt, kl = _ptrs(dev, _I32, parent, child, page_table, kv_len)
    _check("kda_pages_fork", _lib.kda_pages_fork(L, P, nbytes, _count(page_size), R, M, F, pa, ch, pt, kl, _ptr(pool, dev),
                                                 _ptr(workspace, dev), wbytes, _launch(stream, dev)))


def kda_pages_release(page_table, kv_len, rows, page_size, window=0, sinks=0, *, stream=None):
    """Empties the rows (window 0), or drops only the pages that no coming token sees with this
    window and these sinks; in place in page_table (and kv_len)."""
    R, M = page_table.shape
    if kv_len.numel() != R:
        raise ValueError("kv_len must have one entry per table row")
    dev = page_table.get_device()
    r, pt, kl = _ptrs(dev, _I32, rows, page_table, kv_len)
    _check("kda_pages_release", _lib.kda_pages_release(R, M, _count(page_size), rows.numel(), r, _count(window),
                                                       _count(sinks), pt, kl,
                                                       _launch(stream, dev)))


def kda_pages_compact(pool, page_table, *, table_out=None, num_live=None, workspace=None, stream=None):
    """Brings the pages that rows name together at the front of pool [layers, pages, ...].  Returns
    (table_out, num_live): the table with the new names (default: in place) and how many pages are
    live, [1] int32 on the device."""
    L, P, nbytes = _layers(pool)
    R, M = page_table.shape
    table_out = page_table if table_out is None else table_out
    if table_out.shape != page_table.shape:
        raise ValueError("table_out must have page_table's shape")
    if num_live is None:
        num_live = _empty(1, _I32, pool.device, stream)
    workspace, wbytes = _pages_workspace(workspace, P, R, pool.device, stream)
    dev = pool.get_device()
    tin, tout, live = _ptrs(dev, _I32, page_table, table_out, num_live)
    _check("kda_pages_compact", _lib.kda_pages_compact(L, P, nbytes, R, M, tin, tout, live, _ptr(pool, dev),
                                                       _ptr(workspace, dev), wbytes, _launch(stream, dev)))
    return table_out, num_live


def kda_check_prefill_inputs(cu_seqlens, log_alpha=None, total_tokens=None, num_heads=1,
                             stream=None):
    """Queue the contents checks of prefill inputs (offsets, decay range); read the result
    with kda_get_device_status.  log_alpha [T, H, 128] or [T, H] (per-head decay), or None
    to check the offsets alone against total_tokens."""
    N = cu_seqlens.shape[0] - 1
    if log_alpha is None:
        T, H, head = int(total_tokens), int(num_heads), 0
    else:
        T, H = log_alpha.shape[:2]
        head = 1 if log_alpha.dim() == 2 else 0
    rc = _lib.kda_check_prefill_inputs(N, T, H, _p(log_alpha), head, _p(cu_seqlens),
                                       _stream(stream))
    _check("kda_check_prefill_inputs", rc)


def kda_get_device_status(stream=None):
    """Synchronises the stream; returns (status_code, detail) and clears the word."""
    detail = ctypes.c_uint32(0)
    rc = _lib.kda_get_device_status(_stream(stream), ctypes.byref(detail))
    return int(rc), int(detail.value)
