"""Python binding of the B200 KDA recurrence library (ctypes over the C ABI in include/kda.h).

Argument marshalling only: every step of the computation runs in the CUDA kernels of
libkda_b200.so.  There is no CPU fallback; if the library is missing or a call fails,
these functions raise.

    from linear_attention_recurrence_forward_b200 import kda_forward_chunked, kda_decode_step
    o, S_T = kda_forward_chunked(q, k, v, g, beta, S0)        # prefill, torch CUDA tensors
    o, S_T, S_mid = kda_forward_chunked_states(q, k, v, g, beta, S0, interval=512)
    o, S_T = kda_forward_chunked_host(q_cpu, k_cpu, v_cpu, g_cpu, beta_cpu, S0_cpu)  # host tensors in and out
    o = kda_decode_step(q, k, v, g, beta, S)                   # one token, S updated in place

    y, conv_state = kda_short_conv(x, weight, bias, conv_state)   # the short causal convolution before it
    y, S_T = kda_ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0)    # the selective scan, its scalar-decay sibling
    kda_pool_copy(pools, src, dst)                                # slots of the layers' state pools

Layouts (contiguous): q, k, g [B, T, H, dk]; v, o [B, T, H, dv]; beta [B, T, H];
states [B, H, dk, dv] fp32.  Decode drops the T axis.  dtype: bf16 or fp32 (all of q, k,
v, g, beta share it; o gets it too).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
from typing import Optional

import torch

__all__ = [
    "kda_forward_chunked",
    "kda_forward_chunked_states",
    "kda_forward_chunked_host",
    "kda_forward_chunked_host_noalloc",
    "host_workspace_bytes",
    "kda_decode_step",
    "kda_forward_varlen",
    "kda_forward_chunked_fused",
    "kda_decode_step_paged",
    "kda_state_compose",
    "kda_output_correct",
    "kda_short_conv",
    "kda_short_conv_varlen",
    "kda_short_conv_step",
    "kda_short_conv_step_paged",
    "kda_ssm_forward",
    "kda_ssm_forward_varlen",
    "kda_ssm_decode_step",
    "kda_ssm_decode_step_paged",
    "ssm_workspace_bytes",
    "kda_pool_copy",
    "kda_pool_clear",
    "kda_pool_compact",
    "kda_get_device_status",
    "kda_status_string",
    "kda_debug_set_wait_fault",
    "KdaError",
    "lib",
    "LIB_PATH",
    "STATUS",
    "IMPL",
    "ACTIVATION",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda_b200.so")

STATUS = {
    "KDA_OK": 0,
    "KDA_ERR_INVALID_ARG": -1,
    "KDA_ERR_UNSUPPORTED": -2,
    "KDA_ERR_MISALIGNED": -3,
    "KDA_ERR_CUDA": -4,
    "KDA_ERR_TIMEOUT": -5,
}
DTYPE = {torch.bfloat16: 0, torch.float32: 1}
IMPL = {"auto": 0, "tcgen05": 1, "simt": 2}
ACTIVATION = {None: 0, "silu": 1}

_lib: Optional[ctypes.CDLL] = None


class KdaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {kda_status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first (python -m linear_attention_recurrence_forward_b200.build "
                "or __graft_entry__.build()); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        L.kda_forward_chunked.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.kda_forward_chunked.restype = I
        L.kda_forward_chunked_impl.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
        L.kda_forward_chunked_impl.restype = I
        L.kda_forward_chunked_states.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P]
        L.kda_forward_chunked_states.restype = I
        L.kda_forward_chunked_host.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, ctypes.c_size_t, I, P]
        L.kda_forward_chunked_host.restype = I
        L.kda_forward_chunked_host_noalloc.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
        L.kda_forward_chunked_host_noalloc.restype = I
        L.kda_forward_chunked_host_workspace.argtypes = [I, I, I, I, I]
        L.kda_forward_chunked_host_workspace.restype = ctypes.c_size_t
        L.kda_state_compose.argtypes = [P, P, P, P, I, I, I, P]
        L.kda_state_compose.restype = I
        L.kda_output_correct.argtypes = [P, P, P, P, I, I, I, I, I, I, P]
        L.kda_output_correct.restype = I
        L.kda_forward_chunked_fused.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
        L.kda_forward_chunked_fused.restype = I
        L.kda_forward_varlen.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
        L.kda_forward_varlen.restype = I
        L.kda_decode_step_paged.argtypes = [P, P, P, P, P, P, I, P, P, I, I, I, I, I, P]
        L.kda_decode_step_paged.restype = I
        L.kda_decode_step.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P]
        L.kda_decode_step.restype = I
        J = ctypes.c_longlong
        L.kda_short_conv.argtypes = [P, P, P, P, P, P, I, I, I, I, J, J, I, I, P]
        L.kda_short_conv.restype = I
        L.kda_short_conv_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, J, J, I, I, P]
        L.kda_short_conv_varlen.restype = I
        L.kda_short_conv_step.argtypes = [P, P, P, P, P, I, I, I, J, J, I, I, P]
        L.kda_short_conv_step.restype = I
        L.kda_short_conv_step_paged.argtypes = [P, P, P, P, I, P, P, I, I, I, J, J, I, I, P]
        L.kda_short_conv_step_paged.restype = I
        L.kda_ssm_forward.argtypes = [P] * 10 + [I] * 6 + [J] * 4 + [I, I, P, ctypes.c_size_t, P]
        L.kda_ssm_forward.restype = I
        L.kda_ssm_forward_varlen.argtypes = [P] * 11 + [I] * 6 + [J] * 4 + [I, I, P, ctypes.c_size_t, P]
        L.kda_ssm_forward_varlen.restype = I
        L.kda_ssm_workspace.argtypes = [I] * 7
        L.kda_ssm_workspace.restype = ctypes.c_size_t
        L.kda_ssm_decode_step.argtypes = [P] * 9 + [I] * 5 + [J] * 4 + [I, P]
        L.kda_ssm_decode_step.restype = I
        L.kda_ssm_decode_step_paged.argtypes = [P] * 8 + [I, P, P] + [I] * 5 + [J] * 4 + [I, P]
        L.kda_ssm_decode_step_paged.restype = I
        L.kda_pool_copy.argtypes = [P, P, I, I, I, P, P, I, P]
        L.kda_pool_copy.restype = I
        L.kda_pool_clear.argtypes = [P, I, I, P, I, P]
        L.kda_pool_clear.restype = I
        L.kda_pool_compact.argtypes = [P, I, I, P, P, P, I, P, P]
        L.kda_pool_compact.restype = I
        L.kda_get_device_status.argtypes = [P]
        L.kda_get_device_status.restype = I
        L.kda_status_string.argtypes = [I]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_version.argtypes = []
        L.kda_version.restype = I
        L.kda_debug_set_wait_fault.argtypes = [I, ctypes.c_ulonglong]
        L.kda_debug_set_wait_fault.restype = I
        _lib = L
    return _lib


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kda_forward_chunked(q, k, v, g, beta, S0=None, *, o=None, S_T=None, return_state: bool = True,
                        impl: str = "auto", stream=None):
    """Prefill over [B, T, H, *] CUDA tensors.  Returns (o, S_T) (S_T None if not requested).

    S_T may be passed in (and may be S0 itself for an in-place state carry).
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                           ("g", g, (B, T, H, dk)), ("beta", beta, (B, T, H))):
        _check(t, name, shape, dt, dev)
    if S0 is not None:
        _check(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (B, T, H, dv), dt, dev)
    if S_T is None and return_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    elif S_T is not None:
        _check(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_forward_chunked_impl(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
                                            _ptr(o), _ptr(S_T), B, T, H, dk, dv, DTYPE[dt], IMPL[impl],
                                            _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_forward_chunked", rc)
    return o, S_T


def host_workspace_bytes(T: int, H: int, dk: int = 128, dv: int = 128, dtype=torch.bfloat16) -> int:
    """Bytes of device workspace kda_forward_chunked_host needs for T tokens and H heads."""
    if dtype not in DTYPE:
        raise ValueError(f"unsupported dtype {dtype}")
    n = lib().kda_forward_chunked_host_workspace(int(T), int(H), int(dk), int(dv), DTYPE[dtype])
    if n == 0:
        raise ValueError(f"unsupported sizes T={T} H={H} dk={dk} dv={dv}")
    return int(n)


def kda_forward_chunked_host(q, k, v, g, beta, S0=None, *, o=None, S_T=None, return_state: bool = True,
                             workspace=None, impl: str = "auto", stream=None, device=None):
    """Prefill over [B, T, H, *] HOST (CPU) tensors, outputs in host memory.

    The library copies the inputs to the GPU segment by segment, runs the prefill and copies o
    and S_T back, overlapping the copies with the kernels; o and S_T equal kda_forward_chunked's
    bitwise.  Pinned inputs make the copies asynchronous; outputs allocated here are pinned.
    The call is asynchronous on `stream`: read o and S_T after synchronizing it.  `workspace` is
    a CUDA uint8 tensor of at least host_workspace_bytes(T, H, dk, dv, dtype) bytes (allocated on
    `device` if not given).
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    cpu = torch.device("cpu")
    for name, t, shape in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                           ("g", g, (B, T, H, dk)), ("beta", beta, (B, T, H))):
        _check(t, name, shape, dt, cpu)
    if S0 is not None:
        _check(S0, "S0", (B, H, dk, dv), torch.float32, cpu)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, pin_memory=True)
    else:
        _check(o, "o", (B, T, H, dv), dt, cpu)
    if S_T is None and return_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=True)
    elif S_T is not None:
        _check(S_T, "S_T", (B, H, dk, dv), torch.float32, cpu)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    nbytes = host_workspace_bytes(T, H, dk, dv, dt)
    own_workspace = workspace is None
    if own_workspace:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    with torch.cuda.device(workspace.device):
        rc = lib().kda_forward_chunked_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(o),
                                            _ptr(S_T), B, T, H, dk, dv, DTYPE[dt], _ptr(workspace),
                                            workspace.numel() * workspace.element_size(), IMPL[impl],
                                            _stream_handle(stream))
        if rc != 0:
            raise KdaError("kda_forward_chunked_host", rc)
        if own_workspace and stream is not None:
            workspace.record_stream(stream)   # not reused before the call's work on `stream` is done
    return o, S_T


def kda_forward_chunked_host_noalloc(q, k, v, g, beta, S0=None, *, o=None, S_T=None, return_state: bool = True,
                                     impl: str = "auto", stream=None, device=None):
    """kda_forward_chunked_host without a workspace: the library stages the work through its own fixed
    device scratch (KDA_NOALLOC_SCRATCH_BYTES per device), so nothing is allocated on the device.
    Host tensors in, host tensors out (outputs allocated here are pinned); o and S_T equal
    kda_forward_chunked_host's bitwise.  Calls whose work overlaps on the GPU share the scratch and
    race: keep them in order on one stream.  Read o and S_T after synchronizing `stream`.
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    cpu = torch.device("cpu")
    for name, t, shape in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                           ("g", g, (B, T, H, dk)), ("beta", beta, (B, T, H))):
        _check(t, name, shape, dt, cpu)
    if S0 is not None:
        _check(S0, "S0", (B, H, dk, dv), torch.float32, cpu)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, pin_memory=True)
    else:
        _check(o, "o", (B, T, H, dv), dt, cpu)
    if S_T is None and return_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=True)
    elif S_T is not None:
        _check(S_T, "S_T", (B, H, dk, dv), torch.float32, cpu)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        rc = lib().kda_forward_chunked_host_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
                                                    _ptr(o), _ptr(S_T), B, T, H, dk, dv, DTYPE[dt], IMPL[impl],
                                                    _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_forward_chunked_host_noalloc", rc)
    return o, S_T


def kda_forward_chunked_states(q, k, v, g, beta, S0=None, *, interval: int = 512, o=None, S_T=None,
                               S_mid=None, impl: str = "auto", stream=None):
    """Prefill that also returns the state after every `interval` tokens (a multiple of 64).

    Returns (o, S_T, S_mid) with S_mid [B, H, T // interval, dk, dv] fp32: S_mid[:, :, n] is the
    state after the first (n + 1) * interval tokens.
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                           ("g", g, (B, T, H, dk)), ("beta", beta, (B, T, H))):
        _check(t, name, shape, dt, dev)
    if S0 is not None:
        _check(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    n_mid = T // interval if interval > 0 else 0
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (B, T, H, dv), dt, dev)
    if S_T is None:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    else:
        _check(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    if S_mid is None:
        S_mid = torch.empty((B, H, n_mid, dk, dv), dtype=torch.float32, device=dev)
    else:
        _check(S_mid, "S_mid", (B, H, n_mid, dk, dv), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_forward_chunked_states(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
                                              _ptr(o), _ptr(S_T), _ptr(S_mid) if n_mid > 0 else None,
                                              int(interval), B, T, H, dk, dv, DTYPE[dt], IMPL[impl],
                                              _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_forward_chunked_states", rc)
    return o, S_T, S_mid


def kda_decode_step(q, k, v, g, beta, S, *, o=None, stream=None):
    """One token for every (b, h).  q, k, g [B, H, dk]; v [B, H, dv]; beta [B, H]; S updated in place."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q", q, (B, H, dk)), ("k", k, (B, H, dk)), ("v", v, (B, H, dv)),
                           ("g", g, (B, H, dk)), ("beta", beta, (B, H))):
        _check(t, name, shape, dt, dev)
    _check(S, "S", (B, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (B, H, dv), dt, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o),
                                   B, H, dk, dv, DTYPE[dt], _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_decode_step", rc)
    return o


def kda_forward_chunked_fused(q_raw, k_raw, v, z_g, z_beta, S0=None, *, o=None, S_T=None,
                              return_state: bool = True, impl: str = "auto", stream=None):
    """Prefill with the prologue in the kernels: g = -5 sigmoid(z_g), beta = sigmoid(z_beta), q and k
    L2-normalised over the head dimension.  Same layouts as kda_forward_chunked."""
    B, T, H, dk = q_raw.shape
    dv = v.shape[-1]
    dev, dt = q_raw.device, q_raw.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q_raw", q_raw, (B, T, H, dk)), ("k_raw", k_raw, (B, T, H, dk)),
                           ("v", v, (B, T, H, dv)), ("z_g", z_g, (B, T, H, dk)), ("z_beta", z_beta, (B, T, H))):
        _check(t, name, shape, dt, dev)
    if S0 is not None:
        _check(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (B, T, H, dv), dt, dev)
    if S_T is None and return_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    elif S_T is not None:
        _check(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_forward_chunked_fused(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(z_g), _ptr(z_beta), _ptr(S0),
                                             _ptr(o), _ptr(S_T), B, T, H, dk, dv, DTYPE[dt], IMPL[impl],
                                             _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_forward_chunked_fused", rc)
    return o, S_T


def kda_forward_varlen(q, k, v, g, beta, cu_seqlens, S0=None, *, o=None, S_T=None, return_state: bool = True,
                       impl: str = "auto", stream=None):
    """Prefill over packed sequences: q, k, g [T_total, H, dk]; v [T_total, H, dv]; beta [T_total, H];
    cu_seqlens int32 [N + 1] on the device (sequence n = tokens cu_seqlens[n] .. cu_seqlens[n+1]-1).
    States [N, H, dk, dv] fp32.  Returns (o [T_total, H, dv], S_T or None).
    """
    T_total, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    dev, dt = q.device, q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q", q, (T_total, H, dk)), ("k", k, (T_total, H, dk)), ("v", v, (T_total, H, dv)),
                           ("g", g, (T_total, H, dk)), ("beta", beta, (T_total, H))):
        _check(t, name, shape, dt, dev)
    _check(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    if S0 is not None:
        _check(S0, "S0", (N, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty((T_total, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (T_total, H, dv), dt, dev)
    if S_T is None and return_state:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    elif S_T is not None:
        _check(S_T, "S_T", (N, H, dk, dv), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_forward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(S0),
                                      _ptr(o), _ptr(S_T), N, T_total, H, dk, dv, DTYPE[dt], IMPL[impl],
                                      _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_forward_varlen", rc)
    return o, S_T


def kda_decode_step_paged(q, k, v, g, beta, S_pool, slots, *, o=None, stream=None):
    """One token per sequence with the states in a pool: S_pool [n_slots, H, dk, dv] fp32 (updated in
    place), slots int32 [B] on the device (sequence b uses S_pool[slots[b]]; negative = skip)."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    for name, t, shape in (("q", q, (B, H, dk)), ("k", k, (B, H, dk)), ("v", v, (B, H, dv)),
                           ("g", g, (B, H, dk)), ("beta", beta, (B, H))):
        _check(t, name, shape, dt, dev)
    n_slots = S_pool.shape[0]
    _check(S_pool, "S_pool", (n_slots, H, dk, dv), torch.float32, dev)
    _check(slots, "slots", (B,), torch.int32, dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=dev)
    else:
        _check(o, "o", (B, H, dv), dt, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_decode_step_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_pool), n_slots,
                                         _ptr(slots), _ptr(o), B, H, dk, dv, DTYPE[dt], _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_decode_step_paged", rc)
    return o


def kda_state_compose(M, S, N=None, *, out=None, stream=None):
    """out = M @ S + N per head: M [..., dk, dk], S and N [..., dk, dv] fp32 CUDA tensors (N may be None).

    out may be S or N itself.  The leading dimensions are flattened into heads.
    """
    dk, dv = S.shape[-2], S.shape[-1]
    lead = tuple(S.shape[:-2])
    dev = S.device
    _check(M, "M", lead + (dk, dk), torch.float32, dev)
    if N is not None:
        _check(N, "N", lead + (dk, dv), torch.float32, dev)
    _check(S, "S", lead + (dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty_like(S)
    else:
        _check(out, "out", lead + (dk, dv), torch.float32, dev)
    count = 1
    for x in lead:
        count *= x
    with torch.cuda.device(dev):
        rc = lib().kda_state_compose(_ptr(M), _ptr(S), _ptr(N), _ptr(out), count, dk, dv, _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_state_compose", rc)
    return out


def kda_output_correct(C, S_in, o_in, *, out=None, stream=None):
    """out = o_in + per token S_in^T C: C [B, T, H, dk], o_in [B, T, H, dv] (same dtype) and S_in
    [B, H, dk, dv] fp32 CUDA tensors.  out may be o_in itself.  The output correction of a segment
    run from a zero state (context parallelism): C is the output of the same segment with v = 0 and
    S0 = I."""
    B, T, H, dk = C.shape
    dv = o_in.shape[-1]
    dev, dt = C.device, C.dtype
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    _check(C, "C", (B, T, H, dk), dt, dev)
    _check(o_in, "o_in", (B, T, H, dv), dt, dev)
    _check(S_in, "S_in", (B, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty_like(o_in)
    else:
        _check(out, "out", (B, T, H, dv), dt, dev)
    with torch.cuda.device(dev):
        rc = lib().kda_output_correct(_ptr(C), _ptr(S_in), _ptr(o_in), _ptr(out), B, T, H, dk, dv, DTYPE[dt],
                                      _stream_handle(stream))
    if rc != 0:
        raise KdaError("kda_output_correct", rc)
    return out


# ------------------------------------------------------------------ short convolution, scan, pools


_SAME_DEVICE = contextlib.nullcontext()


def _on_device(dev: torch.device):
    """The device of the tensors made current for a call (nothing to do when it is already)."""
    if dev.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got {dev}")
    if dev.index == torch._C._cuda_getDevice():
        return _SAME_DEVICE
    return torch.cuda.device(dev)


def _stream_on(dev: torch.device, stream) -> Optional[int]:
    """The handle of `stream`, or of the device's current stream (read without making a Stream object, which
    would cost as much as the launch)."""
    return (torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream) or None


def _empty(shape, dtype, dev, stream, like=None) -> torch.Tensor:
    """An output or workspace in memory of the stream the call runs on; `like`: a tensor that may have its shape,
    dtype and a dense layout (the shortest way to it)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=dev)
    if like is not None and like.dtype == dtype and like.shape == shape and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=dev)


def _dense(t, name: str, shape: tuple, dtype, device) -> None:
    """_check, in one expression when all is well (these checks are a good part of a small call's host time)."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device
            and t.is_contiguous()):
        _check(t, name, shape, dtype, device)


def _rows(t, name: str, lead, row, dtype, device) -> int:
    """Check a tensor of shape lead + row whose rows are contiguous and evenly spaced (a slice of wider rows
    is fine); returns the spacing in elements."""
    if isinstance(t, torch.Tensor) and t.is_contiguous() and t.shape == lead + row and t.dtype == dtype \
            and t.device == device:
        return math.prod(row)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != lead + row:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + row}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    stride = t.stride()
    width = 1
    for n, st in zip(reversed(row), reversed(stride)):
        if n > 1 and st != width:
            raise ValueError(f"{name} must have contiguous rows of {row}")
        width *= n
    if 0 in lead:
        return width
    ld, rows = None, 1                   # spacing found so far, and the rows it has spanned
    for n, st in zip(reversed(lead), reversed(stride[:len(lead)])):
        if n > 1:
            if ld is None:
                ld, rows = st, n
            elif st != ld * rows:
                raise ValueError(f"{name} must have evenly spaced rows")
            else:
                rows *= n
    return width if ld is None else ld


def _vector(t, name: str, n: int, dtype, device):
    if t is not None:
        _dense(t, name, (n,), dtype, device)
    return _ptr(t)


def _dtype_code(dt) -> int:
    if dt not in DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    return DTYPE[dt]


def _conv_common(x, lead, weight, bias, y, activation, stream):
    """The checks the convolution's forms share: (C, W, y, ldx, ldy, weight, bias pointers, activation code)."""
    C, W = weight.shape
    dev, dt = x.device, x.dtype
    _dtype_code(dt)
    if activation not in ACTIVATION:
        raise ValueError(f"unknown activation {activation!r}")
    _dense(weight, "weight", (C, W), dt, dev)
    b = _vector(bias, "bias", C, dt, dev)
    ldx = _rows(x, "x", lead, (C,), dt, dev)
    if y is None:
        y, ldy = _empty(lead + (C,), dt, dev, stream, x), C
    else:
        ldy = _rows(y, "y", lead, (C,), dt, dev)
    return C, W, y, ldx, ldy, weight.data_ptr(), b, ACTIVATION[activation]


def kda_short_conv(x, weight, bias=None, state=None, *, activation="silu", y=None, state_out=None,
                   return_state: bool = True, stream=None):
    """The short causal convolution over x [B, T, C] (rows may be slices of wider ones): weight [C, W],
    bias [C] or None, state [B, W-1, C] (the inputs before token 0; None for zeros).  Returns (y [B, T, C],
    state_out [B, W-1, C] or None).  state_out may be state itself.  activation: "silu" or None.

    For the KDA prefill, whose q, k and v are contiguous, convolve each slice of the projection in a call of its
    own: y comes out contiguous."""
    B, T = x.shape[:2]
    C, W, y, ldx, ldy, w, b, act = _conv_common(x, (B, T), weight, bias, y, activation, stream)
    dev, dt = x.device, x.dtype
    if state is not None:
        _dense(state, "state", (B, W - 1, C), dt, dev)
    if state_out is not None:
        _dense(state_out, "state_out", (B, W - 1, C), dt, dev)
    elif return_state:
        state_out = _empty((B, W - 1, C), dt, dev, stream, state)
    with _on_device(dev):
        rc = lib().kda_short_conv(x.data_ptr(), w, b, _ptr(state), y.data_ptr(), _ptr(state_out), B, T, C, W, ldx,
                                  ldy, act, DTYPE[dt], _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_short_conv", rc)
    return y, state_out


def kda_short_conv_varlen(x, weight, cu_seqlens, bias=None, state=None, *, activation="silu", y=None,
                          state_out=None, return_state: bool = True, stream=None):
    """kda_short_conv over packed sequences: x [T_total, C], cu_seqlens int32 [N + 1] on the device (as
    kda_forward_varlen), states [N, W-1, C].  Returns (y [T_total, C], state_out or None)."""
    T_total = x.shape[0]
    N = cu_seqlens.shape[0] - 1
    C, W, y, ldx, ldy, w, b, act = _conv_common(x, (T_total,), weight, bias, y, activation, stream)
    dev, dt = x.device, x.dtype
    _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    if state is not None:
        _dense(state, "state", (N, W - 1, C), dt, dev)
    if state_out is not None:
        _dense(state_out, "state_out", (N, W - 1, C), dt, dev)
    elif return_state:
        state_out = _empty((N, W - 1, C), dt, dev, stream, state)
    with _on_device(dev):
        rc = lib().kda_short_conv_varlen(x.data_ptr(), w, b, cu_seqlens.data_ptr(), _ptr(state), y.data_ptr(),
                                         _ptr(state_out), N, T_total, C, W, ldx, ldy, act, DTYPE[dt],
                                         _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_short_conv_varlen", rc)
    return y, state_out


def kda_short_conv_step(x, weight, state, bias=None, *, activation="silu", y=None, stream=None):
    """One token for every sequence: x [B, C], state [B, W-1, C] shifted in place.  Returns y [B, C]."""
    B = x.shape[0]
    C, W, y, ldx, ldy, w, b, act = _conv_common(x, (B,), weight, bias, y, activation, stream)
    dev, dt = x.device, x.dtype
    _dense(state, "state", (B, W - 1, C), dt, dev)
    with _on_device(dev):
        rc = lib().kda_short_conv_step(x.data_ptr(), w, b, state.data_ptr(), y.data_ptr(), B, C, W, ldx, ldy, act,
                                       DTYPE[dt], _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_short_conv_step", rc)
    return y


def kda_short_conv_step_paged(x, weight, state_pool, slots, bias=None, *, activation="silu", y=None, stream=None):
    """kda_short_conv_step with the states in a pool [n_slots, W-1, C]: slots int32 [B] on the device, as
    kda_decode_step_paged."""
    B = x.shape[0]
    C, W, y, ldx, ldy, w, b, act = _conv_common(x, (B,), weight, bias, y, activation, stream)
    dev, dt = x.device, x.dtype
    n_slots = state_pool.shape[0]
    _dense(state_pool, "state_pool", (n_slots, W - 1, C), dt, dev)
    _dense(slots, "slots", (B,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().kda_short_conv_step_paged(x.data_ptr(), w, b, state_pool.data_ptr(), n_slots, slots.data_ptr(),
                                             y.data_ptr(), B, C, W, ldx, ldy, act, DTYPE[dt], _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_short_conv_step_paged", rc)
    return y


def _ssm_common(x, dt, A, Bm, Cm, D, dt_bias, lead, y, stream):
    """The checks the scan's forms share: (H, G, N, P, y, row spacings, D and dt_bias pointers)."""
    H, P = x.shape[-2:]
    G, N = Bm.shape[-2:]
    dev, ty = x.device, x.dtype
    _dtype_code(ty)
    lds = (_rows(x, "x", lead, (H, P), ty, dev), _rows(dt, "dt", lead, (H,), ty, dev),
           _rows(Bm, "Bm", lead, (G, N), ty, dev), _rows(Cm, "Cm", lead, (G, N), ty, dev))
    _dense(A, "A", (H,), torch.float32, dev)
    d, bias = _vector(D, "D", H, torch.float32, dev), _vector(dt_bias, "dt_bias", H, torch.float32, dev)
    if y is None:
        y = _empty(lead + (H, P), ty, dev, stream, x)
    else:
        _dense(y, "y", lead + (H, P), ty, dev)
    return H, G, N, P, y, lds, d, bias


def ssm_workspace_bytes(n_seq: int, T_total: int, H: int, N: int = 128, P: int = 128, dtype=torch.bfloat16,
                        impl: str = "auto") -> int:
    """Bytes of device workspace kda_ssm_forward (n_seq = B, T_total = B * T) or kda_ssm_forward_varlen needs."""
    return int(lib().kda_ssm_workspace(int(n_seq), int(T_total), int(H), int(N), int(P), _dtype_code(dtype), IMPL[impl]))


def _ssm_workspace(workspace, n_seq, T_total, H, N, P, dt, dev, impl, stream):
    need = lib().kda_ssm_workspace(n_seq, T_total, H, N, P, DTYPE[dt], IMPL[impl])
    if workspace is None:
        return _empty((need,), torch.uint8, dev, stream) if need else None
    if not (isinstance(workspace, torch.Tensor) and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def kda_ssm_forward(x, dt, A, Bm, Cm, D=None, dt_bias=None, S0=None, *, y=None, S_T=None, return_state: bool = True,
                    workspace=None, impl: str = "auto", stream=None):
    """Prefill of the selective scan with one decay per head: x [B, T, H, P], dt [B, T, H], Bm, Cm
    [B, T, G, N] (bf16 or fp32; token rows may be slices of wider ones), A, D, dt_bias [H] fp32, S0
    [B, H, N, P] fp32.  Returns (y [B, T, H, P], S_T [B, H, N, P] or None).  S_T may be S0 itself.
    `workspace`: a device tensor of ssm_workspace_bytes(B, B * T, ...) bytes, allocated if not given.

    bf16 runs on the tensor core ("auto"): the state is held in fp32, but read for y as a bf16 operand, its new
    terms are off by up to 3 * 2**-16, and it loses up to 16 * 2**-23 of itself for each 128 tokens that it
    remembers; a NaN or infinity in one token's x, B or dt may reach other tokens of
    its 128-token block, earlier ones too.  impl="simt" computes in fp32, token by token, and takes many times as
    long."""
    B, T = x.shape[:2]
    H, G, N, P, y, lds, d, bias = _ssm_common(x, dt, A, Bm, Cm, D, dt_bias, (B, T), y, stream)
    dev, ty = x.device, x.dtype
    if S0 is not None:
        _dense(S0, "S0", (B, H, N, P), torch.float32, dev)
    if S_T is not None:
        _dense(S_T, "S_T", (B, H, N, P), torch.float32, dev)
    elif return_state:
        S_T = _empty((B, H, N, P), torch.float32, dev, stream, S0)
    with _on_device(dev):
        workspace = _ssm_workspace(workspace, B, B * T, H, N, P, ty, dev, impl, stream)
        rc = lib().kda_ssm_forward(x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), d, bias,
                                   _ptr(S0), y.data_ptr(), _ptr(S_T), B, T, H, G, N, P, *lds, DTYPE[ty], IMPL[impl],
                                   _ptr(workspace), _nbytes(workspace), _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_ssm_forward", rc)
    return y, S_T


def kda_ssm_forward_varlen(x, dt, A, Bm, Cm, cu_seqlens, D=None, dt_bias=None, S0=None, *, y=None, S_T=None,
                           return_state: bool = True, workspace=None, impl: str = "auto", stream=None):
    """kda_ssm_forward over packed sequences: x [T_total, H, P], dt [T_total, H], Bm, Cm [T_total, G, N],
    cu_seqlens int32 [n_seq + 1] on the device, states [n_seq, H, N, P].  Returns (y [T_total, H, P], S_T or
    None).  Long sequences are cut into parts that run side by side by the mean length: one long sequence among
    many short ones is faster in a call of its own."""
    T_total = x.shape[0]
    n_seq = cu_seqlens.shape[0] - 1
    H, G, N, P, y, lds, d, bias = _ssm_common(x, dt, A, Bm, Cm, D, dt_bias, (T_total,), y, stream)
    dev, ty = x.device, x.dtype
    _dense(cu_seqlens, "cu_seqlens", (n_seq + 1,), torch.int32, dev)
    if S0 is not None:
        _dense(S0, "S0", (n_seq, H, N, P), torch.float32, dev)
    if S_T is not None:
        _dense(S_T, "S_T", (n_seq, H, N, P), torch.float32, dev)
    elif return_state:
        S_T = _empty((n_seq, H, N, P), torch.float32, dev, stream, S0)
    with _on_device(dev):
        workspace = _ssm_workspace(workspace, n_seq, T_total, H, N, P, ty, dev, impl, stream)
        rc = lib().kda_ssm_forward_varlen(x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
                                          cu_seqlens.data_ptr(), d, bias, _ptr(S0), y.data_ptr(), _ptr(S_T), n_seq,
                                          T_total, H, G, N, P, *lds, DTYPE[ty], IMPL[impl], _ptr(workspace),
                                          _nbytes(workspace), _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_ssm_forward_varlen", rc)
    return y, S_T


def kda_ssm_decode_step(x, dt, A, Bm, Cm, S, D=None, dt_bias=None, *, y=None, stream=None):
    """One token of the selective scan for every (b, h): x [B, H, P], dt [B, H], Bm, Cm [B, G, N]; S
    [B, H, N, P] fp32 updated in place.  Returns y [B, H, P]."""
    B = x.shape[0]
    H, G, N, P, y, lds, d, bias = _ssm_common(x, dt, A, Bm, Cm, D, dt_bias, (B,), y, stream)
    dev, ty = x.device, x.dtype
    _dense(S, "S", (B, H, N, P), torch.float32, dev)
    with _on_device(dev):
        rc = lib().kda_ssm_decode_step(x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), d,
                                       bias, S.data_ptr(), y.data_ptr(), B, H, G, N, P, *lds, DTYPE[ty],
                                       _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_ssm_decode_step", rc)
    return y


def kda_ssm_decode_step_paged(x, dt, A, Bm, Cm, S_pool, slots, D=None, dt_bias=None, *, y=None, stream=None):
    """kda_ssm_decode_step with the states in a pool [n_slots, H, N, P]: slots int32 [B] on the device, as
    kda_decode_step_paged."""
    B = x.shape[0]
    H, G, N, P, y, lds, d, bias = _ssm_common(x, dt, A, Bm, Cm, D, dt_bias, (B,), y, stream)
    dev, ty = x.device, x.dtype
    n_slots = S_pool.shape[0]
    _dense(S_pool, "S_pool", (n_slots, H, N, P), torch.float32, dev)
    _dense(slots, "slots", (B,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().kda_ssm_decode_step_paged(x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
                                             d, bias, S_pool.data_ptr(), n_slots, slots.data_ptr(), y.data_ptr(), B,
                                             H, G, N, P, *lds, DTYPE[ty], _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_ssm_decode_step_paged", rc)
    return y


def _dense_from(t) -> int:
    """The first dimension, 1 or later, from which on a pool tensor is one contiguous run."""
    shape, stride = t.shape, t.stride()
    run, d = 1, len(shape)
    while d > 1 and (stride[d - 1] == run or shape[d - 1] == 1):
        d -= 1
        run *= shape[d]
    return d


def _pools(pools, name: str, device=None, beside=None):
    """The kda_pool descriptions of a list of pool tensors [n_slots, ...]: (their bytes, number of slots, device).

    Dimension 0 counts the slots and may be spaced wider than a slot.  The others are contiguous, or dimension 1
    is spaced wider (the boundary states of one batch entry, S_mid[b].transpose(0, 1) of
    kda_forward_chunked_states).  A pool whose counterpart in `beside` is split along dimension 1 is split there
    too, so that both are described by the same runs."""
    if not pools:
        raise ValueError(f"{name} is empty")
    flat, n_slots = [], pools[0].shape[0]
    if device is None:
        device = pools[0].device
    for i, t in enumerate(pools):
        shape = t.shape
        if t.device != device:
            raise ValueError(f"{name}: a pool is on {t.device}, expected {device}")
        if len(shape) < 2 or shape[0] != n_slots:
            raise ValueError(f"{name}: pools have shape [{n_slots}, ...], got {tuple(shape)}")
        if t.is_contiguous() and (beside is None or beside[i].is_contiguous()):
            slot = t.nbytes // n_slots if n_slots else 0
            flat += (t.data_ptr(), slot, 1, 0, slot)
            continue
        first = _dense_from(t)
        if first > 2:
            raise ValueError(f"{name}: a pool's slots must be contiguous, or contiguous runs along dimension 1")
        if beside is not None:
            first = max(first, min(_dense_from(beside[i]), 2))
        stride, es = t.stride(), t.element_size()
        run = math.prod(shape[first:])
        pieces, apart = (1, 0) if first == 1 else (shape[1], stride[1])
        flat += (t.data_ptr(), (stride[0] if n_slots > 1 else max(stride[0], run)) * es, pieces, apart * es, run * es)
    return struct.pack(f"{len(flat)}q", *flat), n_slots, device


def kda_pool_copy(pools, src, dst, *, src_pools=None, stream=None) -> None:
    """Copy slots, in every pool of the list at once: slot dst[i] of each pool becomes its slot src[i] (of the
    pool in the same place of `src_pools`, when given).  Pools are tensors [n_slots, ...]; src, dst int32 [n]
    on the device, negative entries skip the pair.  One source may feed many destinations; a destination that
    another pair has too, or (within one pool) reads, is left as it was and reported by the status word."""
    if src_pools is None:
        to, n_dst, dev = _pools(pools, "pools")
        frm, n_src = to, n_dst
    else:
        if len(src_pools) != len(pools):
            raise ValueError(f"{len(src_pools)} source pools for {len(pools)} pools")
        for a, b in zip(pools, src_pools):
            if a.dtype != b.dtype or a.shape[1:] != b.shape[1:]:
                raise ValueError("a pool and its source pool must have slots of one shape and dtype")
        to, n_dst, dev = _pools(pools, "pools", beside=src_pools)
        frm, n_src, _ = _pools(src_pools, "src_pools", dev, beside=pools)
    n = src.shape[0]
    _dense(src, "src", (n,), torch.int32, dev)
    _dense(dst, "dst", (n,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().kda_pool_copy(to, frm, len(pools), n_dst, n_src, src.data_ptr(), dst.data_ptr(), n,
                                 _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_pool_copy", rc)


def kda_pool_clear(pools, slots, *, stream=None) -> None:
    """Set the listed slots (int32 [n] on the device, negative entries skipped) of every pool to zero."""
    to, n_slots, dev = _pools(pools, "pools")
    n = slots.shape[0]
    _dense(slots, "slots", (n,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().kda_pool_clear(to, len(pools), n_slots, slots.data_ptr(), n, _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_pool_clear", rc)


def kda_pool_compact(pools, slots, done=None, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Drop the sequences that ended (done [B] bool or uint8, or slots[b] < 0) and move the others' slots to
    the front of every pool.  Returns the new slot table, int32 [B] (-1 for ended sequences); `out` may be
    `slots` itself.  `workspace`: int32 [n_slots + 1] on the device, allocated if not given."""
    to, n_slots, dev = _pools(pools, "pools")
    B = slots.shape[0]
    _dense(slots, "slots", (B,), torch.int32, dev)
    if done is not None:
        _dense(done, "done", (B,), torch.uint8 if done.dtype == torch.uint8 else torch.bool, dev)
    if out is None:
        out = _empty((B,), torch.int32, dev, stream, slots)
    else:
        _dense(out, "out", (B,), torch.int32, dev)
    if workspace is None:
        workspace = _empty((n_slots + 1,), torch.int32, dev, stream)
    else:
        _dense(workspace, "workspace", (n_slots + 1,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().kda_pool_compact(to, len(pools), n_slots, slots.data_ptr(), _ptr(done), out.data_ptr(), B,
                                    workspace.data_ptr(), _stream_on(dev, stream))
    if rc != 0:
        raise KdaError("kda_pool_compact", rc)
    return out


def kda_get_device_status(stream=None, device=None) -> int:
    """Synchronise the stream, then return and clear the device status word (0 = OK)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().kda_get_device_status(_stream_handle(stream)))


def kda_debug_set_wait_fault(mode: int, timeout_ns: int = 0) -> None:
    """Test hook: mode 1 makes tensor-core prefill launches time out a bounded device wait."""
    rc = lib().kda_debug_set_wait_fault(int(mode), int(timeout_ns))
    if rc != 0:
        raise KdaError("kda_debug_set_wait_fault", rc)
