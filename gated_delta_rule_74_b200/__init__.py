"""gated_delta_rule_74_b200: B200 (sm_100a) Kimi Delta Attention (KDA).

Thin ctypes binding over libkda.so, whose C ABI is declared in include/kda.h.
The functions here only marshal torch CUDA tensors into pointers and sizes and
call the library on the current torch stream; every step of the computation runs
in the library's CUDA kernels.  There is no fallback: if libkda.so is missing or a
call fails, an exception is raised.

    out, hT = kda_chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None)
    out     = kda_decode_step(q, k, v, g, beta, S)        # S updated in place
    kda_latent_append(kv, kv_cache, page_table, seq_lens, rank=512, ...)
    out, lse = kda_latent_attn(q, kv_cache, page_table, seq_lens, rank=512, scale=s)
    tokens, accepted = kda_verify_tokens(target, draft, draft_tokens, uniforms)
    grads   = kda_chunk_bwd(q, k, v, g, beta, dout, h0=None, dhT=None, cu_seqlens=None)
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

__all__ = ["kda_chunk_fwd", "kda_chunk_fwd_fused", "kda_chunk_bwd", "kda_device_status",
           "kda_decode_chunk", "kda_decode_step", "kda_decode_tokens", "kda_status_string", "kda_version",
           "kda_launch_count",
           "lib", "library_path", "header_symbols", "KdaError",
           "KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_UNSUPPORTED", "KDA_ERR_CUDA",
           "KDA_ERR_TIMEOUT", "KDA_BF16", "KDA_F32", "KDA_OP_CHUNK_FWD", "KDA_OP_CHUNK_BWD",
           "kda_workspace_size", "kda_pool_usage", "kda_latent_append", "kda_latent_attn",
           "kda_latent_attn_workspace_size", "kda_verify_tokens"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_SO = os.path.join(_PKG, "libkda.so")
_HEADER = os.path.join(_ROOT, "include", "kda.h")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT = 0, -1, -2, -3, -4
KDA_BF16, KDA_F32 = 0, 1
KDA_OP_CHUNK_FWD, KDA_OP_CHUNK_BWD = 0, 1

_DTYPES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_lib = None


class KdaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {kda_status_string(status)} ({status})")


def _check_status(rc: int, fn: str = "kda_timing") -> None:
    if rc != 0:
        raise KdaError(fn, rc)


def library_path() -> str:
    return _SO


def lib() -> ctypes.CDLL:
    """Load libkda.so (built in-tree by gated_delta_rule_74_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_SO):
            raise RuntimeError(f"libkda.so is not built ({_SO}); run "
                               "`python -m gated_delta_rule_74_b200.build`")
        L = ctypes.CDLL(_SO)
        vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.kda_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp,
                                    ip, ip, ip, ip, ip, ip, vp]
        L.kda_chunk_fwd.restype = ctypes.c_int
        L.kda_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp,
                                            ip, ip, ip, ip, ip, ip, vp]
        L.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        L.kda_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, ip, ip, ip, ip, ip, vp]
        L.kda_decode_step.restype = ctypes.c_int
        L.kda_decode_tokens.argtypes = [vp, vp, vp, fp, fp, fp, vp, ip, ip, ip, ip, ip, ip, vp]
        L.kda_decode_tokens.restype = ctypes.c_int
        L.kda_decode_chunk.argtypes = [vp, vp, vp, fp, fp, fp, vp, ip, ip, ip, ip, ip, ip, vp]
        L.kda_decode_chunk.restype = ctypes.c_int
        L.kda_decode_tokens_grouped.argtypes = [vp, vp, vp, fp, fp, fp, vp] + [ip] * 7 + [vp]
        L.kda_decode_tokens_grouped.restype = ctypes.c_int
        L.kda_chunk_fwd_grouped.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp] + [ip] * 7 + [vp]
        L.kda_chunk_fwd_grouped.restype = ctypes.c_int
        L.kda_chunk_fwd_fused.argtypes = [vp, vp, vp, fp, fp, ip, fp, fp, vp, fp, vp, vp, fp] + \
            [ip] * 6 + [vp]
        L.kda_chunk_fwd_fused.restype = ctypes.c_int
        L.kda_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp,
                                    fp, fp, fp, fp, fp, fp] + [ip] * 6 + [vp]
        L.kda_chunk_bwd.restype = ctypes.c_int
        L.kda_chunk_bwd_grouped.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp,
                                            fp, fp, fp, fp, fp, fp] + [ip] * 7 + [vp]
        L.kda_chunk_bwd_grouped.restype = ctypes.c_int
        L.kda_chunk_bwd_recurrent.argtypes = L.kda_chunk_bwd_grouped.argtypes
        L.kda_chunk_bwd_recurrent.restype = ctypes.c_int
        L.kda_device_status.argtypes = [ip]
        L.kda_device_status.restype = ctypes.c_int
        L.kda_selftest_bounded_wait.argtypes = [ctypes.c_uint, vp]
        L.kda_selftest_bounded_wait.restype = ctypes.c_int
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_version.argtypes = []
        L.kda_version.restype = ctypes.c_int
        L.kda_launch_count.argtypes = []
        L.kda_launch_count.restype = ctypes.c_ulonglong
        L.kda_prefill_plan.argtypes = [ctypes.c_int] * 5 + [ctypes.POINTER(ctypes.c_int)] * 2
        L.kda_prefill_plan.restype = ctypes.c_int
        L.kda_timing_start.argtypes = []
        L.kda_timing_start.restype = ctypes.c_int
        L.kda_timing_stop.argtypes = []
        L.kda_timing_stop.restype = ctypes.c_int
        L.kda_timing_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_ulonglong),
                                      ctypes.POINTER(ctypes.c_double)]
        L.kda_timing_read.restype = ctypes.c_int
        sz = ctypes.c_size_t
        L.kda_workspace_size.argtypes = [ctypes.c_int] * 9 + [ctypes.POINTER(sz)]
        L.kda_workspace_size.restype = ctypes.c_int
        L.kda_chunk_fwd_ws.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp] + [ip] * 7 + [vp, sz, vp]
        L.kda_chunk_fwd_ws.restype = ctypes.c_int
        L.kda_chunk_bwd_ws.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp,
                                       fp, fp, fp, fp, fp, fp] + [ip] * 7 + [vp, sz, vp]
        L.kda_chunk_bwd_ws.restype = ctypes.c_int
        ll, cf = ctypes.c_longlong, ctypes.c_float
        L.kda_latent_append.argtypes = [vp] * 9 + [ip] * 8 + [ll] * 7 + [cf, ip, ip, vp]
        L.kda_latent_append.restype = ctypes.c_int
        L.kda_latent_attn.argtypes = [vp] * 7 + [ip] * 8 + [ll, ll, cf, ip, vp]
        L.kda_latent_attn.restype = ctypes.c_int
        L.kda_latent_attn_ws.argtypes = L.kda_latent_attn.argtypes[:-1] + [vp, sz, vp]
        L.kda_latent_attn_ws.restype = ctypes.c_int
        L.kda_selftest_latent_waits.argtypes = [ctypes.c_uint, *L.kda_latent_attn.argtypes[:-2], vp]
        L.kda_selftest_latent_waits.restype = ctypes.c_int
        L.kda_latent_attn_workspace_size.argtypes = [ip] * 9 + [ctypes.POINTER(sz)]
        L.kda_latent_attn_workspace_size.restype = ctypes.c_int
        L.kda_verify_tokens.argtypes = [vp] * 7 + [ip] * 3 + [vp]
        L.kda_verify_tokens.restype = ctypes.c_int
        L.kda_pool_usage.argtypes = [ip, ctypes.POINTER(ctypes.c_ulonglong)]
        L.kda_pool_usage.restype = ctypes.c_int
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Names of the functions include/kda.h declares."""
    with open(_HEADER) as f:
        text = f.read()
    return re.findall(r"^KDA_API\s+[\w\s\*]*?\b(kda_\w+)\s*\(", text, flags=re.M)


def kda_workspace_size(op: int, B: int, T: int, H: int, dk: int, dv: int, packed: bool = False,
                       dtype: int = KDA_BF16, sms: int = 0) -> int:
    """Workspace bytes of one kda_chunk_fwd_ws (op KDA_OP_CHUNK_FWD) or kda_chunk_bwd_ws
    (KDA_OP_CHUNK_BWD) call; sms = 0 asks the current device."""
    out = ctypes.c_size_t(0)
    rc = lib().kda_workspace_size(int(op), int(B), int(T), int(H), int(dk), int(dv),
                                  1 if packed else 0, int(dtype), int(sms), ctypes.byref(out))
    if rc != KDA_OK:
        raise KdaError("kda_workspace_size", rc)
    return int(out.value)


def kda_pool_usage(reset: bool = False) -> int:
    """Most bytes the library pool of the current device has had in use at once."""
    out = ctypes.c_ulonglong(0)
    rc = lib().kda_pool_usage(1 if reset else 0, ctypes.byref(out))
    if rc != KDA_OK:
        raise KdaError("kda_pool_usage", rc)
    return int(out.value)


def _workspace_args(workspace: Optional[torch.Tensor]):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return int(lib().kda_version())


def kda_device_status(reset: bool = True) -> int:
    """KDA_OK, or KDA_ERR_TIMEOUT if a bounded device-side wait of the library's kernels
    gave up since the last reset (synchronizes the device; see include/kda.h)."""
    rc = int(lib().kda_device_status(1 if reset else 0))
    if rc not in (KDA_OK, KDA_ERR_TIMEOUT):
        raise KdaError("kda_device_status", rc)
    return rc


def kda_selftest_bounded_wait(polls: int = 1000, stream=None) -> None:
    """Launch the self-test whose wait nothing completes (see include/kda.h)."""
    rc = lib().kda_selftest_bounded_wait(int(polls), _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_selftest_bounded_wait", rc)


def kda_launch_count() -> int:
    """Kernels launched by libkda in this process so far."""
    return int(lib().kda_launch_count())


def kda_prefill_plan(B: int, T: int, H: int, packed: bool = False, sms: int = 148) -> tuple:
    """(chunks per segment, chunks of a half point) that kda_chunk_fwd's split takes for
    B sequences of T tokens (packed: T tokens in B documents) over H heads on `sms` SMs;
    (0, 0) when sequences are not split.  Host only."""
    G, half = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().kda_prefill_plan(B, T, H, int(bool(packed)), sms, ctypes.byref(G),
                                ctypes.byref(half))
    _check_status(rc, "kda_prefill_plan")
    return int(G.value), int(half.value)


KERNEL_KINDS = {"prep": 0, "state": 1, "combine": 2, "fused": 3, "simt": 4, "decode": 5,
                "bwd": 6, "bwd_prep": 7, "bwd_chain": 8, "bwd_grad": 9, "latent_append": 10,
                "latent_attn": 11, "verify": 12}


def kda_timing_start() -> None:
    """Start bracketing every library kernel launch with CUDA events."""
    _check_status(lib().kda_timing_start())


def kda_timing_stop() -> None:
    _check_status(lib().kda_timing_stop())


def kda_timing_read() -> dict:
    """{kind: (launches, total_ms)} since kda_timing_start(); waits for the events."""
    res = {}
    for name, kind in KERNEL_KINDS.items():
        n = ctypes.c_ulonglong(0)
        ms = ctypes.c_double(0.0)
        _check_status(lib().kda_timing_read(kind, ctypes.byref(n), ctypes.byref(ms)))
        res[name] = (int(n.value), float(ms.value))
    return res


def _decay_group(g: torch.Tensor, dk: int) -> int:
    """Channels per decay value implied by g's last dimension."""
    n = g.shape[-1]
    if n < 1 or dk % n != 0 or (dk // n) & (dk // n - 1):
        raise ValueError(f"g's last dimension {n} must be dk / G with G a power of two")
    return dk // n


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (0.07 us a call, not 3), and
# the current device without the check that CUDA is up.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    """Handle of `stream`, by default of the current device's current stream."""
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _new(stream, like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """An output that the call writes on `stream`: its memory comes from that stream's pool, as
    memory of the current stream's may still be in use there."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _check(name: str, t: torch.Tensor, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def kda_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, h0: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  hT: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  stream=None, noalloc: bool = False, workspace: Optional[torch.Tensor] = None):
    """KDA prefill (chunked form).  q, k [B,T,H,dk]; v [B,T,H,dv]; g [B,T,H,dk] f32
    (or [B,T,H,dk/G] for one decay per group of G key channels, G a power of two:
    kda_chunk_fwd_grouped); beta [B,T,H] f32; h0 [Nseq,H,dk,dv] f32 or None;
    cu_seqlens int32 [Nseq+1] on the device, or None.  Returns (out, hT) (hT None
    if output_final_state is False and no hT buffer was given).  noalloc=True calls
    kda_chunk_fwd_noalloc instead (per-channel decay only); a ``workspace`` tensor
    (kda_workspace_size bytes, e.g. torch.uint8) calls kda_chunk_fwd_ws on it."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, dk]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check("q", q)
    _check("k", k, q.dtype, (Bt, T, H, dk))
    _check("v", v, q.dtype, (Bt, T, H, dv))
    G = _decay_group(g, dk)
    _check("g", g, torch.float32, (Bt, T, H, dk // G))
    _check("beta", beta, torch.float32, (Bt, T, H))
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32)
        if Bt != 1:
            raise ValueError("packed inputs (cu_seqlens) must have B == 1")
        nseq = cu_seqlens.numel() - 1
    else:
        nseq = Bt
    if h0 is not None:
        _check("h0", h0, torch.float32, (nseq, H, dk, dv))
    if out is None:
        out = _new(stream, q, (Bt, T, H, dv), q.dtype)
    _check("out", out, q.dtype, (Bt, T, H, dv))
    if hT is None and output_final_state:
        hT = _new(stream, q, (nseq, H, dk, dv), torch.float32)
    if hT is not None:
        _check("hT", hT, torch.float32, (nseq, H, dk, dv))
    if noalloc and G != 1:
        raise ValueError("kda_chunk_fwd_noalloc takes one decay per key channel")
    if workspace is not None:
        wp, wb = _workspace_args(workspace)
        rc = lib().kda_chunk_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                    _ptr(cu_seqlens), _ptr(out), _ptr(hT), nseq, T, H, dk, dv, G,
                                    dt, wp, wb, _stream(stream))
        if rc != KDA_OK:
            raise KdaError("kda_chunk_fwd_ws", rc)
        return out, hT
    if G == 1:
        fn = lib().kda_chunk_fwd_noalloc if noalloc else lib().kda_chunk_fwd
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                _ptr(cu_seqlens), _ptr(out), _ptr(hT), nseq, T, H, dk, dv, dt, _stream(stream))
    else:
        rc = lib().kda_chunk_fwd_grouped(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         _ptr(h0), _ptr(cu_seqlens), _ptr(out), _ptr(hT),
                                         nseq, T, H, dk, dv, G, dt, _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_chunk_fwd_noalloc" if noalloc else "kda_chunk_fwd", rc)
    return out, hT


def kda_chunk_fwd_fused(q_raw: torch.Tensor, k_raw: torch.Tensor, v: torch.Tensor,
                        g: torch.Tensor, beta: torch.Tensor,
                        conv_q: Optional[torch.Tensor] = None,
                        conv_k: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                        cu_seqlens: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, hT: Optional[torch.Tensor] = None,
                        output_final_state: bool = True, stream=None):
    """KDA prefill with the q/k prep and the output gate fused (bf16 only):
    q = dk^-1/2 n(conv_q * q_raw), k = n(conv_k * k_raw) (causal per-channel convolutions
    of width W, conv_* [H, dk, W] f32, n = L2 normalisation per token and head),
    out = o * sigmoid(gate) (gate [B,T,H,dv] bf16 or None).  Returns (out, hT)."""
    if q_raw.dim() != 4:
        raise ValueError("q_raw must be [B, T, H, dk]")
    Bt, T, H, dk = q_raw.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q_raw.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q_raw.dtype}")
    _check("q_raw", q_raw)
    _check("k_raw", k_raw, q_raw.dtype, (Bt, T, H, dk))
    _check("v", v, q_raw.dtype, (Bt, T, H, dv))
    _check("g", g, torch.float32, (Bt, T, H, dk))
    _check("beta", beta, torch.float32, (Bt, T, H))
    W = 0
    if (conv_q is None) != (conv_k is None):
        raise ValueError("give both conv_q and conv_k, or neither")
    if conv_q is not None:
        W = conv_q.shape[-1]
        _check("conv_q", conv_q, torch.float32, (H, dk, W))
        _check("conv_k", conv_k, torch.float32, (H, dk, W))
    if gate is not None:
        _check("gate", gate, q_raw.dtype, (Bt, T, H, dv))
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32)
        if Bt != 1:
            raise ValueError("packed inputs (cu_seqlens) must have B == 1")
        nseq = cu_seqlens.numel() - 1
    else:
        nseq = Bt
    if h0 is not None:
        _check("h0", h0, torch.float32, (nseq, H, dk, dv))
    if out is None:
        out = _new(stream, q_raw, (Bt, T, H, dv), q_raw.dtype)
    _check("out", out, q_raw.dtype, (Bt, T, H, dv))
    if hT is None and output_final_state:
        hT = _new(stream, q_raw, (nseq, H, dk, dv), torch.float32)
    if hT is not None:
        _check("hT", hT, torch.float32, (nseq, H, dk, dv))
    rc = lib().kda_chunk_fwd_fused(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(conv_q), _ptr(conv_k),
                                   W, _ptr(g), _ptr(beta), _ptr(gate), _ptr(h0),
                                   _ptr(cu_seqlens), _ptr(out), _ptr(hT), nseq, T, H, dk, dv, dt,
                                   _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_chunk_fwd_fused", rc)
    return out, hT


def kda_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, dout: torch.Tensor, h0: Optional[torch.Tensor] = None,
                  dhT: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  grads: Optional[dict] = None, stream=None,
                  workspace: Optional[torch.Tensor] = None, recurrent: bool = False) -> dict:
    """Gradients of L = sum(out * dout) + sum(hT * dhT) for kda_chunk_fwd with the same
    inputs.  g [B,T,H,dk] f32, or [B,T,H,dk/G] for one decay per group of G key channels
    (kda_chunk_bwd_grouped; dg then has g's shape).  dout has out's shape and dtype; dhT
    [Nseq,H,dk,dv] f32 or None.  Returns a dict of fp32 tensors dq, dk, dv, dg, dbeta, dh0
    (dh0 None when h0 is None); ``grads`` may hold preallocated outputs under those names;
    a ``workspace`` tensor (kda_workspace_size bytes) calls kda_chunk_bwd_ws on it;
    ``recurrent`` calls kda_chunk_bwd_recurrent (the fp32 reverse sweep) instead."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, dk]")
    Bt, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check("q", q)
    _check("k", k, q.dtype, (Bt, T, H, dk))
    _check("v", v, q.dtype, (Bt, T, H, dv))
    G = _decay_group(g, dk)
    _check("g", g, torch.float32, (Bt, T, H, dk // G))
    _check("beta", beta, torch.float32, (Bt, T, H))
    _check("dout", dout, q.dtype, (Bt, T, H, dv))
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32)
        if Bt != 1:
            raise ValueError("packed inputs (cu_seqlens) must have B == 1")
        nseq = cu_seqlens.numel() - 1
    else:
        nseq = Bt
    if h0 is not None:
        _check("h0", h0, torch.float32, (nseq, H, dk, dv))
    if dhT is not None:
        _check("dhT", dhT, torch.float32, (nseq, H, dk, dv))
    shapes = {"dq": (Bt, T, H, dk), "dk": (Bt, T, H, dk), "dv": (Bt, T, H, dv),
              "dg": (Bt, T, H, dk // G), "dbeta": (Bt, T, H), "dh0": (nseq, H, dk, dv)}
    res = dict(grads or {})
    for name, shp in shapes.items():
        if name == "dh0" and h0 is None and res.get(name) is None:
            res[name] = None
            continue
        if res.get(name) is None:
            res[name] = _new(stream, q, shp, torch.float32)
        _check(name, res[name], torch.float32, shp)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
            _ptr(dout), _ptr(dhT), _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]),
            _ptr(res["dg"]), _ptr(res["dbeta"]), _ptr(res["dh0"]), nseq, T, H, dk, dv]
    if recurrent:
        if workspace is not None:
            raise ValueError("the recurrent backward takes no workspace")
        rc = lib().kda_chunk_bwd_recurrent(*args, G, dt, _stream(stream))
        if rc != KDA_OK:
            raise KdaError("kda_chunk_bwd_recurrent", rc)
        return res
    if workspace is not None:
        wp, wb = _workspace_args(workspace)
        rc = lib().kda_chunk_bwd_ws(*args, G, dt, wp, wb, _stream(stream))
        if rc != KDA_OK:
            raise KdaError("kda_chunk_bwd_ws", rc)
        return res
    if G == 1:
        rc = lib().kda_chunk_bwd(*args, dt, _stream(stream))
    else:
        rc = lib().kda_chunk_bwd_grouped(*args, G, dt, _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_chunk_bwd", rc)
    return res


def kda_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, S: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """One KDA decode step.  q, k [N,H,dk]; v [N,H,dv]; g [N,H,dk] f32; beta [N,H] f32;
    S [N,H,dk,dv] f32, updated in place.  Returns out [N,H,dv]."""
    if q.dim() != 3:
        raise ValueError("q must be [N, H, dk]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check("q", q)
    _check("k", k, q.dtype, (N, H, dk))
    _check("v", v, q.dtype, (N, H, dv))
    _check("g", g, torch.float32, (N, H, dk))
    _check("beta", beta, torch.float32, (N, H))
    _check("S", S, torch.float32, (N, H, dk, dv))
    if out is None:
        out = _new(stream, q, (N, H, dv), q.dtype)
    _check("out", out, q.dtype, (N, H, dv))
    rc = lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
                               _ptr(out), N, H, dk, dv, dt, _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_decode_step", rc)
    return out


def kda_decode_tokens(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                      beta: torch.Tensor, S: torch.Tensor, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """L consecutive KDA decode steps in one launch.  q, k [N,L,H,dk]; v [N,L,H,dv];
    g [N,L,H,dk] f32; beta [N,L,H] f32; S [N,H,dk,dv] f32, updated in place (state
    after the last token).  Returns out [N,L,H,dv]; identical to L kda_decode_step
    calls."""
    if q.dim() != 4:
        raise ValueError("q must be [N, L, H, dk]")
    N, L, H, dk = q.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check("q", q)
    _check("k", k, q.dtype, (N, L, H, dk))
    _check("v", v, q.dtype, (N, L, H, dv))
    G = _decay_group(g, dk)
    _check("g", g, torch.float32, (N, L, H, dk // G))
    _check("beta", beta, torch.float32, (N, L, H))
    _check("S", S, torch.float32, (N, H, dk, dv))
    if out is None:
        out = _new(stream, q, (N, L, H, dv), q.dtype)
    _check("out", out, q.dtype, (N, L, H, dv))
    if G == 1:
        rc = lib().kda_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
                                     _ptr(out), N, L, H, dk, dv, dt, _stream(stream))
    else:
        rc = lib().kda_decode_tokens_grouped(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                             _ptr(S), _ptr(out), N, L, H, dk, dv, G, dt,
                                             _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_decode_tokens", rc)
    return out


def kda_decode_chunk(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, S: torch.Tensor, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """L <= 16 tokens per (sequence, head) as one chunk of the chunked form on the tensor
    cores (bf16, dk = dv = 128).  Same layout and in-place S update as kda_decode_tokens;
    equal to L single steps up to the tensor-core rounding.  Returns out [N,L,H,dv]."""
    if q.dim() != 4:
        raise ValueError("q must be [N, L, H, dk]")
    N, L, H, dk = q.shape
    dv = v.shape[-1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check("q", q)
    _check("k", k, q.dtype, (N, L, H, dk))
    _check("v", v, q.dtype, (N, L, H, dv))
    _check("g", g, torch.float32, (N, L, H, dk))
    _check("beta", beta, torch.float32, (N, L, H))
    _check("S", S, torch.float32, (N, H, dk, dv))
    if out is None:
        out = _new(stream, q, (N, L, H, dv), q.dtype)
    _check("out", out, q.dtype, (N, L, H, dv))
    rc = lib().kda_decode_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
                                _ptr(out), N, L, H, dk, dv, dt, _stream(stream))
    if rc != KDA_OK:
        raise KdaError("kda_decode_chunk", rc)
    return out


# ------------------------------------------------ latent attention, drafted tokens

def _run_on(dev: int, stream, fn, args, name: str) -> None:
    """fn(*args, stream handle) with device `dev` current (the library works on that one)."""
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != KDA_OK:
        raise KdaError(name, rc)


def _device_of(name: str, t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _take(name: str, t: Optional[torch.Tensor], dev: int, dtype, shape) -> Optional[int]:
    """Pointer of an optional contiguous tensor on device `dev`; one test for all of it, as a
    decode step's calls are as short as their checks."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _check(name, t, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")


def _latent_args(B: int, T: int, D: int, dtype, dev: int, kv_cache: torch.Tensor,
                 page_table: torch.Tensor, seq_lens: torch.Tensor,
                 cu_seqlens: Optional[torch.Tensor], rank: int):
    """Checks shared by kda_latent_append and kda_latent_attn: (the pointers of cache, table,
    lengths and offsets), sequences, (cache and table sizes and strides), dtype id."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    if not 0 < rank <= D:
        raise ValueError(f"rank {rank} does not fit rows of {D}")
    shape = kv_cache.shape
    if len(shape) != 3 or shape[2] != D or kv_cache.dtype is not dtype:
        raise ValueError(f"kv_cache must be [pages, page_size, {D}] of {dtype}, got "
                         f"{tuple(shape)} of {kv_cache.dtype}")
    page_stride, row_stride, one = kv_cache.stride()
    if one != 1 or kv_cache.get_device() != dev:
        raise ValueError(f"kv_cache must be a tensor on cuda:{dev} with contiguous rows")
    nseq = seq_lens.numel()
    cu = None
    if cu_seqlens is not None:
        cu = _take("cu_seqlens", cu_seqlens, dev, torch.int32, (nseq + 1,))
        if B != 1:
            raise ValueError("packed inputs (cu_seqlens) must have B == 1")
    elif nseq != B:
        raise ValueError(f"seq_lens has {nseq} entries for {B} sequences")
    most = page_table.shape[-1] if page_table.dim() == 2 else -1
    return ((kv_cache.data_ptr(), _take("page_table", page_table, dev, torch.int32, (nseq, most)),
             _take("seq_lens", seq_lens, dev, torch.int32, (nseq,)), cu), nseq,
            (shape[0], shape[1], most, page_stride, row_stride), dt)


def _token_stride(name: str, t: torch.Tensor, dense: int) -> int:
    """Elements from one token of t [B, T, ..] to the next, which has to hold across B
    (`dense` where there is but one token)."""
    (B, T), s = t.shape[:2], t.stride()
    if T > 1:
        if B > 1 and s[0] != T * s[1]:
            raise ValueError(f"{name}'s sequences must follow each other at its token stride")
        return s[1]
    return s[0] if B > 1 else dense


def _position_values(name: str, t: torch.Tensor, shape, dtype, dev: int):
    """Pointer, token stride and head stride of the queries' position values."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    s = t.stride()
    if s[3] != 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev} with contiguous rows")
    H, rope = shape[2:]
    return t.data_ptr(), _token_stride(name, t, H * rope), s[2] if H > 1 else rope


def kda_latent_append(kv: torch.Tensor, kv_cache: torch.Tensor, page_table: torch.Tensor,
                      seq_lens: torch.Tensor, *, rank: int,
                      cu_seqlens: Optional[torch.Tensor] = None,
                      norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                      q_pe: Optional[torch.Tensor] = None,
                      q_pe_out: Optional[torch.Tensor] = None, stream=None):
    """Norm, rotate and write the new tokens' latent rows to the paged cache, in place.
    kv [N, L, rank + rope] (or [1, T, ..] with cu_seqlens int32 [N+1]); kv_cache
    [pages, page_size, rank + rope]; page_table int32 [N, max_pages]; seq_lens int32 [N],
    lengths with the new tokens; norm_weight f32 [rank] or None; inv_freq f32 [rope/2] or
    None.  With q_pe [N, L, H, rope], its rotation goes to q_pe_out (default: a new
    tensor), e.g. the view q[..., rank:] of the queries kda_latent_attn takes.  kv, q_pe
    and q_pe_out may be strided over tokens and heads.  Returns q_pe_out (None without)."""
    if kv.dim() != 3:
        raise ValueError("kv must be [B, T, rank + rope]")
    B, T, D = kv.shape
    dev, dtype, rope = _device_of("kv", kv), kv.dtype, D - rank
    ptrs, nseq, sizes, dt = _latent_args(B, T, D, dtype, dev, kv_cache, page_table, seq_lens,
                                         cu_seqlens, rank)
    if kv.stride(2) != 1:
        raise ValueError("kv must have contiguous rows")
    H, qp, qt, qh, op, ot, oh = 1, None, 0, 0, None, 0, 0
    if q_pe is not None:
        if q_pe_out is None:
            q_pe_out = _new(stream, q_pe, q_pe.shape, q_pe.dtype)
        H = q_pe.shape[2] if q_pe.dim() == 4 else 0
        qp, qt, qh = _position_values("q_pe", q_pe, (B, T, H, rope), dtype, dev)
        op, ot, oh = _position_values("q_pe_out", q_pe_out, (B, T, H, rope), dtype, dev)
    elif q_pe_out is not None:
        raise ValueError("q_pe_out needs q_pe")
    _run_on(dev, stream, lib().kda_latent_append,
            (kv.data_ptr(), _take("norm_weight", norm_weight, dev, torch.float32, (rank,)),
             _take("inv_freq", inv_freq, dev, torch.float32, (rope // 2,)), qp, op, *ptrs, nseq, T, H,
             rank, rope, *sizes, _token_stride("kv", kv, D), qt, qh, ot, oh, eps, interleaved, dt),
            "kda_latent_append")
    return q_pe_out


def kda_latent_attn_workspace_size(N: int, L: int, H: int, rank: int, rope: int, page_size: int,
                                   packed: bool = False, dtype: int = KDA_BF16,
                                   sms: int = 0) -> int:
    """Workspace bytes of one kda_latent_attn call (L: new tokens a sequence, packed: in
    all); sms = 0 asks the current device."""
    out = ctypes.c_size_t(0)
    rc = lib().kda_latent_attn_workspace_size(N, L, H, rank, rope, page_size, int(bool(packed)),
                                              int(dtype), int(sms), ctypes.byref(out))
    if rc != KDA_OK:
        raise KdaError("kda_latent_attn_workspace_size", rc)
    return int(out.value)


def kda_latent_attn(q: torch.Tensor, kv_cache: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, *, rank: int, scale: float,
                    cu_seqlens: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Absorbed latent attention of the new tokens over the paged cache, causal.
    q [N, L, H, rank + rope] (or [1, T, H, ..] with cu_seqlens int32 [N+1]); kv_cache
    [pages, page_size, rank + rope]; page_table int32 [N, max_pages]; seq_lens int32 [N],
    lengths with the new tokens.  Returns (out [.., H, rank] in q's type, lse [.., H] f32,
    the natural log of the scores' summed exponentials); a token that sees nothing gives 0
    and -inf.  A ``workspace`` tensor (kda_latent_attn_workspace_size bytes) calls
    kda_latent_attn_ws on it."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, rank + rope]")
    B, T, H, D = q.shape
    dev, dtype = _device_of("q", q), q.dtype
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    ptrs, nseq, sizes, dt = _latent_args(B, T, D, dtype, dev, kv_cache, page_table, seq_lens,
                                         cu_seqlens, rank)
    if out is None:
        out = _new(stream, q, (B, T, H, rank), dtype)
        op = out.data_ptr()
    else:
        op = _take("out", out, dev, dtype, (B, T, H, rank))
    if lse is None:
        lse = _new(stream, q, (B, T, H), torch.float32)
        lp = lse.data_ptr()
    else:
        lp = _take("lse", lse, dev, torch.float32, (B, T, H))
    args = (q.data_ptr(), *ptrs, op, lp, nseq, T, H, rank, D - rank, *sizes, scale, dt)
    if workspace is not None:
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be on cuda:{dev}")
        _run_on(dev, stream, lib().kda_latent_attn_ws, args + _workspace_args(workspace),
                "kda_latent_attn_ws")
    else:
        _run_on(dev, stream, lib().kda_latent_attn, args, "kda_latent_attn")
    return out, lse


def kda_verify_tokens(target: torch.Tensor, draft: Optional[torch.Tensor],
                      draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                      draft_lens: Optional[torch.Tensor] = None,
                      tokens: Optional[torch.Tensor] = None,
                      accepted: Optional[torch.Tensor] = None, stream=None):
    """Which drafted tokens stand, and the token after them.  target [N, L+1, V] f32;
    draft [N, L, V] f32, or None where each drafted token was certain; draft_tokens int32
    [N, L]; uniforms f32 [N, L+1] in [0, 1) (the last draws the token after the accepted
    ones); draft_lens int32 [N] or None (L each).  Returns (tokens int32 [N, L+1]: the
    accepted drafts, the drawn token, then -1; accepted int32 [N])."""
    if target.dim() != 3:
        raise ValueError("target must be [N, L + 1, V]")
    N, L1, V = target.shape
    L = L1 - 1
    dev = _device_of("target", target)
    xp = _take("draft_tokens", draft_tokens, dev, torch.int32, (N, L))
    if tokens is None:
        tokens = _new(stream, draft_tokens, (N, L1), torch.int32)
        tp = tokens.data_ptr()
    else:
        tp = _take("tokens", tokens, dev, torch.int32, (N, L1))
    if accepted is None:
        accepted = _new(stream, draft_tokens, (N,), torch.int32)
        ap = accepted.data_ptr()
    else:
        ap = _take("accepted", accepted, dev, torch.int32, (N,))
    _run_on(dev, stream, lib().kda_verify_tokens,
            (_take("target", target, dev, torch.float32, (N, L1, V)),
             _take("draft", draft, dev, torch.float32, (N, L, V)), xp,
             _take("uniforms", uniforms, dev, torch.float32, (N, L1)),
             _take("draft_lens", draft_lens, dev, torch.int32, (N,)), tp, ap, N, L, V),
            "kda_verify_tokens")
    return tokens, accepted
