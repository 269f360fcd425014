"""Gated Delta Product (GDP) forward pass for NVIDIA GB300 (sm_103a).

Thin ctypes binding over ``libgdp.so`` (C ABI in ``include/gdp.h``). The
Python functions carry the C names and only marshal arguments: they allocate
outputs and workspace with PyTorch (device memory and streams are all PyTorch
is used for), pass raw device pointers and the current CUDA stream, and raise
on a non-OK status. Every step of the computation runs in the library's CUDA
kernels; there is no CPU path. ``load()`` raises if the library has not been
built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

__all__ = [
    "load", "GDPError", "gdp_prefill_prepare", "gdp_decode_prepare", "gdp_chunk_fwd",
    "gdp_chunk_fwd_workspace_size", "gdp_chunk_fwd_stage_offsets", "gdp_recurrent_update",
    "gdp_read_status", "gdp_version", "gdp_set_stage_events", "gdp_chunk_fwd_noalloc",
    "gdp_recurrent_update_slots", "gdp_debug_wait_fault", "gdp_prefill_conv_prepare",
    "gdp_decode_conv_prepare",
    "gdp_linear_chunk_fwd", "gdp_linear_chunk_fwd_paged", "gdp_linear_chunk_fwd_workspace_size",
    "gdp_linear_recurrent_update", "gdp_linear_recurrent_update_paged", "gdp_block_plan",
    "gdp_group_norm", "gdp_group_norm_workspace_size",
    "gdp_rotary_frequencies", "gdp_rotary", "gdp_cache_append", "gdp_attention_paged",
    "gdp_attention_paged_workspace_size",
    "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdp.so")

GDP_OK, GDP_ERR_INVALID_ARG, GDP_ERR_UNSUPPORTED, GDP_ERR_CUDA = 0, 1, 2, 3
GDP_ERR_DEVICE_TIMEOUT, GDP_ERR_WORKSPACE = 4, 5
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_lock = threading.Lock()
_lib = None


class GDPError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {text} (status {status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libgdp.so once; raises if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() first")
            lib = ctypes.CDLL(LIB_PATH)
            P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
            prep = [P, I64, I64, P, I64, I64, P, P] + [I] * 7 + [I] + [P] * 5 + [P]
            lib.gdp_prefill_prepare.argtypes = prep
            lib.gdp_decode_prepare.argtypes = prep
            lib.gdp_prefill_conv_prepare.argtypes = ([P, I64, I64, P, P, I, P, P, P, I, P, I64, I64,
                                                      P, P] + [I] * 8 + [P] * 6)
            lib.gdp_decode_conv_prepare.argtypes = ([P, I64, I64, P, P, I, P, P, I, P, I64, I64, P,
                                                     P] + [I] * 8 + [P] * 7)
            lib.gdp_chunk_fwd_workspace_size.argtypes = [I] * 9 + [I]
            lib.gdp_chunk_fwd_workspace_size.restype = SZ
            lib.gdp_chunk_fwd_stage_offsets.argtypes = [I] * 9 + [I, P]
            lib.gdp_chunk_fwd.argtypes = ([P] * 7 + [I] * 9 + [F, I, I] + [P, P, P, SZ, P])
            lib.gdp_recurrent_update.argtypes = [P] * 6 + [I] * 6 + [F, I, I, P, P]
            lib.gdp_recurrent_update_slots.argtypes = ([P] * 7 + [I] * 7 + [F, I, I, P, P, P])
            lib.gdp_chunk_fwd_noalloc.argtypes = [P] * 7 + [I] * 9 + [F, I, I] + [P, P, P]
            lib.gdp_chunk_fwd_noalloc.restype = I
            lin = [P] * 5 + [I]  # q, k, v, strides, g, g_per_token
            pages = [P, I, P, I, P, I]  # pool, n_pages, tables, max_blocks, contexts, block_size
            lib.gdp_linear_chunk_fwd_workspace_size.argtypes = [I] * 8
            lib.gdp_linear_chunk_fwd_workspace_size.restype = SZ
            lib.gdp_linear_chunk_fwd.argtypes = lin + [P, P] + [I] * 7 + [F, I, P, P, P, SZ, P]
            lib.gdp_linear_chunk_fwd_paged.argtypes = (lin + [P] + [I] * 6 + [F, I] + pages
                                                       + [P, P, SZ, P])
            lib.gdp_linear_recurrent_update.argtypes = lin + [P] + [I] * 6 + [F, I, P, P]
            lib.gdp_linear_recurrent_update_paged.argtypes = (lin + pages + [I] * 6
                                                              + [F, I, P, P, P])
            lib.gdp_block_plan.argtypes = [P, P, I, P, I, P, I, P, I, I] + [P] * 7
            lib.gdp_group_norm.argtypes = ([P, I64, I64, P, I64, I64, P, P, I64, I64, I, I, F, I,
                                            I, I, P, P])
            lib.gdp_group_norm_ws.argtypes = lib.gdp_group_norm.argtypes[:-1] + [P, SZ, P]
            lib.gdp_group_norm_workspace_size.argtypes = [I64, I64, I, I, I]
            lib.gdp_group_norm_workspace_size.restype = SZ
            D = ctypes.c_double
            lib.gdp_rotary_frequencies.argtypes = [I, D, I] + [D] * 4 + [P, P]
            lib.gdp_rotary.argtypes = [P] * 4 + [I] * 3 + [F] + [I] * 6 + [P] * 3
            lib.gdp_cache_append.argtypes = ([P] * 6 + [I] * 3 + [F] + [I] * 7 + [P] * 5 + [I, I]
                                             + [P] * 3)
            lib.gdp_attention_paged.argtypes = ([P] * 6 + [I, I, P, I, P, P, I, P] + [I] * 6
                                                + [F, I, P, P, P, SZ, P])
            lib.gdp_attention_paged_workspace_size.argtypes = [I] * 8
            lib.gdp_attention_paged_workspace_size.restype = SZ
            for f in ("gdp_linear_chunk_fwd", "gdp_linear_chunk_fwd_paged",
                      "gdp_linear_recurrent_update", "gdp_linear_recurrent_update_paged",
                      "gdp_block_plan", "gdp_group_norm", "gdp_group_norm_ws",
                      "gdp_rotary_frequencies", "gdp_rotary", "gdp_cache_append",
                      "gdp_attention_paged"):
                getattr(lib, f).restype = I
            lib.gdp_read_status.argtypes = [P, P]
            lib.gdp_debug_wait_fault.argtypes = [I, ctypes.c_double]
            lib.gdp_debug_wait_fault.restype = I
            lib.gdp_set_stage_events.argtypes = [P, I]
            lib.gdp_set_stage_events.restype = I
            lib.gdp_status_string.argtypes = [I]
            lib.gdp_status_string.restype = ctypes.c_char_p
            lib.gdp_version.argtypes = []
            for f in ("gdp_prefill_prepare", "gdp_decode_prepare", "gdp_chunk_fwd",
                      "gdp_prefill_conv_prepare", "gdp_decode_conv_prepare",
                      "gdp_recurrent_update", "gdp_recurrent_update_slots", "gdp_read_status",
                      "gdp_chunk_fwd_stage_offsets",
                      "gdp_version"):
                getattr(lib, f).restype = I
            _lib = lib
    return _lib


def _check(fn: str, status: int):
    if status != GDP_OK:
        raise GDPError(fn, status, load().gdp_status_string(status).decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libgdp works on CUDA tensors only")


def _a(t):
    """Address of an optional tensor."""
    return None if t is None else t.data_ptr()


# The handle of a device's current stream without a Stream object in between: a call of the
# small operators below takes about 10 us of host time, 2 of them that object's.
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(t):
    if _raw_stream_of is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream_of(t.device.index)


def _out_ok(t, shape, dtype):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() \
            or not t.is_cuda:
        raise ValueError(f"an output must be a contiguous CUDA tensor {list(shape)} of {dtype}")


def _status_ok(t):
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1 or not t.is_cuda):
        raise ValueError("status must be an int32 device tensor")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _one_device(*ts):
    """The kernels run on the current device, and read every tensor there."""
    current = _current_device()
    for t in ts:
        if t is not None and t.get_device() != current:
            raise ValueError("every tensor must be on the current CUDA device")


def _here():
    """The current device; None without one (sizes can be asked for there too)."""
    try:
        return _current_device()
    except (RuntimeError, AssertionError):
        return None


def gdp_version() -> int:
    return int(load().gdp_version())


# ----------------------------------------------------------------------------------
# prepare
# ----------------------------------------------------------------------------------

def _prepare(name, x, ba, A_log, dt_bias, M, H, G, P, N, decode, out=None):
    _need_cuda(x, ba, A_log, dt_bias)
    if x.dtype not in _DTYPE or ba.dtype != x.dtype:
        raise ValueError("x and ba must share a dtype in {bf16, fp16, fp32}")
    if x.dim() != 3 or ba.dim() != 3 or x.stride(-1) != 1 or ba.stride(-1) != 1:
        raise ValueError("x and ba must be [n, T, D] with a contiguous last dimension")
    n, T, D = x.shape
    if D != M * H * P + M * G * N + G * N or tuple(ba.shape) != (n, T, M * H + H):
        raise ValueError("x/ba last dimensions do not match M, H, G, P, N")
    A_log = A_log.to(torch.float32).contiguous()
    dt_bias = dt_bias.to(torch.float32).contiguous()
    L = T * M
    dev = x.device
    if out is None:
        q = torch.empty((n, L if decode else T, H, N), dtype=x.dtype, device=dev)
        k = torch.empty((n, L, H, N), dtype=x.dtype, device=dev)
        v = torch.empty((n, L, H, P), dtype=x.dtype, device=dev)
        beta = torch.empty((n, L, H), dtype=torch.float32, device=dev)
        g = torch.empty((n, L if decode else T, H), dtype=torch.float32, device=dev)
    else:
        q, k, v, beta, g = out
    fn = getattr(load(), name)
    st = fn(_p(x), x.stride(0), x.stride(1), _p(ba), ba.stride(0), ba.stride(1), _p(A_log),
            _p(dt_bias), n, T, M, H, G, P, N, _DTYPE[x.dtype], _p(q), _p(k), _p(v), _p(beta),
            _p(g), _stream(dev))
    _check(name, st)
    return q, k, v, beta, g


def gdp_prefill_prepare(x, ba, A_log, dt_bias, num_householder: int, num_heads: int,
                        num_groups: int, head_dim: int, state_dim: int, out=None):
    """Split/expand/gate a prefill step: returns (q [n,T,H,N], k [n,T*M,H,N],
    v [n,T*M,H,P], beta [n,T*M,H] fp32, g [n,T,H] fp32)."""
    return _prepare("gdp_prefill_prepare", x, ba, A_log, dt_bias, num_householder, num_heads,
                    num_groups, head_dim, state_dim, False, out)


def gdp_decode_prepare(x, ba, A_log, dt_bias, num_householder: int, num_heads: int,
                       num_groups: int, head_dim: int, state_dim: int, out=None):
    """Split/expand/gate a decode step (q on the last copy, g on the first):
    returns (q, k [n,S*M,H,N], v [n,S*M,H,P], beta, g [n,S*M,H] fp32)."""
    return _prepare("gdp_decode_prepare", x, ba, A_log, dt_bias, num_householder, num_heads,
                    num_groups, head_dim, state_dim, True, out)


# ----------------------------------------------------------------------------------
# chunked forward
# ----------------------------------------------------------------------------------

def gdp_chunk_fwd_workspace_size(B, T, N_seq, H, HV, K, V, M, chunk_size, dtype) -> int:
    return int(load().gdp_chunk_fwd_workspace_size(B, T, N_seq, H, HV, K, V, M, chunk_size,
                                                   _DTYPE[dtype]))


def gdp_chunk_fwd_stage_offsets(B, T, N_seq, H, HV, K, V, M, chunk_size, dtype):
    out = (ctypes.c_size_t * 8)()
    _check("gdp_chunk_fwd_stage_offsets",
           load().gdp_chunk_fwd_stage_offsets(B, T, N_seq, H, HV, K, V, M, chunk_size,
                                              _DTYPE[dtype], out))
    return list(out)


def gdp_chunk_fwd(q, k, v, beta, g=None, cu_seqlens=None, chunk_size: int = 64,
                  num_householder: int = 1, scale: float | None = None, initial_state=None,
                  use_qk_l2norm: bool = False, output_final_state: bool = True, workspace=None,
                  out=None):
    """Chunked GDP forward: returns (o [B,T,HV,V] fp32, final_state [N,HV,K,V] fp32 or None).

    q [B,T,H,K], k [B,T*M,H,K], v [B,T*M,HV,V] (bf16/fp16/fp32), beta [B,T*M,HV]
    fp32, g [B,T,HV] fp32 natural-log decay per token (None: ungated),
    cu_seqlens [N+1] int32 on the device (B must be 1), initial_state [N,HV,K,V]
    fp32. ``scale`` defaults to K**-0.5. ``workspace``: optional uint8 device
    tensor of at least gdp_chunk_fwd_workspace_size() bytes.
    """
    _need_cuda(q, k, v, beta, g, cu_seqlens, initial_state)
    M = int(num_householder)
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if tuple(k.shape) != (B, T * M, H, K) or tuple(v.shape[:2]) != (B, T * M):
        raise ValueError("k/v must be [B, T*M, ...]")
    if tuple(beta.shape) != (B, T * M, HV) or (g is not None and tuple(g.shape) != (B, T, HV)):
        raise ValueError("beta must be [B,T*M,HV] and g [B,T,HV]")
    for t in (q, k, v, beta, g, initial_state):
        if t is not None and not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    if beta.dtype != torch.float32 or (g is not None and g.dtype != torch.float32):
        raise ValueError("beta and g must be fp32")
    if q.dtype != k.dtype or q.dtype != v.dtype or q.dtype not in _DTYPE:
        raise ValueError("q, k, v must share a dtype in {bf16, fp16, fp32}")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    if initial_state is not None and (tuple(initial_state.shape) != (N, HV, K, V)
                                      or initial_state.dtype != torch.float32):
        raise ValueError("initial_state must be fp32 [N, HV, K, V]")
    if scale is None:
        scale = K ** -0.5
    dev = q.device
    need = gdp_chunk_fwd_workspace_size(B, T, N, H, HV, K, V, M, chunk_size, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if out is None:
        o = torch.empty((B, T, HV, V), dtype=torch.float32, device=dev)
        fs = (torch.empty((N, HV, K, V), dtype=torch.float32, device=dev)
              if output_final_state else None)
    else:
        o, fs = out
    st = load().gdp_chunk_fwd(_p(q), _p(k), _p(v), _p(beta), _p(g), _p(initial_state),
                              _p(cu_seqlens), N, B, T, H, HV, K, V, M, int(chunk_size),
                              float(scale), 1 if use_qk_l2norm else 0, _DTYPE[q.dtype], _p(o),
                              _p(fs), _p(workspace), workspace.numel(), _stream(dev))
    _check("gdp_chunk_fwd", st)
    return o, fs


GDP_STAGE_EVENTS = 5


def gdp_set_stage_events(events):
    """Profiling hook: record ``events`` (5 torch.cuda.Event, or None to switch
    off) at the stage boundaries of every later gdp_chunk_fwd call: entry, after
    the chunk tables, after the WY stage, after the state recurrence, after the
    output stage."""
    lib = load()
    if events is None:
        _check("gdp_set_stage_events", lib.gdp_set_stage_events(None, 0))
        return
    for e in events:
        e.record()  # forces the lazy creation of the CUDA event
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check("gdp_set_stage_events", lib.gdp_set_stage_events(arr, len(events)))


def gdp_chunk_fwd_noalloc(q, k, v, beta, g=None, cu_seqlens=None, chunk_size: int = 64,
                          num_householder: int = 1, scale: float | None = None,
                          initial_state=None, use_qk_l2norm: bool = False,
                          output_final_state: bool = True, out=None):
    """gdp_chunk_fwd without a caller workspace: the library's fixed 32 MiB device
    scratch array is used instead, for callers that cannot allocate device memory
    (fixed memory budgets, allocator callbacks, loops that must not reach
    cudaMalloc). Outputs are still allocated here unless ``out`` is given; pass
    ``out`` to allocate nothing. Larger problems raise GDPError (workspace).
    Calls sharing the array must not overlap on the GPU."""
    _need_cuda(q, k, v, beta, g, cu_seqlens, initial_state)
    M = int(num_householder)
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    if out is None:
        o = torch.empty((B, T, HV, V), dtype=torch.float32, device=q.device)
        fs = (torch.empty((N, HV, K, V), dtype=torch.float32, device=q.device)
              if output_final_state else None)
    else:
        o, fs = out
    st = load().gdp_chunk_fwd_noalloc(_p(q), _p(k), _p(v), _p(beta), _p(g), _p(initial_state),
                                      _p(cu_seqlens), N, B, T, H, HV, K, V, M, int(chunk_size),
                                      float(scale), 1 if use_qk_l2norm else 0, _DTYPE[q.dtype],
                                      _p(o), _p(fs), _stream(q.device))
    _check("gdp_chunk_fwd_noalloc", st)
    return o, fs


def gdp_read_status(workspace) -> int:
    """Synchronise and read the device status word of a chunk_fwd workspace."""
    return int(load().gdp_read_status(_p(workspace), _stream(workspace.device)))


# ----------------------------------------------------------------------------------
# decode recurrent update
# ----------------------------------------------------------------------------------

def gdp_recurrent_update(q, k, v, beta, g, state, scale: float | None = None,
                         use_qk_l2norm: bool = False, out=None):
    """Recurrent update over L = S*M steps per request; ``state`` [n,HV,K,V] fp32 is
    updated in place. Returns o [n,L,HV,V] fp32 (one row per step)."""
    _need_cuda(q, k, v, beta, g, state)
    n, L, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if tuple(k.shape) != (n, L, H, K) or tuple(v.shape[:2]) != (n, L):
        raise ValueError("q, k must be [n,L,H,K] and v [n,L,HV,V]")
    if tuple(beta.shape) != (n, L, HV) or tuple(g.shape) != (n, L, HV):
        raise ValueError("beta and g must be [n,L,HV]")
    if tuple(state.shape) != (n, HV, K, V) or state.dtype != torch.float32:
        raise ValueError("state must be fp32 [n,HV,K,V]")
    for t in (q, k, v, beta, g, state):
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    if scale is None:
        scale = K ** -0.5
    o = out if out is not None else torch.empty((n, L, HV, V), dtype=torch.float32,
                                                device=q.device)
    st = load().gdp_recurrent_update(_p(q), _p(k), _p(v), _p(beta), _p(g), _p(state), n, L, H,
                                     HV, K, V, float(scale), 1 if use_qk_l2norm else 0,
                                     _DTYPE[q.dtype], _p(o), _stream(q.device))
    _check("gdp_recurrent_update", st)
    return o


def gdp_recurrent_update_slots(q, k, v, beta, g, state_pool, state_slot, scale=None,
                               use_qk_l2norm: bool = False, status=None, out=None):
    """Recurrent update of a decode batch whose states live in a pool: request r
    updates ``state_pool[state_slot[r]]`` in place (``state_slot`` int32 [n] on the
    device; -1 marks a padding request, whose o rows are zero and which touches no
    state). ``status`` (optional int32 device tensor, one element) is set to 1 when
    a slot is out of range or repeated; those requests are skipped. Returns o."""
    _need_cuda(q, k, v, beta, g, state_pool, state_slot, status)
    n, L, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if tuple(k.shape) != (n, L, H, K) or tuple(v.shape[:2]) != (n, L):
        raise ValueError("q, k must be [n,L,H,K] and v [n,L,HV,V]")
    if tuple(beta.shape) != (n, L, HV) or tuple(g.shape) != (n, L, HV):
        raise ValueError("beta and g must be [n,L,HV]")
    if (state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (HV, K, V)
            or state_pool.dtype != torch.float32):
        raise ValueError("state_pool must be fp32 [n_slots,HV,K,V]")
    if tuple(state_slot.shape) != (n,) or state_slot.dtype != torch.int32:
        raise ValueError("state_slot must be int32 [n]")
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 device tensor")
    for t in (q, k, v, beta, g, state_pool, state_slot):
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    if scale is None:
        scale = K ** -0.5
    o = out if out is not None else torch.empty((n, L, HV, V), dtype=torch.float32,
                                                device=q.device)
    st = load().gdp_recurrent_update_slots(
        _p(q), _p(k), _p(v), _p(beta), _p(g), _p(state_pool), _p(state_slot),
        state_pool.shape[0], n, L, H, HV, K, V, float(scale), 1 if use_qk_l2norm else 0,
        _DTYPE[q.dtype], _p(o), _p(status), _stream(q.device))
    _check("gdp_recurrent_update_slots", st)
    return o


def gdp_debug_wait_fault(arm: bool | int, budget_seconds: float = 0.0):
    """Test hook (off by default): arm a one-shot missing tensor-core commit in the
    next 128-position WY launch (True), the next tensor-core launch of linear attention
    (2) or of gdp_attention_paged (3) so that one bounded device wait runs out, and/or set
    the wait budget (<= 0: the default 2 s)."""
    code = int(arm) if arm in (2, 3) else 1 if arm else 0
    _check("gdp_debug_wait_fault", load().gdp_debug_wait_fault(code, float(budget_seconds)))


def _conv_common(xp, conv_w, conv_b, ba, A_log, dt_bias, M, H, G, P, N):
    _need_cuda(xp, conv_w, conv_b, ba, A_log, dt_bias)
    if xp.dtype not in _DTYPE or ba.dtype != xp.dtype:
        raise ValueError("xp and ba must share a dtype in {bf16, fp16, fp32}")
    if xp.dim() != 3 or ba.dim() != 3 or xp.stride(-1) != 1 or ba.stride(-1) != 1:
        raise ValueError("xp and ba must be [n, T, D] with a contiguous last dimension")
    n, T, C = xp.shape
    if C != M * H * P + M * G * N + G * N or tuple(ba.shape) != (n, T, M * H + H):
        raise ValueError("xp/ba last dimensions do not match M, H, G, P, N")
    if conv_w.dim() != 2 or conv_w.shape[0] != C:
        raise ValueError("conv_w must be [C, W]")
    W = conv_w.shape[1]
    conv_w = conv_w.to(torch.float32).contiguous()
    conv_b = None if conv_b is None else conv_b.to(torch.float32).contiguous()
    return n, T, C, W, conv_w, conv_b, A_log.to(torch.float32).contiguous(), \
        dt_bias.to(torch.float32).contiguous()


def gdp_prefill_conv_prepare(xp, conv_w, conv_b, ba, A_log, dt_bias, num_householder: int,
                             num_heads: int, num_groups: int, head_dim: int, state_dim: int,
                             conv_state=None, cu_seqlens=None, return_conv_state=True,
                             out=None):
    """Short causal conv (+ SiLU) fused with the prefill prepare. Returns
    (q, k, v, beta, g, conv_state_out or None); conv_state_out [N, C, W-1]."""
    M, H, G, P, N = num_householder, num_heads, num_groups, head_dim, state_dim
    n, T, C, W, conv_w, conv_b, A_log, dt_bias = _conv_common(xp, conv_w, conv_b, ba, A_log,
                                                              dt_bias, M, H, G, P, N)
    NS = n if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    if conv_state is not None and (tuple(conv_state.shape) != (NS, C, W - 1)
                                   or conv_state.dtype != xp.dtype
                                   or not conv_state.is_contiguous()):
        raise ValueError("conv_state must be [N, C, W-1] in xp's dtype")
    dev = xp.device
    if out is None:
        out = (torch.empty((n, T, H, N), dtype=xp.dtype, device=dev),
               torch.empty((n, T * M, H, N), dtype=xp.dtype, device=dev),
               torch.empty((n, T * M, H, P), dtype=xp.dtype, device=dev),
               torch.empty((n, T * M, H), dtype=torch.float32, device=dev),
               torch.empty((n, T, H), dtype=torch.float32, device=dev))
    q, k, v, beta, g = out
    st_out = (torch.empty((NS, C, W - 1), dtype=xp.dtype, device=dev)
              if return_conv_state else None)
    st = load().gdp_prefill_conv_prepare(
        _p(xp), xp.stride(0), xp.stride(1), _p(conv_w), _p(conv_b), W, _p(conv_state),
        _p(st_out), _p(cu_seqlens), NS, _p(ba), ba.stride(0), ba.stride(1), _p(A_log),
        _p(dt_bias), n, T, M, H, G, P, N, _DTYPE[xp.dtype], _p(q), _p(k), _p(v), _p(beta),
        _p(g), _stream(dev))
    _check("gdp_prefill_conv_prepare", st)
    return q, k, v, beta, g, st_out


def gdp_decode_conv_prepare(xp, conv_w, conv_b, ba, A_log, dt_bias, num_householder: int,
                            num_heads: int, num_groups: int, head_dim: int, state_dim: int,
                            conv_state_pool, conv_slot, status=None, out=None):
    """Short causal conv (+ SiLU) fused with the decode prepare; conv states live in
    ``conv_state_pool`` [n_slots, C, W-1] (updated in place), ``conv_slot`` int32 [n]
    names each request's entry (-1: padding, zero q/k/v). Returns (q, k, v, beta, g)."""
    M, H, G, P, N = num_householder, num_heads, num_groups, head_dim, state_dim
    n, S, C, W, conv_w, conv_b, A_log, dt_bias = _conv_common(xp, conv_w, conv_b, ba, A_log,
                                                              dt_bias, M, H, G, P, N)
    _need_cuda(conv_state_pool, conv_slot, status)
    if (conv_state_pool.dim() != 3 or tuple(conv_state_pool.shape[1:]) != (C, W - 1)
            or conv_state_pool.dtype != xp.dtype or not conv_state_pool.is_contiguous()):
        raise ValueError("conv_state_pool must be [n_slots, C, W-1] in xp's dtype")
    if tuple(conv_slot.shape) != (n,) or conv_slot.dtype != torch.int32:
        raise ValueError("conv_slot must be int32 [n]")
    dev = xp.device
    L = S * M
    if out is None:
        out = (torch.empty((n, L, H, N), dtype=xp.dtype, device=dev),
               torch.empty((n, L, H, N), dtype=xp.dtype, device=dev),
               torch.empty((n, L, H, P), dtype=xp.dtype, device=dev),
               torch.empty((n, L, H), dtype=torch.float32, device=dev),
               torch.empty((n, L, H), dtype=torch.float32, device=dev))
    q, k, v, beta, g = out
    st = load().gdp_decode_conv_prepare(
        _p(xp), xp.stride(0), xp.stride(1), _p(conv_w), _p(conv_b), W, _p(conv_state_pool),
        _p(conv_slot), conv_state_pool.shape[0], _p(ba), ba.stride(0), ba.stride(1), _p(A_log),
        _p(dt_bias), n, S, M, H, G, P, N, _DTYPE[xp.dtype], _p(q), _p(k), _p(v), _p(beta),
        _p(g), _p(status), _stream(dev))
    _check("gdp_decode_conv_prepare", st)
    return q, k, v, beta, g


# ----------------------------------------------------------------------------------
# linear attention with a decay for each head
# ----------------------------------------------------------------------------------

_pack_strides = struct.Struct("9q").pack


def _linear_args(q, k, v, g):
    """Checks shared by the linear-attention calls: (B, T, H, HV, K, V, strides, g per token)."""
    if not (q.is_cuda and k.is_cuda and v.is_cuda and (g is None or g.is_cuda)):
        raise ValueError("libgdp works on CUDA tensors only")
    shape, vshape, dt = q.shape, v.shape, q.dtype
    if (len(shape) != 4 or len(vshape) != 4 or k.shape != shape or vshape[0] != shape[0]
            or vshape[1] != shape[1]):
        raise ValueError("q, k must be [B, T, H, K] and v [B, T, HV, V]")
    B, T, H, K = shape
    HV, V = vshape[2], vshape[3]
    if dt != k.dtype or dt != v.dtype or dt not in _DTYPE:
        raise ValueError("q, k, v must share a dtype in {bf16, fp16, fp32}")
    (a0, a1, a2, a3), (b0, b1, b2, b3), (c0, c1, c2, c3) = q.stride(), k.stride(), v.stride()
    if ((a3 != 1 or b3 != 1) and K > 1) or (c3 != 1 and V > 1):
        raise ValueError("the last dimension of q, k, v must be contiguous")
    per_token = 0
    if g is not None:
        if g.dtype != torch.float32 or not g.is_contiguous():
            raise ValueError("g must be fp32 and contiguous")
        if g.shape == (B, T, HV):
            per_token = 1
        elif g.shape != (HV,):
            raise ValueError("g must be [B, T, HV] or [HV]")
    return B, T, H, HV, K, V, _pack_strides(a0, a1, a2, b0, b1, b2, c0, c1, c2), per_token


def _state_ok(name, t, shape):
    if t is not None and (t.shape != shape or t.dtype != torch.float32 or not t.is_contiguous()
                          or not t.is_cuda):
        raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor {list(shape)}")


def _tables_ok(n, HV, K, V, state_pool, block_tables, context_lens):
    _need_cuda(state_pool, block_tables, context_lens)
    if (state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (HV, K, V)
            or state_pool.dtype != torch.float32 or not state_pool.is_contiguous()):
        raise ValueError("state_pool must be contiguous fp32 [n_pages, HV, K, V]")
    if (block_tables.dim() != 2 or block_tables.shape[0] != n or context_lens.shape != (n,)
            or block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32
            or not block_tables.is_contiguous() or not context_lens.is_contiguous()):
        raise ValueError("block_tables must be int32 [n, max_blocks] and context_lens int32 [n]")


def gdp_linear_chunk_fwd_workspace_size(B, T, N_seq, H, HV, K, V, dtype) -> int:
    return int(load().gdp_linear_chunk_fwd_workspace_size(B, T, N_seq, H, HV, K, V,
                                                          _DTYPE[dtype]))


def _linear_workspace(workspace, B, T, N, H, HV, K, V, q):
    if workspace is None:
        need = load().gdp_linear_chunk_fwd_workspace_size(B, T, N, H, HV, K, V, _DTYPE[q.dtype])
        return torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need_cuda(workspace)
    return workspace


def _linear_out(v, out):
    """The output: v's shape and dtype, contiguous."""
    if out is None:
        return torch.empty_like(v, memory_format=torch.contiguous_format)
    _out_ok(out, v.shape, v.dtype)
    return out


def _copy_status(status, workspace):
    """The workspace's status word into the caller's."""
    if status is not None:
        status.view(-1)[:1].copy_(workspace.view(torch.uint8)[:4].view(torch.int32))


def _packed(cu_seqlens, B):
    _need_cuda(cu_seqlens)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
            or cu_seqlens.numel() < 1 or B != 1:
        raise ValueError("cu_seqlens must be int32 [N + 1], with B == 1")
    return cu_seqlens.numel() - 1


def gdp_linear_chunk_fwd(q, k, v, g=None, cu_seqlens=None, scale: float | None = None,
                         initial_state=None, output_final_state: bool = True, workspace=None,
                         out=None, status=None):
    """Chunked linear attention with a decay for each head:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [B,T,H,K], v [B,T,HV,V] (bf16/fp16/fp32; any strides with a contiguous last
    dimension), g fp32 natural-log decay [B,T,HV] per token, [HV] per head or None,
    cu_seqlens [N+1] int32 on the device (B must be 1), initial_state [N,HV,K,V] fp32.
    ``scale`` defaults to K**-0.5. ``status`` (optional int32 device tensor) is set to 0, 1
    (bad offsets: o is left as it was) or 2 (a wait on the device ran out); without it the
    word is in the workspace (gdp_read_status). Returns (o [B,T,HV,V] in q's dtype,
    final_state [N,HV,K,V] fp32 or None)."""
    B, T, H, HV, K, V, strides, per_token = _linear_args(q, k, v, g)
    N = B if cu_seqlens is None else _packed(cu_seqlens, B)
    _state_ok("initial_state", initial_state, (N, HV, K, V))
    _status_ok(status)
    ws = _linear_workspace(workspace, B, T, N, H, HV, K, V, q)
    if out is None:
        o = _linear_out(v, None)
        fs = (torch.empty((N, HV, K, V), dtype=torch.float32, device=q.device)
              if output_final_state else None)
    else:
        o, fs = out
        _state_ok("final_state", fs, (N, HV, K, V))
        _linear_out(v, o)
    st = load().gdp_linear_chunk_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, _a(g), per_token, _a(initial_state),
        _a(cu_seqlens), N, B, T, H, HV, K, V, K ** -0.5 if scale is None else scale,
        _DTYPE[q.dtype], o.data_ptr(), _a(fs), ws.data_ptr(), ws.numel(), _raw_stream(q))
    if st:
        _check("gdp_linear_chunk_fwd", st)
    _copy_status(status, ws)
    return o, fs


def gdp_linear_chunk_fwd_paged(q, k, v, g, cu_seqlens, state_pool, block_tables, context_lens,
                               block_size: int, scale: float | None = None, workspace=None,
                               out=None, status=None):
    """Chunked linear attention over packed prompts whose states live in pages:
    request r starts from the page of its token context_lens[r] - 1 (zeros for a new
    request) and writes ``state_pool`` [n_pages,HV,K,V] fp32 at every block of
    block_size tokens (a multiple of 64) that it ends and at its last token;
    block_tables [n, max_blocks] names the pages. q, k [1,T,H,K], v [1,T,HV,V].
    ``status`` as in gdp_linear_chunk_fwd, 1 also for a skipped request (a negative
    context or a page outside the pool). Returns o."""
    B, T, H, HV, K, V, strides, per_token = _linear_args(q, k, v, g)
    N = _packed(cu_seqlens, B)
    _tables_ok(N, HV, K, V, state_pool, block_tables, context_lens)
    _status_ok(status)
    ws = _linear_workspace(workspace, B, T, N, H, HV, K, V, q)
    o = _linear_out(v, out)
    st = load().gdp_linear_chunk_fwd_paged(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, _a(g), per_token,
        cu_seqlens.data_ptr(), N, T, H, HV, K, V, K ** -0.5 if scale is None else scale,
        _DTYPE[q.dtype], state_pool.data_ptr(), state_pool.shape[0], block_tables.data_ptr(),
        block_tables.shape[1], context_lens.data_ptr(), block_size, o.data_ptr(),
        ws.data_ptr(), ws.numel(), _raw_stream(q))
    if st:
        _check("gdp_linear_chunk_fwd_paged", st)
    _copy_status(status, ws)
    return o


def gdp_linear_recurrent_update(q, k, v, g, state, scale: float | None = None, out=None):
    """One decode step of linear attention with a decay for each head: S (1..16) tokens
    for each of n requests; ``state`` [n,HV,K,V] fp32 is updated in place. q, k
    [n,S,H,K], v [n,S,HV,V], g [n,S,HV], [HV] or None. Returns o [n,S,HV,V] in q's
    dtype."""
    n, S, H, HV, K, V, strides, per_token = _linear_args(q, k, v, g)
    _state_ok("state", state, (n, HV, K, V))
    o = _linear_out(v, out)
    st = load().gdp_linear_recurrent_update(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, _a(g), per_token, state.data_ptr(), n,
        S, H, HV, K, V, K ** -0.5 if scale is None else scale, _DTYPE[q.dtype], o.data_ptr(),
        _raw_stream(q))
    if st:
        _check("gdp_linear_recurrent_update", st)
    return o


def gdp_linear_recurrent_update_paged(q, k, v, g, state_pool, block_tables, context_lens,
                                      block_size: int, scale: float | None = None, status=None,
                                      out=None):
    """gdp_linear_recurrent_update with the states in pages, addressed as in
    gdp_linear_chunk_fwd_paged (any block_size). A request whose last token has no
    page (-1) is padding: zero o rows, no state touched. ``status`` (optional int32
    device tensor) is set to 1 when a request's pages lie outside the pool or clash
    with another's; those requests are skipped like padding. Returns o."""
    n, S, H, HV, K, V, strides, per_token = _linear_args(q, k, v, g)
    _tables_ok(n, HV, K, V, state_pool, block_tables, context_lens)
    _status_ok(status)
    o = _linear_out(v, out)
    st = load().gdp_linear_recurrent_update_paged(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, _a(g), per_token,
        state_pool.data_ptr(), state_pool.shape[0], block_tables.data_ptr(),
        block_tables.shape[1], context_lens.data_ptr(), block_size, n, S, H, HV, K, V,
        K ** -0.5 if scale is None else scale, _DTYPE[q.dtype], o.data_ptr(), _a(status),
        _raw_stream(q))
    if st:
        _check("gdp_linear_recurrent_update_paged", st)
    return o


# ----------------------------------------------------------------------------------
# block plan, group norm
# ----------------------------------------------------------------------------------

def gdp_block_plan(context_lens, query_lens, block_tables, free_pages, free_used, block_size: int,
                   max_tokens: int, status=None, out=None):
    """Plan of a serving step from request lengths, on the device: writes the new
    entries of ``block_tables`` [n, max_blocks] in place from ``free_pages`` (its first
    free_used[0] entries are taken) and returns (cu_seqlens [n+1], token_req
    [max_tokens], token_pos [max_tokens], slot_map [max_tokens] int64, free_used_out
    [1]); see include/gdp.h for ``status`` and for requests that do not fit."""
    _need_cuda(context_lens, query_lens, block_tables, free_pages, free_used)
    for t in (context_lens, query_lens, block_tables, free_pages, free_used):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("lengths, tables and free pages must be contiguous int32")
    n = context_lens.numel()
    if (context_lens.shape != (n,) or query_lens.shape != (n,) or block_tables.dim() != 2
            or block_tables.shape[0] != n or free_used.numel() != 1):
        raise ValueError("lengths must be [n], block_tables [n, max_blocks], free_used [1]")
    _status_ok(status)
    dev = context_lens.device
    if out is None:
        ints = torch.empty(n + 2 + 2 * max_tokens, dtype=torch.int32, device=dev)
        cu, used, req, pos = ints.split_with_sizes((n + 1, 1, max_tokens, max_tokens))
        out = (cu, req, pos, torch.empty(max_tokens, dtype=torch.int64, device=dev), used)
    else:
        for t, m, dt in zip(out, (n + 1, max_tokens, max_tokens, max_tokens, 1),
                            (torch.int32,) * 3 + (torch.int64, torch.int32)):
            _out_ok(t, (m,), dt)
    cu, req, pos, slot, used = out
    st = load().gdp_block_plan(
        context_lens.data_ptr(), query_lens.data_ptr(), n, block_tables.data_ptr(),
        block_tables.shape[1], free_pages.data_ptr(), free_pages.numel(), free_used.data_ptr(),
        block_size, max_tokens, cu.data_ptr(), req.data_ptr(), pos.data_ptr(), slot.data_ptr(),
        used.data_ptr(), _a(status), _raw_stream(context_lens))
    if st:
        _check("gdp_block_plan", st)
    return out


_ACTIVATION = {"none": 0, "silu": 1}


@functools.lru_cache(maxsize=256)
def _norm_bytes(device, *args):
    return int(load().gdp_group_norm_workspace_size(*args))


def gdp_group_norm_workspace_size(N, L, C, num_groups, dtype) -> int:
    """Bytes of gdp_group_norm's workspace on the current device."""
    return _norm_bytes(_here(), N, L, C, num_groups, _DTYPE[dtype])


def gdp_group_norm(x, num_groups: int, weight=None, bias=None, gate=None, eps: float = 1e-5,
                   activation: str = "silu", out_dtype=None, out=None, workspace=None):
    """Group norm with an activation, channels last: x [N, L, C] (or [N, C]: one
    position per sample, such as a token's heads), statistics over the positions and
    the C / num_groups channels of a group, z = (x - mean) / sqrt(var + eps) * weight
    + bias; returns act(z), or z * act(gate) with a gate. weight, bias [C] fp32;
    out_dtype is x's dtype, or bf16/fp16 for an fp32 x; the gate has it too. Rows of
    x and gate may be strided (contiguous channels). ``workspace``: uint8 of
    gdp_group_norm_workspace_size bytes (allocated where it is needed and None)."""
    _need_cuda(x, weight, bias, gate)
    if x.dim() not in (2, 3) or x.stride(-1) != 1:
        raise ValueError("x must be [N, L, C] or [N, C] with contiguous channels")
    dt_out = x.dtype if out_dtype is None else out_dtype
    if x.dtype not in _DTYPE or dt_out not in _DTYPE:
        raise ValueError("x and out_dtype must be bf16, fp16 or fp32")
    if activation not in _ACTIVATION:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATION)}")
    shape = x.shape
    N, L, C = (shape[0], 1, shape[1]) if x.dim() == 2 else shape
    x_sn, x_sl = (x.stride(0), 0) if x.dim() == 2 else x.stride()[:2]
    g_sn = g_sl = 0
    if gate is not None:
        if gate.shape != shape or gate.dtype != dt_out or gate.stride(-1) != 1:
            raise ValueError("gate must have x's shape, the output's dtype, contiguous channels")
        g_sn, g_sl = (gate.stride(0), 0) if x.dim() == 2 else gate.stride()[:2]
    for t in (weight, bias):
        if t is not None and (t.dtype != torch.float32 or t.shape != (C,)
                              or not t.is_contiguous()):
            raise ValueError("weight and bias must be contiguous fp32 [C]")
    if out is None:
        out = torch.empty(shape, dtype=dt_out, device=x.device)
    else:
        _out_ok(out, shape, dt_out)
    args = (x.data_ptr(), x_sn, x_sl, _a(gate), g_sn, g_sl, _a(weight), _a(bias), N, L, C,
            num_groups, eps, _ACTIVATION[activation], _DTYPE[x.dtype], _DTYPE[dt_out],
            out.data_ptr())
    if L > 1 and workspace is None:
        need = gdp_group_norm_workspace_size(N, L, C, num_groups, x.dtype)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if workspace is None:
        st = load().gdp_group_norm(*args, _raw_stream(x))
    else:
        _need_cuda(workspace)
        st = load().gdp_group_norm_ws(*args, workspace.data_ptr(), workspace.numel(),
                                      _raw_stream(x))
    if st:
        _check("gdp_group_norm", st)
    return out


# ----------------------------------------------------------------------------------
# attention layers: position rotation, a paged cache, attention over it
# ----------------------------------------------------------------------------------

_pack3 = struct.Struct("3q").pack
_SCALING = {"none": 0, "linear": 1, "ramp": 2, "wavelength": 3}


def gdp_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                           factor: float = 1.0, original_length: float = 0.0,
                           low: float = 1.0, high: float = 32.0, device="cuda"):
    """Angles per position of a rotation's rotary_dim / 2 pairs, base^(-2 i / rotary_dim),
    or scaled for long contexts: "linear" (all divided by factor), "ramp" (pairs that turn
    at most ``low`` times within original_length positions divided, those that turn
    ``high`` times or more kept, between them a ramp over the pairs; amplitude
    0.1 ln(factor) + 1), "wavelength" (the same by the pairs' own turns, amplitude 1). Host
    arithmetic in fp64. Returns (frequencies [rotary_dim / 2] fp64 on ``device``, amplitude)."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
    f = (ctypes.c_double * max(rotary_dim // 2, 1))()
    amplitude = ctypes.c_double()
    _check("gdp_rotary_frequencies",
           load().gdp_rotary_frequencies(rotary_dim, base, _SCALING[scaling], factor,
                                         original_length, low, high, f,
                                         ctypes.byref(amplitude)))
    return (torch.tensor(f[:rotary_dim // 2], dtype=torch.float64, device=device),
            amplitude.value)


# The library's sizes are 32-bit: a larger one would arrive as its low half. (`or` of the sizes: a tenth of a
# microsecond, of the 10 to 20 that a small call takes.)
def _too_large(*shapes):
    return ValueError(f"sizes of more than 31 bits: {[list(s) for s in shapes]}")


def _heads(name, t, dtype):
    """[T, H, D] or [B, T, H, D] as (shape, B, T, H, D, three strides)."""
    shape, stride = t.shape, t.stride()
    if not t.is_cuda:
        raise ValueError("libgdp works on CUDA tensors only")
    if t.dtype != dtype or len(shape) not in (3, 4) or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be [T, H, D] or [B, T, H, D] in one dtype of "
                         "{bf16, fp16, fp32} with a contiguous last dimension")
    if len(shape) == 3:
        T, H, D = shape
        if (T | H | D) >> 31:
            raise _too_large(shape)
        return shape, 1, T, H, D, (0, stride[0], stride[1])
    B, T, H, D = shape
    if (B | T | H | D) >> 31:
        raise _too_large(shape)
    return shape, B, T, H, D, stride[:3]


def _rotation(lead, positions, frequencies, D, offset):
    """Checks of a rotation's arguments: (positions, frequencies, rotary_dim)."""
    if frequencies is None:
        return None, None, 0
    if frequencies.dtype != torch.float64 or frequencies.dim() != 1 \
            or not frequencies.is_contiguous() or not frequencies.is_cuda:
        raise ValueError("frequencies must be a contiguous fp64 CUDA tensor [rotary_dim / 2]")
    if positions is None or positions.dtype != torch.int32 or not positions.is_cuda \
            or positions.shape != lead or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 CUDA tensor {list(lead)}")
    R = 2 * frequencies.numel()
    if offset < 0 or offset + R > D:
        raise ValueError("the rotated part must lie inside the head")
    return positions.data_ptr(), frequencies.data_ptr(), R


def gdp_rotary(x, positions, frequencies, offset: int = 0, interleaved: bool = False,
               amplitude: float = 1.0, backward: bool = False, out=None):
    """Position rotation of heads: x [T, H, D] or [B, T, H, D] (rows may be strided),
    positions [T] or [B, T] int32, frequencies [R / 2] fp64 (gdp_rotary_frequencies). Pair i
    of the elements [offset, offset + R), (i, i + R / 2) or neighbours (2 i, 2 i + 1) where
    ``interleaved``, turns by position * frequency; ``backward`` turns back (the gradient's
    pass, or undoing). ``out``: contiguous, or x itself. All on the current device. Returns y
    in x's dtype."""
    if x.dtype not in _DTYPE or frequencies is None:
        raise ValueError("x must be bf16, fp16 or fp32, with frequencies")
    shape, B, T, H, D, xs = _heads("x", x, x.dtype)
    pos, freq, R = _rotation(shape[:-2], positions, frequencies, D, offset)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out is not x:
        _out_ok(out, shape, x.dtype)
    _one_device(x, positions, frequencies, out)
    ys = xs if out is x else (T * H * D, H * D, D)
    st = load().gdp_rotary(x.data_ptr(), _pack3(*xs), pos, freq, R, offset, interleaved, amplitude,
                           backward, B, T, H, D, _DTYPE[x.dtype], out.data_ptr(), _pack3(*ys),
                           _raw_stream(x))
    if st:
        _check("gdp_rotary", st)
    return out


def _cache_ok(k_cache, v_cache, dtype):
    """Caches [n_pages, block_size, HKV, D]: (n_pages, block_size, HKV, D, DV, strides of both)."""
    (ks, kt), (vs, vt) = (k_cache.shape, k_cache.stride()), (v_cache.shape, v_cache.stride())
    if not (k_cache.is_cuda and v_cache.is_cuda):
        raise ValueError("libgdp works on CUDA tensors only")
    if (len(ks) != 4 or len(vs) != 4 or k_cache.dtype != dtype or v_cache.dtype != dtype
            or (kt[3] != 1 and ks[3] > 1) or (vt[3] != 1 and vs[3] > 1)):
        raise ValueError("caches must be [n_pages, block_size, HKV, D] in q, k, v's dtype with "
                         "a contiguous last dimension")
    if ks[:3] != vs[:3]:
        raise ValueError("the caches must have the same pages, block size and heads")
    pages, block, H, D = ks
    DV = vs[3]
    if (pages | block | H | D | DV) >> 31:
        raise _too_large(ks, vs)
    return (pages, block, H, D, DV, _pack3(kt[0], kt[1], kt[2]), _pack3(vt[0], vt[1], vt[2]))


def gdp_cache_append(k, v, k_cache, v_cache, slot_map, positions=None, frequencies=None,
                     offset: int = 0, interleaved: bool = False, amplitude: float = 1.0, q=None,
                     q_out=None, status=None):
    """Writes new tokens' keys and values into a paged cache, the keys (and ``q``, in the same
    launch) rotated as by gdp_rotary on the way; without frequencies nothing is rotated.

    k [T, HKV, D], v [T, HKV, DV], q [T, H, D] or None (or with a batch dimension in front;
    rows may be strided), k_cache [n_pages, block_size, HKV, D] and v_cache [n_pages,
    block_size, HKV, DV] with any strides of the first three dimensions, slot_map [T] int64
    and positions [T] int32 as gdp_block_plan gives them (-1: not kept). ``status`` (optional
    int32 device tensor) is raised to 1 by a slot outside the cache, which is not kept either.
    Slots must differ, and k, v and q lie apart from them (tokens are written in no order);
    all tensors are on the current device. Returns the rotated q (None without one)."""
    dt = k.dtype
    if dt not in _DTYPE:
        raise ValueError("k, v and q must be bf16, fp16 or fp32")
    shape, B, T, HKV, D, ks = _heads("k", k, dt)
    vshape, _, _, _, DV, vs = _heads("v", v, dt)
    pages, block, cH, cD, cDV, kst, vst = _cache_ok(k_cache, v_cache, dt)
    if vshape[:-1] != shape[:-1] or cH != HKV or cD != D or cDV != DV:
        raise ValueError("k and v must have the same tokens and the caches' heads")
    lead = shape[:-2]
    if slot_map.dtype != torch.int64 or slot_map.shape != lead or not slot_map.is_contiguous() \
            or not slot_map.is_cuda:
        raise ValueError(f"slot_map must be a contiguous int64 CUDA tensor {list(lead)}")
    _status_ok(status)
    pos, freq, R = _rotation(lead, positions, frequencies, D, offset)
    H, qs = 0, (0, 0, 0)
    if q is not None:
        qshape, _, _, H, qD, qs = _heads("q", q, dt)
        if qshape[:-2] != lead or qD != D:
            raise ValueError("q must have k's tokens and head size")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _out_ok(q_out, qshape, dt)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _one_device(k, v, q, k_cache, v_cache, slot_map, q_out, status)
    if R:
        _one_device(positions, frequencies)
    st = load().gdp_cache_append(
        _a(q), k.data_ptr(), v.data_ptr(), _pack_strides(*qs, *ks, *vs), pos, freq, R, offset,
        interleaved, amplitude, B, T, H, HKV, D, DV, _DTYPE[dt], slot_map.data_ptr(),
        k_cache.data_ptr(), kst, v_cache.data_ptr(), vst, pages, block, _a(q_out), _a(status),
        _raw_stream(k))
    if st:
        _check("gdp_cache_append", st)
    return q_out


@functools.lru_cache(maxsize=256)
def _attention_bytes(device, *args):
    return int(load().gdp_attention_paged_workspace_size(*args))


def gdp_attention_paged_workspace_size(B, T, N_seq, H, HKV, D, DV, dtype) -> int:
    """Bytes of gdp_attention_paged's workspace on the current device."""
    return _attention_bytes(_here(), B, T, N_seq, H, HKV, D, DV, _DTYPE[dtype])


def gdp_attention_paged(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens=None,
                        tree_mask=None, scale: float | None = None, workspace=None, out=None,
                        status=None):
    """Attention of new tokens over a paged cache that holds them already (gdp_cache_append):
    single tokens, trees of drafted tokens, or pieces of prompts.

    q [B, T, H, D] (rows may be strided): T new tokens for each of B requests, or with
    cu_seqlens [n+1] int32 on the device the tokens of n requests packed along T (B must be
    1). k_cache [n_pages, block_size, HKV, D], v_cache [n_pages, block_size, HKV, DV],
    block_tables [n, max_blocks] int32 (-1: not there), context_lens [n] int32: tokens before
    the new ones. tree_mask [B, T] int64: bit j of a token set where it sees its request's new
    token j (at most 64 tokens a request); without it each sees the new ones up to itself.
    ``scale`` defaults to D**-0.5. ``status`` (optional int32 device tensor) is raised to 1 by
    bad pages, contexts or offsets and to 2 where a wait on the device ran out; it is never
    lowered, so calls may share one. All tensors are on the current device. Returns o [B, T, H, DV] in q's dtype;
    rows that see nothing are 0. Rows past cu_seqlens[n], and all of them where the offsets
    are refused, are not written: they hold what ``out`` held, or without it anything."""
    dt = q.dtype
    if dt not in _DTYPE or q.dim() != 4:
        raise ValueError("q must be [B, T, H, D] in bf16, fp16 or fp32")
    _, B, T, H, D, qs = _heads("q", q, dt)
    pages, block, HKV, cD, DV, kst, vst = _cache_ok(k_cache, v_cache, dt)
    if cD != D:
        raise ValueError("q and k_cache must have the same head size")
    n = B if cu_seqlens is None else _packed(cu_seqlens, B)
    if not (block_tables.is_cuda and context_lens.is_cuda):
        raise ValueError("libgdp works on CUDA tensors only")
    if (block_tables.dim() != 2 or block_tables.shape[0] != n or context_lens.shape != (n,)
            or block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32
            or not block_tables.is_contiguous() or not context_lens.is_contiguous()):
        raise ValueError("block_tables must be int32 [n, max_blocks] and context_lens int32 [n]")
    if block_tables.shape[1] >> 31:
        raise _too_large(block_tables.shape)
    if tree_mask is not None:
        if tree_mask.dtype != torch.int64 or tree_mask.shape != (B, T) \
                or not tree_mask.is_contiguous() or not tree_mask.is_cuda:
            raise ValueError("tree_mask must be a contiguous int64 CUDA tensor [B, T]")
        if cu_seqlens is None and T > 64:
            raise ValueError("a tree has at most 64 tokens")
    _status_ok(status)
    shape = (B, T, H, DV)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device)
    else:
        _out_ok(out, shape, dt)
    if workspace is None:
        need = gdp_attention_paged_workspace_size(B, T, n, H, HKV, D, DV, dt)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    else:
        _need_cuda(workspace)
    _one_device(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, tree_mask, out, workspace, status)
    st = load().gdp_attention_paged(
        q.data_ptr(), _pack3(*qs), k_cache.data_ptr(), kst, v_cache.data_ptr(), vst, pages, block,
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), _a(cu_seqlens), n, _a(tree_mask), B, T, H,
        HKV, D, DV, D ** -0.5 if scale is None else scale, _DTYPE[dt], out.data_ptr(), _a(status),
        workspace.data_ptr(), workspace.numel(), _raw_stream(q))
    if st:
        _check("gdp_attention_paged", st)
    return out
