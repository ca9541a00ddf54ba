"""Python binding of libgdn.so, the MI355X Gated DeltaNet token mixer.

Argument marshalling only: each function checks dtypes, devices, shapes and
contiguity of torch tensors, allocates the outputs it is not given, and
calls the C entry point of the same name with raw device pointers and the
current HIP stream. Every step of the computation runs in the library's HIP
kernels; there is no fallback path. If libgdn.so is missing or cannot be
loaded, the first call raises.

The recurrence, per sequence and value head h (q/k head h // (Hv // Hk)):
    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
    o_t = scale * S_t q_t
States are fp32 [.., Hv, Dv, Dk] (S in R^{Dv x Dk}, row-major).
`flags` (GDN_QK_L2NORM | GDN_GATE_LOGITS) moves the input preparation into
the kernels: raw q/k rows are L2-normalised, alpha/beta are given as logits.

Beside the mixer: the gated linear recurrence with its gradients (gdn_scan_*),
RMS norm with the residual's addition and an 8-bit output (gdn_rms_norm*),
beam search's selection over state slots (gdn_beam_select,
gdn_gather_states), and the stack's softmax attention: whole prompts and their
gradients (gdn_attn_*prefill, gdn_attn_*backward), new tokens against a paged
cache with shared prefixes (gdn_attn_decode), appending to it (gdn_kv_append)
and rotary positions (gdn_rotary).

No call here records a graph for automatic differentiation: results carry no
history, whatever requires_grad says of the inputs. To train through the norm,
the scan or attention, call the *_backward functions in the backward method of a
torch.autograd.Function (gdn_rotary with GDN_ROPE_INVERSE for the rotation).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
# input preparation inside the kernels (the `flags` argument)
GDN_QK_L2NORM, GDN_GATE_LOGITS = 1, 2
# of the rotary calls: neighbouring columns are pairs; turn back
GDN_ROPE_PAIRS, GDN_ROPE_INVERSE = 4, 8
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL_POINTER", 2: "GDN_ERR_BAD_SHAPE",
           3: "GDN_ERR_UNSUPPORTED", 4: "GDN_ERR_MISALIGNED", 5: "GDN_ERR_ALIAS",
           6: "GDN_ERR_HIP"}
EXPORTS = ("gdn_prefill_chunked", "gdn_decode_step", "gdn_varlen_prefill", "gdn_decode_multi",
           "gdn_prefill_workspace_size", "gdn_status_string", "gdn_version",
           "gdn_prefill_chunked_noalloc", "gdn_scan_prefill", "gdn_scan_varlen_prefill",
           "gdn_scan_backward", "gdn_scan_varlen_backward", "gdn_scan_decode",
           "gdn_scan_workspace_size", "gdn_rms_norm", "gdn_rms_norm_backward",
           "gdn_rms_norm_workspace_size", "gdn_beam_select", "gdn_beam_workspace_size",
           "gdn_gather_states", "gdn_attn_prefill", "gdn_attn_varlen_prefill",
           "gdn_attn_backward", "gdn_attn_varlen_backward", "gdn_attn_backward_workspace_size",
           "gdn_attn_decode", "gdn_attn_decode_workspace_size", "gdn_rotary", "gdn_kv_append")
SCAN_TILE = 128  # prefix states that gdn_scan_backward needs: every 64 or 128 tokens

_lib = None


class GDNError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {detail}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (after torch, so that both share torch's HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m gated_deltanet_token_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    u32 = ctypes.c_uint32
    sz = ctypes.c_size_t
    lib.gdn_prefill_chunked.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, i32,
                                        i32, i32, i32, ctypes.c_int, f32, u32, vp, sz, vp]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i64,
                                                i32, i32, i32, i32, ctypes.c_int, f32, u32, vp]
    lib.gdn_prefill_chunked_noalloc.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                    ctypes.c_int, f32, u32, vp]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_multi.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32,
                                     i32, i32, i32, ctypes.c_int, f32, u32, vp]
    lib.gdn_decode_multi.restype = ctypes.c_int
    lib.gdn_varlen_prefill.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp, i32,
                                       i32, i32, i32, i32, ctypes.c_int, f32, u32, vp, sz, vp]
    lib.gdn_varlen_prefill.restype = ctypes.c_int
    lib.gdn_prefill_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int, i32]
    lib.gdn_prefill_workspace_size.restype = sz
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = i32
    ci = ctypes.c_int
    lib.gdn_scan_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, i32, ci, u32, vp,
                                     sz, vp]
    lib.gdn_scan_varlen_prefill.argtypes = [vp, vp, vp, vp, i32, i64, vp, vp, vp, vp, i32, i32, ci,
                                            u32, vp, sz, vp]
    lib.gdn_scan_backward.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i64,
                                      i32, ci, u32, vp, sz, vp]
    lib.gdn_scan_varlen_backward.argtypes = [vp, vp, vp, vp, vp, i32, i64, vp, vp, i32, vp, vp, vp,
                                             vp, vp, i32, ci, u32, vp, sz, vp]
    lib.gdn_scan_decode.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, ci, u32, vp]
    lib.gdn_scan_workspace_size.argtypes = [i32, i64, i32, ci, i32]
    lib.gdn_rms_norm.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, ci, f32, vp]
    lib.gdn_rms_norm_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, ci, f32, vp, sz, vp]
    lib.gdn_rms_norm_workspace_size.argtypes = [i64, i32]
    lib.gdn_beam_select.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i64, i32, ci, vp,
                                    sz, vp]
    lib.gdn_beam_workspace_size.argtypes = [i32, i32, i64, ci]
    lib.gdn_gather_states.argtypes = [vp, i64, vp, vp, i64, i64, vp]
    lib.gdn_attn_prefill.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, ci, f32, vp]
    lib.gdn_attn_varlen_prefill.argtypes = [vp, vp, vp, vp, i32, i64, vp, vp, i32, i32, i32, ci,
                                            f32, vp]
    lib.gdn_attn_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                      ci, f32, vp, sz, vp]
    lib.gdn_attn_varlen_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, i32,
                                             i32, i32, ci, f32, vp, sz, vp]
    lib.gdn_attn_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32, ci, i32]
    lib.gdn_attn_decode.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp, i32, vp, vp,
                                    i32, i32, i32, i32, i32, ci, f32, vp, sz, vp]
    lib.gdn_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, ci]
    lib.gdn_rotary.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i64, i32, i32, i32, ci, u32,
                               vp]
    lib.gdn_kv_append.argtypes = [vp, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32,
                                  vp, i32, vp, i32, i64, i32, i32, i32, ci, u32, vp]
    for name in ("gdn_scan_prefill", "gdn_scan_varlen_prefill", "gdn_scan_backward",
                 "gdn_scan_varlen_backward", "gdn_scan_decode", "gdn_rms_norm",
                 "gdn_rms_norm_backward", "gdn_beam_select", "gdn_gather_states",
                 "gdn_attn_prefill", "gdn_attn_varlen_prefill", "gdn_attn_backward",
                 "gdn_attn_varlen_backward", "gdn_attn_decode", "gdn_rotary", "gdn_kv_append"):
        getattr(lib, name).restype = ci
    for name in ("gdn_scan_workspace_size", "gdn_rms_norm_workspace_size",
                 "gdn_beam_workspace_size", "gdn_attn_backward_workspace_size",
                 "gdn_attn_decode_workspace_size"):
        getattr(lib, name).restype = sz
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise GDNError(status, _lib.gdn_status_string(status).decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"data tensors must be bfloat16 or float32, got {t.dtype}")


_INT32 = 0x7FFFFFFF  # the library takes sizes in 32 bits; ctypes drops the bits above


def _out_of_range(**values):
    raise ValueError("out of range: " + ", ".join(f"{k} = {v}" for k, v in values.items()))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device, stream):
    return stream if stream is not None else torch.cuda.current_stream(device)


def _keep_for(stream, *tensors):
    """Memory of tensors that were made on another stream: freed by their owner,
    it is not handed out again before what `stream` has been given so far is done."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)


def _keeps(fn):
    """Keeps a call's tensors, results among them, for its `stream` argument."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        out = fn(*args, stream=stream, **kw)
        if stream is not None and stream != torch.cuda.current_stream(stream.device):
            _keep_for(stream, *args, *kw.values(), *(out if isinstance(out, tuple) else (out,)))
        return out
    return call


def gdn_prefill_workspace_size(num_seqs, tokens, Hk, Hv, Dk, Dv, dtype, packed) -> int:
    """Workspace bytes the prefill calls can use (0: they would not use one)."""
    code = _dtype_code(torch.empty(0, dtype=dtype)) if isinstance(dtype, torch.dtype) else dtype
    return int(load_library().gdn_prefill_workspace_size(num_seqs, tokens, Hk, Hv, Dk, Dv, code,
                                                         int(bool(packed))))


def _workspace(workspace, num_seqs, tokens, Hk, Hv, Dk, Dv, dtype_code, packed, dev, stream):
    """(pointer, bytes, keep-alive) of the workspace argument: None = no
    workspace; "auto" = allocate what the library asks for; a uint8 tensor."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be None, 'auto' or a tensor")
        n = _lib.gdn_prefill_workspace_size(num_seqs, tokens, Hk, Hv, Dk, Dv, dtype_code,
                                            int(packed))
        if n == 0:
            return None, 0, None
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    workspace.record_stream(stream)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def prefix_state_rows(num_seqs: int, tokens: int, interval: int, packed: bool) -> int:
    """Rows of the prefix_states buffer for blocks of 64 * interval tokens:
    num_seqs * floor(T / L) for a dense batch (tokens = T per sequence),
    floor(total / L) + N for a packed one (tokens = total)."""
    L = 64 * interval
    return tokens // L + num_seqs if packed else num_seqs * (tokens // L)


def _prefix(prefix_states, prefix_interval, rows, Hv, Dv, Dk, dev):
    if prefix_states is None:
        return None, 0
    if int(prefix_interval) < 1:
        raise ValueError("prefix_interval must be >= 1 with prefix_states")
    if int(prefix_interval) > _INT32:
        _out_of_range(prefix_interval=prefix_interval)
    _need(prefix_states, "prefix_states", torch.float32, (rows, Hv, Dv, Dk), dev)
    return prefix_states, int(prefix_interval)


@_keeps
def gdn_prefill_chunked(q, k, v, alpha, beta, initial_state=None, *, out=None,
                        final_state=None, scale: float = 1.0, want_final_state: bool = True,
                        prefix_states=None, prefix_interval: int = 0, flags: int = 0,
                        workspace="auto", stream=None):
    """Chunked prefill. q,k [B,T,Hk,D]; v [B,T,Hv,D]; alpha,beta [B,T,Hv] fp32;
    initial_state [B,Hv,D,D] fp32 or None. Returns (out, final_state).
    prefix_states: optional fp32 [B * floor(T / L), Hv, D, D] (L = 64 *
    prefix_interval) receiving the state after every whole block of L tokens.
    workspace: "auto" (allocate what the library asks for), None, or a
    device uint8 tensor."""
    lib = load_library()
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (B, T, Hv, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, T, Hv), dev)
    _need(beta, "beta", torch.float32, (B, T, Hv), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (B, Hv, Dv, Dk), dev)
    if out is None:
        out = torch.empty((B, T, Hv, Dv), dtype=q.dtype, device=dev)
    _need(out, "out", q.dtype, (B, T, Hv, Dv), dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, Hv, Dv, Dk), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (B, Hv, Dv, Dk), dev)
    pre, pint = _prefix(prefix_states, prefix_interval,
                        prefix_state_rows(B, T, max(int(prefix_interval), 1), False), Hv, Dv, Dk,
                        dev)
    st = _stream(dev, stream)
    wp, wb, _keep = _workspace(workspace, B, T, Hk, Hv, Dk, Dv, _dtype_code(q), False, dev, st)
    _check(lib.gdn_prefill_chunked(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(initial_state), _ptr(out),
        _ptr(final_state), _ptr(pre), pint, B, T, Hk, Hv, Dk, Dv, _dtype_code(q), float(scale),
        int(flags), wp, wb, st.cuda_stream))
    return out, final_state


@_keeps
def gdn_prefill_chunked_noalloc(q, k, v, alpha, beta, initial_state=None, *, out=None,
                                final_state=None, scale: float = 1.0,
                                want_final_state: bool = True, prefix_states=None,
                                prefix_interval: int = 0, flags: int = 0, stream=None):
    """gdn_prefill_chunked on the library's static device scratch (no
    workspace argument, nothing allocated by the library; outputs the caller
    does not pass are allocated here by torch, as for the other calls).
    Calls that overlap in time on one device race on that scratch."""
    lib = load_library()
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (B, T, Hv, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, T, Hv), dev)
    _need(beta, "beta", torch.float32, (B, T, Hv), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (B, Hv, Dv, Dk), dev)
    if out is None:
        out = torch.empty((B, T, Hv, Dv), dtype=q.dtype, device=dev)
    _need(out, "out", q.dtype, (B, T, Hv, Dv), dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, Hv, Dv, Dk), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (B, Hv, Dv, Dk), dev)
    pre, pint = _prefix(prefix_states, prefix_interval,
                        prefix_state_rows(B, T, max(int(prefix_interval), 1), False), Hv, Dv, Dk,
                        dev)
    _check(lib.gdn_prefill_chunked_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(initial_state), _ptr(out),
        _ptr(final_state), _ptr(pre), pint, B, T, Hk, Hv, Dk, Dv, _dtype_code(q), float(scale),
        int(flags), _stream(dev, stream).cuda_stream))
    return out, final_state


@_keeps
def gdn_varlen_prefill(q, k, v, alpha, beta, cu_seqlens, initial_state=None, *, out=None,
                       final_state=None, scale: float = 1.0, want_final_state: bool = True,
                       prefix_states=None, prefix_interval: int = 0, flags: int = 0,
                       workspace="auto", stream=None):
    """Packed prefill. q,k [total,Hk,D]; v [total,Hv,D]; alpha,beta [total,Hv];
    cu_seqlens int32 [N+1] on the device. Returns (out, final_state [N,Hv,D,D]).
    prefix_states: optional fp32 [floor(total / L) + N, Hv, D, D]; block i of
    sequence n lands in row floor(cu_seqlens[n] / L) + n + i."""
    lib = load_library()
    total, Hk, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[2]
    dev = q.device
    _need(cu_seqlens, "cu_seqlens", torch.int32, device=dev)
    N = cu_seqlens.shape[0] - 1
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (total, Hv, Dv), dev)
    _need(alpha, "alpha", torch.float32, (total, Hv), dev)
    _need(beta, "beta", torch.float32, (total, Hv), dev)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (N, Hv, Dv, Dk), dev)
    if out is None:
        out = torch.empty((total, Hv, Dv), dtype=q.dtype, device=dev)
    _need(out, "out", q.dtype, (total, Hv, Dv), dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((N, Hv, Dv, Dk), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (N, Hv, Dv, Dk), dev)
    pre, pint = _prefix(prefix_states, prefix_interval,
                        prefix_state_rows(N, total, max(int(prefix_interval), 1), True), Hv, Dv,
                        Dk, dev)
    st = _stream(dev, stream)
    wp, wb, _keep = _workspace(workspace, N, total, Hk, Hv, Dk, Dv, _dtype_code(q), True, dev, st)
    _check(lib.gdn_varlen_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(cu_seqlens), N, total,
        _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(pre), pint, Hk, Hv, Dk, Dv,
        _dtype_code(q), float(scale), int(flags), wp, wb, st.cuda_stream))
    return out, final_state


@_keeps
def gdn_decode_step(q, k, v, alpha, beta, state, *, out=None, scale: float = 1.0, flags: int = 0,
                    stream=None):
    """One token per sequence; `state` [B,Hv,D,D] fp32 is updated in place.
    q,k [B,Hk,D]; v [B,Hv,D]; alpha,beta [B,Hv]. Returns out [B,Hv,D]."""
    lib = load_library()
    B, Hk, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[2]
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (B, Hv, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, Hv), dev)
    _need(beta, "beta", torch.float32, (B, Hv), dev)
    _need(state, "state", torch.float32, (B, Hv, Dv, Dk), dev)
    if out is None:
        out = torch.empty((B, Hv, Dv), dtype=q.dtype, device=dev)
    _need(out, "out", q.dtype, (B, Hv, Dv), dev)
    _check(lib.gdn_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(out), B, Hk, Hv,
        Dk, Dv, _dtype_code(q), float(scale), int(flags), _stream(dev, stream).cuda_stream))
    return out


@_keeps
def gdn_decode_multi(q, k, v, alpha, beta, state_pool, src_slot, dst_slot, *, out=None,
                     step_states=None, want_step_states: bool = False, scale: float = 1.0,
                     flags: int = 0, stream=None):
    """K tokens per sequence against a pool of state slots.
    q,k [B,K,Hk,D]; v [B,K,Hv,D]; alpha,beta [B,K,Hv] fp32; state_pool
    [num_slots,Hv,D,D] fp32; src_slot, dst_slot int32 [B] on the device
    (negative src = zero state, negative dst = final state not written).
    Returns (out [B,K,Hv,D], step_states [B,K,Hv,D,D] fp32 or None)."""
    lib = load_library()
    B, K, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (B, K, Hv, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, K, Hv), dev)
    _need(beta, "beta", torch.float32, (B, K, Hv), dev)
    _need(state_pool, "state_pool", torch.float32, device=dev)
    if state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (Hv, Dv, Dk):
        raise ValueError(f"state_pool must have shape [num_slots, {Hv}, {Dv}, {Dk}], "
                         f"got {tuple(state_pool.shape)}")
    _need(src_slot, "src_slot", torch.int32, (B,), dev)
    _need(dst_slot, "dst_slot", torch.int32, (B,), dev)
    if out is None:
        out = torch.empty((B, K, Hv, Dv), dtype=q.dtype, device=dev)
    _need(out, "out", q.dtype, (B, K, Hv, Dv), dev)
    if step_states is None and want_step_states:
        step_states = torch.empty((B, K, Hv, Dv, Dk), dtype=torch.float32, device=dev)
    if step_states is not None:
        _need(step_states, "step_states", torch.float32, (B, K, Hv, Dv, Dk), dev)
    _check(lib.gdn_decode_multi(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_pool),
        state_pool.shape[0], _ptr(src_slot), _ptr(dst_slot), _ptr(out), _ptr(step_states), B, K,
        Hk, Hv, Dk, Dv, _dtype_code(q), float(scale), int(flags), _stream(dev, stream).cuda_stream))
    return out, step_states


def _on_stream(first):
    """Runs a call on the device of its argument `first` and on its `stream`
    argument: torch allocates and the library launches there, whatever the
    current device and stream are. The call's tensors are kept for that stream."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, stream=None, **kw):
            t = args[0] if args else kw.get(first)
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{first} must be a torch.Tensor")
            index = t.get_device()
            if index < 0:
                return fn(*args, **kw)  # refused there
            if stream is None:
                if torch._C._cuda_getDevice() == index:
                    return fn(*args, **kw)
                stream = torch.cuda.current_stream(index)
            elif stream.device_index != index:
                raise ValueError(f"stream is on device {stream.device_index}, {first} on {index}")
            with torch.cuda.stream(stream):
                out = fn(*args, **kw)
            if stream != torch.cuda.current_stream(index):
                _keep_for(stream, *args, *kw.values())
            return out
        return call
    return wrap


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _like(t, name, dtype, shape, index):
    """_need with the checks that nearly always pass first: these calls are made
    once per token and layer."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous()):
        _need(t, name, dtype, shape, torch.device("cuda", index) if index >= 0 else None)
        raise ValueError(f"{name} is not as required")


def _on_gpu(index):
    if index < 0:
        raise ValueError("tensors must be on a GPU")


def _start(t, name, dims):
    """Type code, device index and shape of a call's first tensor."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _dtype_code(t), t.get_device(), t.shape


def _scratch(workspace, size, index, like):
    """(pointer, bytes, keep-alive) of a workspace argument whose size the
    library names through size(): None, "auto" or a tensor. Allocated in the
    element type of `like`, a tensor of the call (the quickest way to allocate)."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be None, 'auto' or a tensor")
        n = size()
        if n == 0:
            return None, 0, None
        workspace = like.new_empty((n + 3) // like.element_size())
        return workspace.data_ptr(), n, workspace
    _need(workspace, "workspace", device=torch.device("cuda", index))
    workspace.record_stream(torch.cuda.current_stream(index))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def gdn_scan_workspace_size(num_seqs, tokens, D, dtype, packed) -> int:
    """Workspace bytes the scan calls can use (0: they would not use one)."""
    code = _dtype_code(torch.empty(0, dtype=dtype)) if isinstance(dtype, torch.dtype) else dtype
    if max(num_seqs, D) > _INT32:
        return 0
    return int(load_library().gdn_scan_workspace_size(num_seqs, tokens, D, code,
                                                      int(bool(packed))))


def _scan_sizes(x, cu, index):
    """(sequences, tokens of one or of the batch, channels)."""
    if cu is None:
        return x.shape
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1:
        raise ValueError("cu_seqlens must be a one-dimensional tensor")
    _like(cu, "cu_seqlens", torch.int32, cu.shape, index)
    return cu.shape[0] - 1, x.shape[0], x.shape[1]


def _scan_prefix(prefix, interval, n, tokens, packed, D, index):
    interval = int(interval)
    if not -_INT32 <= interval <= _INT32:
        _out_of_range(prefix_interval=interval)
    if prefix is not None:
        if interval < 1:
            raise ValueError("prefix_interval must be >= 1 with prefix_states")
        _like(prefix, "prefix_states", torch.float32,
              (prefix_state_rows(n, tokens, interval, packed), D), index)
    return interval


def _scan_forward(x, alpha, beta, cu, h0, out, final, want_final, prefix, interval, flags,
                  workspace):
    lib = _lib or load_library()
    packed = cu is not None
    code, index, shape = _start(x, "x", 2 if packed else 3)
    dt = x.dtype
    _like(alpha, "alpha", dt, shape, index)
    if beta is not None:
        _like(beta, "beta", dt, shape, index)
    n, tokens, D = _scan_sizes(x, cu, index)
    if n > _INT32 or D > _INT32 or flags >> 32:
        _out_of_range(sequences=n, D=D, flags=flags)
    if h0 is not None:
        _like(h0, "initial_state", torch.float32, (n, D), index)
    interval = _scan_prefix(prefix, interval, n, tokens, packed, D, index)
    _on_gpu(index)
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", dt, shape, index)
    if final is not None:
        _like(final, "final_state", torch.float32, (n, D), index)
    elif want_final:
        final = torch.empty_like(h0) if h0 is not None else x.new_empty((n, D), dtype=torch.float32)
    wp, wb, _keep = _scratch(
        workspace, lambda: lib.gdn_scan_workspace_size(n, tokens, D, code, int(packed)), index,
        x)
    if packed:
        rc = lib.gdn_scan_varlen_prefill(
            x.data_ptr(), alpha.data_ptr(), _ptr(beta), cu.data_ptr(), n, tokens, _ptr(h0),
            out.data_ptr(), _ptr(final), _ptr(prefix), interval, D, code, flags, wp, wb,
            _raw_stream(index))
    else:
        rc = lib.gdn_scan_prefill(
            x.data_ptr(), alpha.data_ptr(), _ptr(beta), _ptr(h0), out.data_ptr(), _ptr(final),
            _ptr(prefix), interval, n, tokens, D, code, flags, wp, wb, _raw_stream(index))
    if rc:
        _check(rc)
    return out, final


@_on_stream("x")
def gdn_scan_prefill(x, alpha, beta=None, initial_state=None, *, out=None, final_state=None,
                     want_final_state: bool = True, prefix_states=None, prefix_interval: int = 0,
                     flags: int = 0, workspace="auto"):
    """Gated linear recurrence h_t = alpha_t h_{t-1} + beta_t x_t per channel.
    x, alpha, beta [B,T,D] of one dtype (beta None: 1 - alpha); initial_state
    [B,D] fp32 or None. Returns (out [B,T,D], final_state [B,D] fp32).
    prefix_states: optional fp32 [prefix_state_rows(B, T, interval, False), D]
    receiving the state after every whole block of 64 * prefix_interval tokens
    (gdn_scan_backward takes them with an interval of 1 or 2). `stream` (a
    torch.cuda.Stream, here and in the calls below): where to run, the current
    one by default. It is for the caller to let it wait for the inputs; their
    memory may be freed at once. Outputs made by the call belong to it. Results
    have no autograd history: gdn_scan_backward gives the gradients."""
    return _scan_forward(x, alpha, beta, None, initial_state, out, final_state, want_final_state,
                         prefix_states, prefix_interval, flags, workspace)


@_on_stream("x")
def gdn_scan_varlen_prefill(x, alpha, beta, cu_seqlens, initial_state=None, *, out=None,
                            final_state=None, want_final_state: bool = True, prefix_states=None,
                            prefix_interval: int = 0, flags: int = 0, workspace="auto"):
    """gdn_scan_prefill over packed sequences: x, alpha, beta [total,D];
    cu_seqlens int32 [N+1] on the device; states [N,D]."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _scan_forward(x, alpha, beta, cu_seqlens, initial_state, out, final_state,
                         want_final_state, prefix_states, prefix_interval, flags, workspace)


def _scan_backward(dout, x, alpha, beta, cu, h0, prefix, interval, dfinal, dx, dalpha, dbeta,
                   dinitial, want_dinitial, flags, workspace):
    lib = _lib or load_library()
    packed = cu is not None
    code, index, shape = _start(dout, "dout", 2 if packed else 3)
    dt = dout.dtype
    _like(x, "x", dt, shape, index)
    _like(alpha, "alpha", dt, shape, index)
    if beta is not None:
        _like(beta, "beta", dt, shape, index)
    elif dbeta is not None:
        raise ValueError("dbeta must be None with tied gates (beta None)")
    n, tokens, D = _scan_sizes(x, cu, index)
    if n > _INT32 or D > _INT32 or flags >> 32:
        _out_of_range(sequences=n, D=D, flags=flags)
    for t, name in ((h0, "initial_state"), (dfinal, "dfinal"), (dinitial, "dinitial")):
        if t is not None:
            _like(t, name, torch.float32, (n, D), index)
    for t, name in ((dx, "dx"), (dalpha, "dalpha"), (dbeta, "dbeta")):
        if t is not None:
            _like(t, name, dt, shape, index)
    interval = _scan_prefix(prefix, interval, n, tokens, packed, D, index)
    if prefix is None and tokens > SCAN_TILE:
        raise ValueError(f"prefix_states are needed for more than {SCAN_TILE} tokens")
    _on_gpu(index)
    dx = torch.empty_like(x) if dx is None else dx
    dalpha = torch.empty_like(x) if dalpha is None else dalpha
    if beta is not None and dbeta is None:
        dbeta = torch.empty_like(x)
    if dinitial is None and want_dinitial:
        dinitial = x.new_empty((n, D), dtype=torch.float32)
    wp, wb, _keep = _scratch(
        workspace, lambda: lib.gdn_scan_workspace_size(n, tokens, D, code, int(packed)), index,
        x)
    tail = (_ptr(prefix), interval, _ptr(dfinal), dx.data_ptr(), dalpha.data_ptr(), _ptr(dbeta),
            _ptr(dinitial))
    if packed:
        rc = lib.gdn_scan_varlen_backward(
            dout.data_ptr(), x.data_ptr(), alpha.data_ptr(), _ptr(beta), cu.data_ptr(), n, tokens,
            _ptr(h0), *tail, D, code, flags, wp, wb, _raw_stream(index))
    else:
        rc = lib.gdn_scan_backward(
            dout.data_ptr(), x.data_ptr(), alpha.data_ptr(), _ptr(beta), _ptr(h0), *tail, n,
            tokens, D, code, flags, wp, wb, _raw_stream(index))
    if rc:
        _check(rc)
    return dx, dalpha, dbeta, dinitial


@_on_stream("dout")
def gdn_scan_backward(dout, x, alpha, beta=None, initial_state=None, *, prefix_states=None,
                      prefix_interval: int = 0, dfinal=None, dx=None, dalpha=None, dbeta=None,
                      dinitial=None, want_dinitial: bool = True, flags: int = 0,
                      workspace="auto"):
    """Gradients of gdn_scan_prefill: dout [B,T,D], dfinal [B,D] fp32 or None,
    and the forward call's inputs, with the prefix states it wrote
    (prefix_interval 1 or 2; None for T <= SCAN_TILE). Returns (dx, dalpha,
    dbeta or None, dinitial [B,D] fp32 or None); with GDN_GATE_LOGITS dalpha
    and dbeta are the logits' gradients."""
    return _scan_backward(dout, x, alpha, beta, None, initial_state, prefix_states,
                          prefix_interval, dfinal, dx, dalpha, dbeta, dinitial, want_dinitial,
                          flags, workspace)


@_on_stream("dout")
def gdn_scan_varlen_backward(dout, x, alpha, beta, cu_seqlens, initial_state=None, *,
                             prefix_states=None, prefix_interval: int = 0, dfinal=None, dx=None,
                             dalpha=None, dbeta=None, dinitial=None, want_dinitial: bool = True,
                             flags: int = 0, workspace="auto"):
    """Gradients of gdn_scan_varlen_prefill: tensors [total,D], states [N,D]."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _scan_backward(dout, x, alpha, beta, cu_seqlens, initial_state, prefix_states,
                          prefix_interval, dfinal, dx, dalpha, dbeta, dinitial, want_dinitial,
                          flags, workspace)


@_on_stream("x")
def gdn_scan_decode(x, alpha, beta, state_pool, src_slot, dst_slot, *, out=None, flags: int = 0):
    """K tokens of the gated linear recurrence per sequence against a pool of
    state slots. x, alpha, beta [B,K,D] (beta None: 1 - alpha); state_pool
    [num_slots,D] fp32; src_slot, dst_slot int32 [B] on the device (negative
    src = zero state, negative dst = not written). Returns out [B,K,D]."""
    lib = _lib or load_library()
    code, index, shape = _start(x, "x", 3)
    B, K, D = shape
    _like(alpha, "alpha", x.dtype, shape, index)
    if beta is not None:
        _like(beta, "beta", x.dtype, shape, index)
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 2:
        raise ValueError("state_pool must be a tensor of shape [num_slots, D]")
    num_slots = state_pool.shape[0]
    if max(B, K, D, num_slots) > _INT32 or flags >> 32:
        _out_of_range(B=B, K=K, D=D, num_slots=num_slots, flags=flags)
    _like(state_pool, "state_pool", torch.float32, (num_slots, D), index)
    _like(src_slot, "src_slot", torch.int32, (B,), index)
    _like(dst_slot, "dst_slot", torch.int32, (B,), index)
    _on_gpu(index)
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", x.dtype, shape, index)
    rc = lib.gdn_scan_decode(x.data_ptr(), alpha.data_ptr(), _ptr(beta), state_pool.data_ptr(),
                             num_slots, src_slot.data_ptr(), dst_slot.data_ptr(), out.data_ptr(),
                             B, K, D, code, flags, _raw_stream(index))
    if rc:
        _check(rc)
    return out


def _rows(t, name):
    """(type code, device index, rows, columns) of a tensor of rows."""
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension of at least 1, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    D = t.shape[-1]
    if D > _INT32:
        _out_of_range(D=D)
    return _dtype_code(t), t.get_device(), t.numel() // D, D


@_on_stream("x")
def gdn_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, group: int = 0,
                 want_out: bool = True, want_out8: bool = False, want_residual: bool = True,
                 out=None, out8=None, scales=None, residual_out=None):
    """RMS norm over the last dimension of x (any leading dimensions), with the
    residual's addition and an output in 8 bits. x, residual, weight [D] of one
    dtype. Returns (out, out8, scales, residual_out), None where not wanted:
    out8 is torch.float8_e4m3fn with fp32 scales, one per row (group 0, shape
    [..., 1]) or per 128 columns (group 128, [..., ceil(D / 128)]);
    residual_out is x + residual (pass residual itself to update it in place).
    Results have no autograd history: gdn_rms_norm_backward gives the gradients."""
    lib = _lib or load_library()
    code, index, rows, D = _rows(x, "x")
    dt, shape = x.dtype, x.shape
    _like(weight, "weight", dt, (D,), index)
    if group != 0 and group != 128:
        raise ValueError(f"group must be 0 (one scale per row) or 128, got {group}")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    _on_gpu(index)
    if residual is not None:
        _like(residual, "residual", dt, shape, index)
        if residual_out is not None:
            _like(residual_out, "residual_out", dt, shape, index)
        elif want_residual:
            residual_out = torch.empty_like(x)
    if out is not None:
        _like(out, "out", dt, shape, index)
    elif want_out:
        out = torch.empty_like(x)
    if want_out8 or out8 is not None or scales is not None:
        sshape = (*shape[:-1], 1 if group == 0 else -(-D // 128))
        if out8 is None:
            out8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        else:
            _like(out8, "out8", torch.float8_e4m3fn, shape, index)
        if scales is None:
            scales = x.new_empty(sshape, dtype=torch.float32)
        else:
            _like(scales, "scales", torch.float32, sshape, index)
    rc = lib.gdn_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(residual_out),
                          _ptr(out), _ptr(out8), _ptr(scales), group, rows, D, code, eps,
                          _raw_stream(index))
    if rc:
        _check(rc)
    return out, out8, scales, residual_out


@_on_stream("dout")
def gdn_rms_norm_backward(dout, r, weight, dresidual=None, *, eps: float = 1e-6,
                          want_dweight: bool = True, dx=None, dweight=None, workspace="auto"):
    """Gradients of gdn_rms_norm at the row sums r (residual_out, or x without
    a residual): dout, r [..., D]; dresidual, the gradient that arrives at
    residual_out, or None. Returns (dx, dweight fp32 [D] or None); dx is the
    gradient of x and of residual alike and may be dresidual itself."""
    lib = _lib or load_library()
    code, index, rows, D = _rows(dout, "dout")
    dt, shape = dout.dtype, dout.shape
    _like(r, "r", dt, shape, index)
    _like(weight, "weight", dt, (D,), index)
    if dresidual is not None:
        _like(dresidual, "dresidual", dt, shape, index)
    _on_gpu(index)
    if dx is None:
        dx = torch.empty_like(r)
    else:
        _like(dx, "dx", dt, shape, index)
    if dweight is not None:
        _like(dweight, "dweight", torch.float32, (D,), index)
    elif want_dweight:
        dweight = torch.empty_like(weight, dtype=torch.float32)
    wp, wb, _keep = None, 0, None
    if dweight is not None:
        wp, wb, _keep = _scratch(workspace, lambda: lib.gdn_rms_norm_workspace_size(rows, D),
                                 index, dweight)
    rc = lib.gdn_rms_norm_backward(dout.data_ptr(), r.data_ptr(), weight.data_ptr(),
                                   _ptr(dresidual), dx.data_ptr(), _ptr(dweight), rows, D, code,
                                   eps, wp, wb, _raw_stream(index))
    if rc:
        _check(rc)
    return dx, dweight


@_on_stream("logits")
def gdn_beam_select(logits, scores, *, finished=None, eos: int = -1, beam_slots=None,
                    new_scores=None, tokens=None, parents=None, new_finished=None,
                    src_slots=None, workspace="auto"):
    """Beam search's selection. logits [B,W,V] (bf16 or fp32); scores [B,W]
    fp32, the beams' summed log-probabilities; finished uint8 [B,W] or None;
    eos the end token (-1: none); beam_slots int32 [B,W] or None, the beams'
    state slots. Returns (new_scores, tokens, parents, new_finished, src_slots),
    all [B,W], best first: parents are beam indices within the batch item,
    src_slots the parents' slots (the src_slot of the next decode call, or
    gdn_gather_states' index). new_finished is None without eos, src_slots
    without beam_slots."""
    lib = _lib or load_library()
    code, index, (B, W, V) = _start(logits, "logits", 3)
    shape = (B, W)
    if max(B, W, abs(eos)) > _INT32:
        _out_of_range(B=B, W=W, eos=eos)
    _like(scores, "scores", torch.float32, shape, index)
    if finished is not None:
        _like(finished, "finished", torch.uint8, shape, index)
        if eos < 0:
            raise ValueError("finished needs eos")
    if beam_slots is not None:
        _like(beam_slots, "beam_slots", torch.int32, shape, index)
    _on_gpu(index)
    if new_scores is None:
        new_scores = torch.empty_like(scores)
    else:
        _like(new_scores, "new_scores", torch.float32, shape, index)
    if tokens is None:
        tokens = torch.empty_like(scores, dtype=torch.int32)
    else:
        _like(tokens, "tokens", torch.int32, shape, index)
    if parents is None:
        parents = torch.empty_like(tokens)
    else:
        _like(parents, "parents", torch.int32, shape, index)
    if new_finished is not None:
        _like(new_finished, "new_finished", torch.uint8, shape, index)
    elif eos >= 0:
        new_finished = torch.empty_like(scores, dtype=torch.uint8)
    if src_slots is not None:
        _like(src_slots, "src_slots", torch.int32, shape, index)
    elif beam_slots is not None:
        src_slots = torch.empty_like(beam_slots)
    wp, wb, _keep = _scratch(workspace, lambda: lib.gdn_beam_workspace_size(B, W, V, code), index,
                             scores)
    rc = lib.gdn_beam_select(logits.data_ptr(), scores.data_ptr(), _ptr(finished),
                             _ptr(beam_slots), new_scores.data_ptr(), tokens.data_ptr(),
                             parents.data_ptr(), _ptr(new_finished), _ptr(src_slots), B, W, V,
                             eos, code, wp, wb, _raw_stream(index))
    if rc:
        _check(rc)
    return new_scores, tokens, parents, new_finished, src_slots


@_on_stream("states")
def gdn_gather_states(states, index, *, out=None):
    """Rows of a state buffer in a new order: out[i] = states[index[i]], any
    dtype, rows of a multiple of 16 bytes. index int32 [R] on the device (negative:
    zeros; past the end: bytes of 0xff). out must not overlap states."""
    lib = _lib or load_library()
    dev = states.get_device()
    if states.dim() < 1 or not states.is_contiguous():
        raise ValueError("states must be contiguous, with a first dimension of rows")
    if not isinstance(index, torch.Tensor) or index.dim() != 1:
        raise ValueError("index must be a one-dimensional tensor")
    _like(index, "index", torch.int32, index.shape, dev)
    R = index.shape[0]
    shape = (R, *states.shape[1:])
    row_bytes = math.prod(shape[1:]) * states.element_size()
    _on_gpu(dev)
    if out is None:
        out = states.new_empty(shape)
    else:
        _like(out, "out", states.dtype, shape, dev)
    rc = lib.gdn_gather_states(states.data_ptr(), states.shape[0], index.data_ptr(),
                               out.data_ptr(), R, row_bytes, _raw_stream(dev))
    if rc:
        _check(rc)
    return out


def _prompt(q, k, v, cu, name="q", first=None):
    """Checks q, k, v of a prompt call. Returns (type code, device index, sequences, tokens of
    one or of the batch, Hq, Hk, D)."""
    packed = cu is not None
    first = q if first is None else first
    code, index, shape = _start(first, name, 3 if packed else 4)
    _like(q, "q", first.dtype, shape, index)
    if not isinstance(k, torch.Tensor) or k.dim() != len(shape):
        raise ValueError(f"k must be a tensor of {len(shape)} dimensions")
    Hq, D, Hk = shape[-2], shape[-1], k.shape[-2]
    kv = (*shape[:-2], Hk, D)
    _like(k, "k", q.dtype, kv, index)
    _like(v, "v", q.dtype, kv, index)
    if packed:
        if not isinstance(cu, torch.Tensor) or cu.dim() != 1:
            raise ValueError("cu_seqlens must be a one-dimensional tensor")
        _like(cu, "cu_seqlens", torch.int32, cu.shape, index)
        n, tokens = cu.shape[0] - 1, shape[0]
    else:
        n, tokens = shape[0], shape[1]
    if max(n, Hq, Hk, D) > _INT32:
        _out_of_range(sequences=n, Hq=Hq, Hk=Hk, D=D)
    return code, index, n, tokens, Hq, Hk, D


def _scale(scale, D):
    if scale is None:
        return D ** -0.5 if D > 0 else 1.0  # heads of no columns are refused by the library
    return float(scale)


def _attn_forward(q, k, v, cu, scale, out, lse, want_lse):
    lib = _lib or load_library()
    code, index, n, tokens, Hq, Hk, D = _prompt(q, k, v, cu)
    _on_gpu(index)
    if out is None:
        out = torch.empty_like(q)
    else:
        _like(out, "out", q.dtype, q.shape, index)
    if lse is not None:
        _like(lse, "lse", torch.float32, q.shape[:-1], index)
    elif want_lse:
        lse = q.new_empty(q.shape[:-1], dtype=torch.float32)
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr())
    tail = (Hq, Hk, D, code, _scale(scale, D), _raw_stream(index))
    if cu is not None:
        rc = lib.gdn_attn_varlen_prefill(*ptrs, cu.data_ptr(), n, tokens, out.data_ptr(),
                                         _ptr(lse), *tail)
    else:
        rc = lib.gdn_attn_prefill(*ptrs, out.data_ptr(), _ptr(lse), n, tokens, *tail)
    if rc:
        _check(rc)
    return out, lse


@_on_stream("q")
def gdn_attn_prefill(q, k, v, *, scale=None, out=None, lse=None, want_lse: bool = False):
    """Causal softmax attention over prompts, grouped heads. q [B,T,Hq,D]; k, v
    [B,T,Hk,D] (Hq a multiple of Hk, D 64, 128 or 256); scale None: D ** -0.5.
    Returns (out [B,T,Hq,D], lse [B,T,Hq] fp32 or None), lse being what
    gdn_attn_backward takes. Results have no autograd history."""
    return _attn_forward(q, k, v, None, scale, out, lse, want_lse)


@_on_stream("q")
def gdn_attn_varlen_prefill(q, k, v, cu_seqlens, *, scale=None, out=None, lse=None,
                            want_lse: bool = False):
    """gdn_attn_prefill over packed prompts: q [total,Hq,D]; k, v [total,Hk,D];
    cu_seqlens int32 [N+1] on the device; lse [total,Hq]."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _attn_forward(q, k, v, cu_seqlens, scale, out, lse, want_lse)


def gdn_attn_backward_workspace_size(num_seqs, tokens, Hq, Hk, D, dtype, packed) -> int:
    """Workspace bytes of the attention backward calls."""
    code = _dtype_code(torch.empty(0, dtype=dtype)) if isinstance(dtype, torch.dtype) else dtype
    if max(num_seqs, Hq, Hk, D) > _INT32:
        return 0
    return int(load_library().gdn_attn_backward_workspace_size(num_seqs, tokens, Hq, Hk, D, code,
                                                               int(bool(packed))))


def _attn_backward(dout, q, k, v, out, lse, cu, scale, dq, dk, dv, workspace):
    lib = _lib or load_library()
    code, index, n, tokens, Hq, Hk, D = _prompt(q, k, v, cu, "dout", dout)
    _like(out, "out", q.dtype, q.shape, index)
    _like(lse, "lse", torch.float32, q.shape[:-1], index)
    _on_gpu(index)
    grads = []
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        if t is None:
            t = torch.empty_like(like)
        else:
            _like(t, name, q.dtype, like.shape, index)
        grads.append(t)
    packed = int(cu is not None)
    wp, wb, _keep = _scratch(
        workspace, lambda: lib.gdn_attn_backward_workspace_size(n, tokens, Hq, Hk, D, code, packed),
        index, lse)
    ptrs = [t.data_ptr() for t in (dout, q, k, v, out, lse)]
    to = [t.data_ptr() for t in grads]
    tail = (Hq, Hk, D, code, _scale(scale, D), wp, wb, _raw_stream(index))
    if packed:
        rc = lib.gdn_attn_varlen_backward(*ptrs, cu.data_ptr(), n, tokens, *to, *tail)
    else:
        rc = lib.gdn_attn_backward(*ptrs, *to, n, tokens, *tail)
    if rc:
        _check(rc)
    return tuple(grads)


@_on_stream("dout")
def gdn_attn_backward(dout, q, k, v, out, lse, *, scale=None, dq=None, dk=None, dv=None,
                      workspace="auto"):
    """Gradients of gdn_attn_prefill: dout [B,T,Hq,D], the forward call's inputs,
    its out and lse, and the same scale. Returns (dq, dk, dv)."""
    return _attn_backward(dout, q, k, v, out, lse, None, scale, dq, dk, dv, workspace)


@_on_stream("dout")
def gdn_attn_varlen_backward(dout, q, k, v, out, lse, cu_seqlens, *, scale=None, dq=None,
                             dk=None, dv=None, workspace="auto"):
    """Gradients of gdn_attn_varlen_prefill: tensors [total,H,D]."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _attn_backward(dout, q, k, v, out, lse, cu_seqlens, scale, dq, dk, dv, workspace)


def _cache(k_cache, v_cache, dtype, Hk, D, index):
    """(pages, tokens per page) of a paged cache."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor of shape [num_pages, page_size, Hk, D]")
    pages, page = k_cache.shape[0], k_cache.shape[1]
    if max(pages, page) > _INT32:
        _out_of_range(num_pages=pages, page_size=page)
    shape = (pages, page, k_cache.shape[2] if Hk is None else Hk, D)
    _like(k_cache, "k_cache", dtype, shape, index)
    _like(v_cache, "v_cache", dtype, shape, index)
    return pages, page


def _table(t, name, rows, index):
    """Columns of a page table of `rows` rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor of two dimensions")
    _like(t, name, torch.int32, (rows, t.shape[1]), index)
    if t.shape[1] > _INT32:
        _out_of_range(max_pages=t.shape[1])
    return t.shape[1]


def gdn_attn_decode_workspace_size(B, K, Hq, Hk, D, page_size, max_pages, G, max_prefix_pages,
                                   dtype) -> int:
    """Workspace bytes of gdn_attn_decode (0: it needs none)."""
    code = _dtype_code(torch.empty(0, dtype=dtype)) if isinstance(dtype, torch.dtype) else dtype
    sizes = (B, K, Hq, Hk, D, page_size, max_pages, G, max_prefix_pages)
    if max(sizes) > _INT32:
        return 0
    return int(load_library().gdn_attn_decode_workspace_size(*sizes, code))


@_on_stream("q")
def gdn_attn_decode(q, k_cache, v_cache, page_table, lengths, *, prefix_table=None,
                    prefix_lengths=None, prefix_groups=None, scale=None, out=None, lse=None,
                    want_lse: bool = False, workspace="auto"):
    """Softmax attention of K new tokens per sequence against a paged cache.
    q [B,K,Hq,D]; caches [num_pages, page_size, Hk, D]; page_table int32
    [B, max_pages]; lengths int32 [B], the K new tokens among them (token t sees
    the first lengths - K + 1 + t). Shared prefixes: prefix_table int32
    [G, max_prefix_pages], prefix_lengths int32 [G] and prefix_groups int32 [G+1],
    sequences prefix_groups[g] .. [g+1] - 1 standing behind prefix g. All on the
    device. scale None: D ** -0.5. Returns (out, lse [B,K,Hq] fp32 or None)."""
    lib = _lib or load_library()
    code, index, (B, K, Hq, D) = _start(q, "q", 4)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor of shape [num_pages, page_size, Hk, D]")
    Hk = k_cache.shape[2]
    if max(B, K, Hq, Hk, D) > _INT32:
        _out_of_range(B=B, K=K, Hq=Hq, Hk=Hk, D=D)
    pages, page = _cache(k_cache, v_cache, q.dtype, Hk, D, index)
    cols = _table(page_table, "page_table", B, index)
    _like(lengths, "lengths", torch.int32, (B,), index)
    G = pcols = 0
    if prefix_table is not None or prefix_lengths is not None or prefix_groups is not None:
        if not isinstance(prefix_lengths, torch.Tensor) or prefix_lengths.dim() != 1:
            raise ValueError("prefix_lengths must be a one-dimensional tensor: prefixes need "
                             "prefix_table, prefix_lengths and prefix_groups")
        G = prefix_lengths.shape[0]
        _like(prefix_lengths, "prefix_lengths", torch.int32, (G,), index)
        _like(prefix_groups, "prefix_groups", torch.int32, (G + 1,), index)
        pcols = _table(prefix_table, "prefix_table", G, index)
    _on_gpu(index)
    if out is None:
        out = torch.empty_like(q)
    else:
        _like(out, "out", q.dtype, q.shape, index)
    if lse is not None:
        _like(lse, "lse", torch.float32, q.shape[:-1], index)
    elif want_lse:
        lse = q.new_empty(q.shape[:-1], dtype=torch.float32)
    wp, wb, _keep = _scratch(
        workspace, lambda: lib.gdn_attn_decode_workspace_size(B, K, Hq, Hk, D, page, cols, G,
                                                              pcols, code), index, q)
    rc = lib.gdn_attn_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pages, page, page_table.data_ptr(),
        cols, lengths.data_ptr(), _ptr(prefix_table), pcols, _ptr(prefix_lengths),
        _ptr(prefix_groups), G, out.data_ptr(), _ptr(lse), B, K, Hq, Hk, D, code,
        _scale(scale, D), wp, wb, _raw_stream(index))
    if rc:
        _check(rc)
    return out, lse


def _angles(inv_freq, positions, pair_axis, lead, index):
    """(R, axes) of a rotation; lead: the shape of the tokens."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a one-dimensional tensor")
    half = inv_freq.shape[0]
    if 2 * half > _INT32:
        _out_of_range(R=2 * half)
    _like(inv_freq, "inv_freq", torch.float32, (half,), index)
    axes = 1
    if positions is not None:
        if isinstance(positions, torch.Tensor) and positions.dim() == len(lead) + 1:
            axes = positions.shape[0]
            _like(positions, "positions", torch.int32, (axes, *lead), index)
        else:
            _like(positions, "positions", torch.int32, tuple(lead), index)
    if pair_axis is not None:
        if positions is None:
            raise ValueError("pair_axis needs positions")
        _like(pair_axis, "pair_axis", torch.int32, (half,), index)
    if axes > _INT32:
        _out_of_range(axes=axes)
    return 2 * half, axes


def _heads(t, name, dims):
    """(type code, device index, leading dimensions, heads, columns) of [.., H, D]."""
    if t.dim() < 3 if dims is None else t.dim() != dims:
        raise ValueError(f"{name} must have {dims or 'at least 3'} dimensions, got "
                         f"{tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    H, D = t.shape[-2], t.shape[-1]
    if max(H, D) > _INT32:
        _out_of_range(heads=H, D=D)
    return _dtype_code(t), t.get_device(), t.shape[:-2], H, D


@_on_stream("q")
def gdn_rotary(q, k, positions, inv_freq, *, pair_axis=None, flags: int = 0, q_out=None,
               k_out=None):
    """Rotary positions. q [..,Hq,D]; k [..,Hk,D] or None; positions int32 [..] or
    [axes,..]; inv_freq fp32 [R/2], the first R columns of a head turning;
    pair_axis int32 [R/2], the axis of every pair (None: axis 0). flags:
    GDN_ROPE_PAIRS (neighbouring columns are pairs), GDN_ROPE_INVERSE (turn back: the
    gradient). Returns (q_out, k_out or None); pass q and k themselves to turn in
    place."""
    lib = _lib or load_library()
    code, index, lead, Hq, D = _heads(q, "q", None)
    Hk = 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
            raise ValueError(f"k must be a tensor of {q.dim()} dimensions")
        Hk = k.shape[-2]
        _like(k, "k", q.dtype, (*lead, Hk, D), index)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    if positions is None:
        raise TypeError("positions must be a torch.Tensor")
    R, axes = _angles(inv_freq, positions, pair_axis, lead, index)
    if max(Hq, Hk) > _INT32 or flags >> 32:
        _out_of_range(Hq=Hq, Hk=Hk, flags=flags)
    _on_gpu(index)
    if q_out is None:
        q_out = torch.empty_like(q)
    else:
        _like(q_out, "q_out", q.dtype, q.shape, index)
    if k is not None:
        if k_out is None:
            k_out = torch.empty_like(k)
        else:
            _like(k_out, "k_out", q.dtype, k.shape, index)
    rc = lib.gdn_rotary(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out),
                        positions.data_ptr(), axes, inv_freq.data_ptr(), _ptr(pair_axis), R,
                        math.prod(lead), Hq, Hk, D, code, flags, _raw_stream(index))
    if rc:
        _check(rc)
    return q_out, k_out


@_on_stream("k")
def gdn_kv_append(k, v, k_cache, v_cache, page_table, lengths, *, cu_seqlens=None, q=None,
                  inv_freq=None, positions=None, pair_axis=None, flags: int = 0, q_out=None,
                  k_out=None, want_k_out: bool = False):
    """New keys and values into a paged cache, rotated on the way. k, v [B,T,Hk,D], or
    packed [total,Hk,D] with cu_seqlens int32 [N+1]; caches [num_pages, page_size, Hk,
    D]; page_table int32 [N, max_pages]; lengths int32 [N], the tokens cached before
    this call: token i of sequence n gets place lengths[n] + i. q [..,Hq,D]: rotated
    beside them. inv_freq fp32 [R/2] or None (no rotation); positions, pair_axis, flags
    as for gdn_rotary (positions None: the places). All on the device. Returns (q_out
    or None, k_out or None); k_out, the rotated keys for the prompts' own attention,
    with want_k_out."""
    lib = _lib or load_library()
    packed = cu_seqlens is not None
    code, index, lead, Hk, D = _heads(k, "k", 3 if packed else 4)
    dt = k.dtype
    _like(v, "v", dt, k.shape, index)
    if packed:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a one-dimensional tensor")
        _like(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, index)
        N, tokens = cu_seqlens.shape[0] - 1, lead[0]
    else:
        N, tokens = lead
    if N > _INT32 or flags >> 32:
        _out_of_range(sequences=N, flags=flags)
    pages, page = _cache(k_cache, v_cache, dt, Hk, D, index)
    cols = _table(page_table, "page_table", N, index)
    _like(lengths, "lengths", torch.int32, (N,), index)
    Hq = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != k.dim():
            raise ValueError(f"q must be a tensor of {k.dim()} dimensions")
        Hq = q.shape[-2]
        if Hq > _INT32:
            _out_of_range(Hq=Hq)
        _like(q, "q", dt, (*lead, Hq, D), index)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    R, axes = 0, 1
    if inv_freq is not None:
        R, axes = _angles(inv_freq, positions, pair_axis, lead, index)
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    _on_gpu(index)
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            _like(q_out, "q_out", dt, q.shape, index)
    if k_out is not None:
        _like(k_out, "k_out", dt, k.shape, index)
    elif want_k_out:
        k_out = torch.empty_like(k)
    rc = lib.gdn_kv_append(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pages, page,
        page_table.data_ptr(), cols, lengths.data_ptr(), _ptr(cu_seqlens), _ptr(q), _ptr(q_out),
        _ptr(k_out), _ptr(inv_freq), R, _ptr(positions), axes, _ptr(pair_axis), N, tokens, Hq, Hk,
        D, code, flags, _raw_stream(index))
    if rc:
        _check(rc)
    return q_out, k_out


def gdn_version() -> int:
    return load_library().gdn_version()
