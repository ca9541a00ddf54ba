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
and beam search's selection over state slots (gdn_beam_select,
gdn_gather_states).

No call here records a graph for automatic differentiation: results carry no
history, whatever requires_grad says of the inputs. To train through the norm
or the scan, call the *_backward functions in the backward method of a
torch.autograd.Function.
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
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL_POINTER", 2: "GDN_ERR_BAD_SHAPE",
           3: "GDN_ERR_UNSUPPORTED", 4: "GDN_ERR_MISALIGNED", 5: "GDN_ERR_ALIAS",
           6: "GDN_ERR_HIP"}
EXPORTS = ("gdn_prefill_chunked", "gdn_decode_step", "gdn_varlen_prefill", "gdn_decode_multi",
           "gdn_prefill_workspace_size", "gdn_status_string", "gdn_version",
           "gdn_prefill_chunked_noalloc", "gdn_scan_prefill", "gdn_scan_varlen_prefill",
           "gdn_scan_backward", "gdn_scan_varlen_backward", "gdn_scan_decode",
           "gdn_scan_workspace_size", "gdn_rms_norm", "gdn_rms_norm_backward",
           "gdn_rms_norm_workspace_size", "gdn_beam_select", "gdn_beam_workspace_size",
           "gdn_gather_states")
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
    for name in ("gdn_scan_prefill", "gdn_scan_varlen_prefill", "gdn_scan_backward",
                 "gdn_scan_varlen_backward", "gdn_scan_decode", "gdn_rms_norm",
                 "gdn_rms_norm_backward", "gdn_beam_select", "gdn_gather_states"):
        getattr(lib, name).restype = ci
    for name in ("gdn_scan_workspace_size", "gdn_rms_norm_workspace_size",
                 "gdn_beam_workspace_size"):
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


def gdn_version() -> int:
    return load_library().gdn_version()
