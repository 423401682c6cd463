"""Torch-facing wrappers of the gated delta rule (per-token test-time training of the linear inner model
with a forget gate) and of gradient clipping: marshalling only, as in ``layer``.

Tensor layout: Q, K [B][qk_heads][N][d_k] and V, Z [B][heads][N][d_v] with a contiguous last dimension and any
other strides the library accepts, so tensors laid out by token ([B][N][heads][d]) are passed as
``x.transpose(1, 2)`` without a copy.  G (log gates) and Beta are [B][heads][N] fp32, any strides.

Unlike the full-batch heads' calls, these allocate their workspace for the call (torch's allocator orders its
reuse on the call's stream), so calls on several streams and captured graphs share nothing.
"""
import ctypes

import torch

from . import capi
from .layer import _DTYPES, _check


class _On:
    """The tensors' device, with `stream` (None: the device's current stream) current on it."""

    def __init__(self, ref, stream):
        self.device, self.stream = ref.device, stream

    def __enter__(self):
        self.guards = []
        if torch.cuda.current_device() != self.device.index:
            self.guards.append(torch.cuda.device(self.device))
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError("the stream belongs to another device than the tensors")
            self.guards.append(torch.cuda.stream(self.stream))
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _view(t):
    """The ttt_view of a [B][heads][N] or [B][heads][N][width] tensor."""
    s = t.stride()
    return capi.TttView(t.data_ptr(), s[0], s[1], s[2])


def _tokens(name, t, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}")
    if len(shape) == 4 and shape[3] != 1 and t.stride(3) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _view(t)


def _delta_shape(Q, K, V):
    if Q.dim() != 4 or V.dim() != 4:
        raise ValueError("Q, K and V must be [B][heads][N][d]")
    if not Q.is_cuda:
        raise ValueError("Q, K and V must be CUDA tensors")
    if Q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {Q.dtype}")
    B, hk, N, dk = Q.shape
    h, dv = V.shape[1], V.shape[3]
    if hk < 1 or h % hk:
        raise ValueError(f"{h} value heads are not a multiple of {hk} key heads")
    return capi.make_delta_shape(B, hk, h, N, dk, dv, _DTYPES[Q.dtype]), B, hk, h, N, dk, dv


def _inputs(Q, K, V, G, Beta, B, hk, h, N, dk, dv):
    dt, dev = Q.dtype, Q.device
    return (_tokens("Q", Q, (B, hk, N, dk), dt, dev), _tokens("K", K, (B, hk, N, dk), dt, dev),
            _tokens("V", V, (B, h, N, dv), dt, dev), _tokens("G", G, (B, h, N), torch.float32, dev),
            _tokens("Beta", Beta, (B, h, N), torch.float32, dev))


def _state(name, W, shape, device):
    if W is None:
        return None
    if W.shape != shape or W.dtype != torch.float32 or W.device != device or not W.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 {list(shape)} tensor on {device}")
    return W.data_ptr()


def _start(W0, B, h, dv, dk, device):
    """(pointer, shared) of the starting weights."""
    if W0 is None:
        return None, 0
    shared = W0.dim() == 3
    return _state("W0", W0, (h, dv, dk) if shared else (B, h, dv, dk), device), int(shared)


def _ints(name, t, n, device):
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != torch.int32 or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} on {device}")
    return t.data_ptr()


def _like(t, lengths):
    """An output of t's shape, by token where t is; zeros where a sequence may leave rows unwritten."""
    make = torch.empty if lengths is None else torch.zeros
    if t.dim() > 2 and t.stride(1) < t.stride(2):
        B, h, N = t.shape[:3]
        return make((B, N, h) + t.shape[3:], dtype=t.dtype, device=t.device).transpose(1, 2)
    return make(t.shape, dtype=t.dtype, device=t.device)


def _delta_workspace(ws, backward, shape, device):
    if ws is None:
        n = capi.ttt_gated_delta_workspace_bytes(backward, shape)
        if n == 0:
            return None                 # the call itself reports why
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    return ws


def _ws_ptr(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def forward_gated_delta(Q, K, V, G, Beta, W0=None, lengths=None, scale=1.0, Z=None, W1_out=None, ws=None, stream=None):
    """The gated delta rule over whole sequences: per value head, from W0,
        W_t = exp(g_t) W_{t-1} + beta_t (v_t - exp(g_t) W_{t-1} k_t) k_t^T,   z_t = scale W_t q_t.
    W0: None (zeros), [heads][d_v][d_k] fp32 shared by the batch, or [B][heads][d_v][d_k].  lengths: None or
    [B] int32: the tokens of each sequence; rows of Z behind them are left as they were (zeros in a Z
    allocated here).  W1_out (optional, [B][heads][d_v][d_k] fp32) receives the last weights.  Returns Z."""
    shape, *n = _delta_shape(Q, K, V)
    B, hk, h, N, dk, dv = n
    with _On(Q, stream) as st:
        views = _inputs(Q, K, V, G, Beta, *n)
        w0, shared = _start(W0, B, h, dv, dk, Q.device)
        w1 = _state("W1_out", W1_out, (B, h, dv, dk), Q.device)
        lens = _ints("lengths", lengths, B, Q.device)
        if Z is None:
            Z = _like(V, lengths)
        z = _tokens("Z", Z, (B, h, N, dv), Q.dtype, Q.device)
        ws = _delta_workspace(ws, 0, shape, Q.device)
        _check(capi.ttt_forward_gated_delta(*views, w0, shared, lens, float(scale), z, w1, shape, *_ws_ptr(ws), st),
               "ttt_forward_gated_delta")
    return Z


def backward_gated_delta(Q, K, V, G, Beta, dZ, W0=None, dW1=None, lengths=None, scale=1.0, out=None, ws=None, stream=None):
    """Backward pass of forward_gated_delta for the upstream gradients dZ of Z and dW1 (None: none) of the last
    weights.  Returns (dQ, dK, dV, dG, dBeta, dW0): dQ and dK summed over the value heads that share a key
    head, dW0 like W0 (None without one; a shared W0's is summed over the batch).  `out` may supply those
    six tensors (dW0 None: not wanted); rows behind a sequence's length are left as they were there, and
    zeros otherwise."""
    shape, *n = _delta_shape(Q, K, V)
    B, hk, h, N, dk, dv = n
    with _On(Q, stream) as st:
        views = _inputs(Q, K, V, G, Beta, *n)
        dz = _tokens("dZ", dZ, (B, h, N, dv), Q.dtype, Q.device)
        w0, shared = _start(W0, B, h, dv, dk, Q.device)
        dw1 = _state("dW1", dW1, (B, h, dv, dk), Q.device)
        lens = _ints("lengths", lengths, B, Q.device)
        if out is None:
            out = [_like(t, lengths) for t in (Q, K, V, G, Beta)] + [None if W0 is None else torch.empty_like(W0)]
        dQ, dK, dV, dG, dBeta, dW0 = out
        if dW0 is not None and W0 is None:
            raise ValueError("dW0 needs W0")
        douts = (_tokens("dQ", dQ, (B, hk, N, dk), Q.dtype, Q.device), _tokens("dK", dK, (B, hk, N, dk), Q.dtype, Q.device),
                 _tokens("dV", dV, (B, h, N, dv), Q.dtype, Q.device), _tokens("dG", dG, (B, h, N), torch.float32, Q.device),
                 _tokens("dBeta", dBeta, (B, h, N), torch.float32, Q.device))
        dw0 = None if dW0 is None else _state("dW0", dW0, W0.shape, Q.device)
        ws = _delta_workspace(ws, 1, shape, Q.device)
        _check(capi.ttt_backward_gated_delta(*views, w0, shared, lens, float(scale), dz, dw1, shape, *_ws_ptr(ws), *douts,
                                             dw0, st), "ttt_backward_gated_delta")
    return dQ, dK, dV, dG, dBeta, dW0


def step_gated_delta(Q, K, V, G, Beta, W, slots=None, scale=1.0, Z=None, stream=None):
    """The recurrent form: the N (one, or a few) new tokens of each row of a batch, on the cache of states W
    [n_slots][heads][d_v][d_k] fp32, which is updated in place.  slots: [B] int32, the state of each row
    (None: row b uses state b); a row whose slot is not in 0 .. n_slots - 1 is unused, its rows of Z are left as
    they were (zeros in a Z allocated here).  Rows that name the same state take their steps in batch
    order.  Returns Z."""
    shape, *n = _delta_shape(Q, K, V)
    B, hk, h, N, dk, dv = n
    with _On(Q, stream) as st:
        views = _inputs(Q, K, V, G, Beta, *n)
        if W.dim() != 4:
            raise ValueError("W must be [n_slots][heads][d_v][d_k]")
        w = _state("W", W, (W.shape[0], h, dv, dk), Q.device)
        at = _ints("slots", slots, B, Q.device)
        if Z is None:
            Z = _like(V, slots)
        z = _tokens("Z", Z, (B, h, N, dv), Q.dtype, Q.device)
        _check(capi.ttt_step_gated_delta(*views, w, W.shape[0], at, float(scale), z, shape, st), "ttt_step_gated_delta")
    return Z


def clip_gradients(grads, max_norm, out=None, ws=None, stream=None):
    """Scales the gradients (bf16 or fp32 CUDA tensors, contiguous) by min(1, max_norm / norm), norm the
    2-norm over all their elements: in place, or into the tensors of `out` (same shapes and dtypes).
    Returns the norm before clipping, a 1-element fp32 tensor; nothing waits for the GPU."""
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("gradients must be CUDA tensors")
    if out is not None and len(out) != n:
        raise ValueError(f"{n} gradients and {len(out)} outputs")
    src, cnt, dts = (ctypes.c_void_p * n)(), (ctypes.c_longlong * n)(), (ctypes.c_int * n)()
    for i, g in enumerate(grads):
        if g.device != dev or not g.is_contiguous():
            raise ValueError("gradients must be contiguous tensors on one device")
        dt = _DTYPES.get(g.dtype)
        if dt is None:
            raise ValueError(f"unsupported dtype {g.dtype}")
        src[i], cnt[i], dts[i] = g.data_ptr(), g.numel(), dt
    dst = src
    if out is not None:
        dst = (ctypes.c_void_p * n)()
        for i, (o, g) in enumerate(zip(out, grads)):
            if o.shape != g.shape or o.dtype != g.dtype or o.device != dev or not o.is_contiguous():
                raise ValueError("outputs must be contiguous and like their gradients")
            dst[i] = o.data_ptr()
    with _On(grads[0], stream) as st:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
        if ws is None:
            ws = torch.empty(capi.ttt_clip_workspace_bytes(n), dtype=torch.uint8, device=dev)
        _check(capi.ttt_clip_gradients(src, dst, cnt, dts, n, float(max_norm), norm.data_ptr(), *_ws_ptr(ws), st),
               "ttt_clip_gradients")
    return norm
