"""Torch-facing wrappers of the gated delta rule (per-token test-time training of the linear inner model
with a forget gate) and of gradient clipping.  They allocate outputs and workspaces; the checks of the
tensors and the marshalling are native (``csrc/native.cpp``), since a call of a few microseconds of GPU work
should not wait for Python.

Tensor layout: Q, K [B][qk_heads][N][d_k] and V, Z [B][heads][N][d_v] with a contiguous last dimension and any
other strides the library accepts, so tensors laid out by token ([B][N][heads][d]) are passed as
``x.transpose(1, 2)`` without a copy.  G (log gates) and Beta are [B][heads][N] fp32, any strides.

Unlike the full-batch heads' calls, these allocate their workspace for the call (torch's allocator orders its
reuse on the call's stream), so calls on several streams and captured graphs share nothing.

A device-side wait that runs out (a copy that does not come within a second) leaves outputs unwritten and is recorded in the
call's workspace only.  A caller who wants to know passes a workspace (``gated_delta_workspace``) and reads it with
``workspace_status`` after the call.
"""
import torch

from . import capi

_native = None


def _lib():
    """The native binding (loaded once, with libttt.so).  Raises if it was not built."""
    global _native
    if _native is None:
        capi.lib()
        try:
            from . import _native as m
        except ImportError as e:
            raise RuntimeError(f"{e}: run `python -m vision_test_token_b200.build`") from e
        _native = m
    return _native


class _On:
    """A tensor's device, with `stream` (None: the device's current stream) current on it; gives the stream's handle."""

    __slots__ = ("device", "stream", "guards")

    def __init__(self, ref, stream):
        if not ref.is_cuda:
            raise ValueError("the tensors must be CUDA tensors")
        self.device, self.stream, self.guards = ref.device, stream, ()

    def __enter__(self):
        index = self.device.index
        if self.stream is not None and self.stream.device != self.device:
            raise ValueError("the stream belongs to another device than the tensors")
        if torch._C._cuda_getDevice() != index:
            self.guards = (torch.cuda.device(index),)
            self.guards[0].__enter__()
        if self.stream is not None:
            self.guards += (torch.cuda.stream(self.stream),)
            self.guards[-1].__enter__()
        return torch._C._cuda_getCurrentRawStream(index)

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _check(st, where):
    if st != capi.TTT_OK:
        raise capi.TttError(st, where)


def _like(t, lengths):
    """An output of t's shape, by token where t is; zeros where a sequence may leave rows unwritten."""
    make = torch.empty if lengths is None else torch.zeros
    if t.dim() > 2 and t.stride(1) < t.stride(2):
        B, h, N = t.shape[:3]
        return make((B, N, h) + t.shape[3:], dtype=t.dtype, device=t.device).transpose(1, 2)
    return make(t.shape, dtype=t.dtype, device=t.device)


def _workspace(backward, Q, V):
    n = _lib().workspace(backward, Q, V)
    return torch.empty(n, dtype=torch.uint8, device=Q.device) if n else None      # 0: the call itself reports why


def gated_delta_workspace(Q, V, backward=False):
    """A workspace for forward_gated_delta (backward: backward_gated_delta) on tensors of these shapes and type, to pass as `ws`.
    Calls that may run at the same time need distinct ones.  ``workspace_status(ws)`` waits for the stream and tells
    whether a device-side wait of the last call on it ran out."""
    with _On(Q, None):
        ws = _workspace(backward, Q, V)
    if ws is None:
        raise ValueError("no such gated delta shape (d_k and d_v are 64 or 128)")
    return ws


def forward_gated_delta(Q, K, V, G, Beta, W0=None, lengths=None, scale=1.0, Z=None, W1_out=None, ws=None, stream=None):
    """The gated delta rule over whole sequences: per value head, from W0,
        W_t = exp(g_t) W_{t-1} + beta_t (v_t - exp(g_t) W_{t-1} k_t) k_t^T,   z_t = scale W_t q_t.
    W0: None (zeros), [heads][d_v][d_k] fp32 shared by the batch, or [B][heads][d_v][d_k].  lengths: None or
    [B] int32: the tokens of each sequence; rows of Z behind them are left as they were (zeros in a Z
    allocated here).  W1_out (optional, [B][heads][d_v][d_k] fp32) receives the last weights.  ws: None (allocated for the call), or
    a gated_delta_workspace, whose status tells of a device-side wait that ran out.  Returns Z."""
    with _On(Q, stream) as st:
        if ws is None:
            ws = _workspace(False, Q, V)
        if Z is None:
            Z = _like(V, lengths)
        _check(_lib().forward(Q, K, V, G, Beta, W0, lengths, scale, Z, W1_out, ws, st), "ttt_forward_gated_delta")
    return Z


def backward_gated_delta(Q, K, V, G, Beta, dZ, W0=None, dW1=None, lengths=None, scale=1.0, out=None, ws=None, stream=None):
    """Backward pass of forward_gated_delta for the upstream gradients dZ of Z and dW1 (None: none) of the last
    weights.  Returns (dQ, dK, dV, dG, dBeta, dW0): dQ and dK summed over the value heads that share a key
    head, dW0 like W0 (None without one; a shared W0's is summed over the batch).  `out` may supply those
    six tensors (dW0 None: not wanted); rows behind a sequence's length are left as they were there, and
    zeros otherwise.  ws as in forward_gated_delta (with backward=True)."""
    with _On(Q, stream) as st:
        if ws is None:
            ws = _workspace(True, Q, V)
        if out is None:
            out = [_like(t, lengths) for t in (Q, K, V, G, Beta)] + [None if W0 is None else torch.empty_like(W0)]
        dQ, dK, dV, dG, dBeta, dW0 = out
        _check(_lib().backward(Q, K, V, G, Beta, dZ, W0, dW1, lengths, scale, dQ, dK, dV, dG, dBeta, dW0, ws, st),
               "ttt_backward_gated_delta")
    return dQ, dK, dV, dG, dBeta, dW0


def step_gated_delta(Q, K, V, G, Beta, W, slots=None, scale=1.0, Z=None, stream=None):
    """The recurrent form: the N (one, or a few) new tokens of each row of a batch, on the cache of states W
    [n_slots][heads][d_v][d_k] fp32, which is updated in place.  slots: [B] int32, the state of each row
    (None: row b uses state b); a row whose slot is not in 0 .. n_slots - 1 is unused, its rows of Z are left as
    they were (zeros in a Z allocated here).  Rows that name the same state take their steps in batch
    order.  Returns Z."""
    with _On(Q, stream) as st:
        if Z is None:
            Z = _like(V, slots)
        _check(_lib().step(Q, K, V, G, Beta, W, slots, scale, Z, st), "ttt_step_gated_delta")
    return Z


def clip_gradients(grads, max_norm, out=None, ws=None, stream=None):
    """Scales the gradients (bf16 or fp32 CUDA tensors, contiguous, or laid out by token as the gradients of
    backward_gated_delta are for such inputs: x.transpose(1, 2) is contiguous) by min(1, max_norm / norm), norm the
    2-norm over all their elements: in place, or into the tensors of `out` (same shapes, dtypes and layouts).
    Returns the norm before clipping, a 1-element fp32 tensor; nothing waits for the GPU."""
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    if out is not None and not isinstance(out, (list, tuple)):
        out = list(out)
    if not grads:
        raise ValueError("no gradients")
    with _On(grads[0], stream) as st:
        norm = torch.empty(1, dtype=torch.float32, device=grads[0].device)
        if ws is None:
            ws = torch.empty(capi.ttt_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device=norm.device)
        _check(_lib().clip(grads, out, max_norm, norm, ws, st), "ttt_clip_gradients")
    return norm
