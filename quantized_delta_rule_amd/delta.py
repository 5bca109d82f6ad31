"""Python binding of libstepq's sequence calls: the gated delta rule over whole sequences and single
tokens on FP32 states, and its gradient (argument marshalling only; see include/stepq.h for each call).

    from quantized_delta_rule_amd import delta
    delta.forward(q, k, v, alpha, beta, out, state_in=S0, state_out=S1, cu_seqlens=cu)   # prompts
    delta.forward(q, k, v, alpha, beta, out, state_in=S, state_out=S, slots=slots,       # decode
                  n_seqs=B, kind=delta.GDN)
    delta.backward(q, k, v, alpha, beta, d_out, dq, dk, dv, dalpha, dbeta, state_in=S0)

q, k are [tokens, key heads, d], v and out [tokens, value heads, d] (float32, bfloat16 or float16; the
token dimension may be strided, in multiples of 16 bytes), alpha [tokens, value heads] (GDN) or [tokens,
value heads, d] (KDA), beta [tokens, value heads], states [n, value heads, d, d], all float32.  Calls
enqueue kernels on `stream` (default: the current stream of the tensors' device) and return; every tensor
must stay alive until then as for any stream work.  A workspace is taken from torch's allocator on that
stream unless one is passed (uint8, 256-byte aligned, of forward_workspace(), backward_workspace() or
Plan.prefill_workspace() bytes; calls that may run at once need one each).

No call records an autograd graph: a program that trains calls forward() and backward() from the forward and
backward of a torch.autograd.Function.  forward() warns where a graph is wanted and none is recorded.
"""
from __future__ import annotations

import ctypes
import warnings

from .stepq import (DECAY_FIRST, DELTA_FIRST, GDN, KDA, StepqError, _check, _dev_tensor, lib)  # noqa: F401


class _SeqDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("order", ctypes.c_int), ("dtype", ctypes.c_int),
                ("n_qk_heads", ctypes.c_int), ("n_heads", ctypes.c_int), ("d", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("n_tokens", ctypes.c_int), ("device", ctypes.c_int),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong),
                ("cu_seqlens", ctypes.c_void_p), ("status", ctypes.c_void_p)]


_codes = None


def dtype_code(dtype):
    global _codes
    if _codes is None:
        import torch
        _codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, bfloat16 or float16 (got {dtype})")
    return code


def _tensor(t, name, dtype, shape, device):
    """Refuses what is no tensor of this type and shape on this device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != device:  # -1: not on a GPU
        raise ValueError(f"{name} must live on cuda:{device} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")


def _dense(t, name, dtype, shape, device):
    """Address of a contiguous tensor."""
    _tensor(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, shape, device):
    """(address, token stride in elements) of a [tokens, heads, d] tensor whose heads are packed."""
    _tensor(t, name, dtype, shape, device)
    n, heads, d = shape
    st = t.stride()
    if (d > 1 and st[2] != 1) or (heads > 1 and st[1] != d):
        raise ValueError(f"{name}: the heads of a token must be packed (strides {list(st)})")
    if n <= 1:
        return t.data_ptr(), heads * d
    if st[0] < heads * d:
        raise ValueError(f"{name}: tokens must not overlap (strides {list(st)})")
    return t.data_ptr(), st[0]


class _Sequences:
    """One call's checked description: shapes, strides, offsets, stream."""

    def __init__(self, q, k, v, alpha, beta, out, out_name, cu_seqlens, n_seqs, kind, order, status,
                 stream):
        import torch
        for t, name in ((q, "q"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch tensor")
            if t.dim() != 3:
                raise ValueError(f"{name} must be [tokens, heads, d]")
        self.device = dev = q.get_device()
        if dev < 0:
            raise ValueError(f"q must live on a GPU (got {q.device})")
        T, Hq, d = q.shape
        H = v.shape[1]
        dt, f = q.dtype, torch.float32
        self.T, self.Hq, self.H, self.d, self.dtype = T, Hq, H, d, dt
        code = dtype_code(dt)
        kind = int(kind)
        self.q, qs = _rows(q, "q", dt, (T, Hq, d), dev)
        self.k, ks = _rows(k, "k", dt, (T, Hq, d), dev)
        self.v, vs = _rows(v, "v", dt, (T, H, d), dev)
        self.out, os_ = _rows(out, out_name, dt, (T, H, d), dev)
        self.alpha = _dense(alpha, "alpha", f, (T, H, d) if kind == KDA else (T, H), dev)
        self.beta = _dense(beta, "beta", f, (T, H), dev)
        cu = None
        if cu_seqlens is not None:
            if not isinstance(cu_seqlens, torch.Tensor):
                raise TypeError("cu_seqlens must be a torch tensor")
            n = cu_seqlens.numel() - 1
            if cu_seqlens.dim() != 1 or n < 0:
                raise ValueError("cu_seqlens must be [n_seqs + 1]")
            if n_seqs is not None and n_seqs != n:
                raise ValueError(f"cu_seqlens holds {n} sequences, n_seqs is {n_seqs}")
            cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
        else:
            n = 1 if n_seqs is None else int(n_seqs)
        if T > 0x7FFFFFFF or n > 0x7FFFFFFF:
            raise ValueError(f"{T} tokens and {n} sequences: at most 2^31 - 1")
        self.N = n
        st = None if status is None else _dev_tensor(status, "status", torch.int32, 1, dev)
        self.desc = _SeqDesc(kind, int(order), code, Hq, H, d, n, T, dev, qs, ks, vs, os_, cu, st)
        self.current = stream is None
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        elif stream.device.index != dev:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{dev}")
        self.stream = stream

    def state(self, S, name, n=None):
        import torch
        if S is None:
            return None
        return _dense(S, name, torch.float32, (self.N if n is None else n, self.H, self.d, self.d), self.device)

    def workspace(self, given, need):
        """(pointer, bytes, keep-alive) of `need` bytes on the call's stream."""
        import torch
        if given is None:
            if need == 0:
                return None, 0, None
            if self.current:  # the allocator's block belongs to the stream that the call runs on
                given = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", self.device))
            else:
                with torch.cuda.stream(self.stream):
                    given = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", self.device))
            return given.data_ptr(), need, given
        p = _dev_tensor(given, "workspace", torch.uint8, given.numel(), self.device)
        return p, given.numel(), given

    def ptr(self):
        return self.stream.cuda_stream


def _need(fn, what, *args):
    n = ctypes.c_size_t()
    _check(fn(*args, ctypes.byref(n)), what)
    return int(n.value)


def _slots(slots, N, device):
    import torch
    return None if slots is None else _dense(slots, "slots", torch.int32, (N,), device)


def forward_workspace(q, k, v, alpha, beta, out, *, cu_seqlens=None, n_seqs=None, kind=GDN,
                      order=DELTA_FIRST):
    """Bytes of workspace that forward() with these arguments takes."""
    a = _Sequences(q, k, v, alpha, beta, out, "out", cu_seqlens, n_seqs, kind, order, None, None)
    return _need(lib().stepq_delta_forward_workspace, "delta_forward_workspace", ctypes.byref(a.desc))


def backward_workspace(q, k, v, alpha, beta, d_out, *, cu_seqlens=None, n_seqs=None, order=DELTA_FIRST):
    """Bytes of workspace that backward() with these arguments takes."""
    a = _Sequences(q, k, v, alpha, beta, d_out, "d_out", cu_seqlens, n_seqs, GDN, order, None, None)
    return _need(lib().stepq_delta_backward_workspace, "delta_backward_workspace", ctypes.byref(a.desc))


def _no_graph():
    import torch
    if torch.is_grad_enabled():
        warnings.warn("delta.forward records no graph: out and state_out get no gradient (call it from a "
                      "torch.autograd.Function, with delta.backward as its backward, or under torch.no_grad)",
                      stacklevel=3)


def forward(q, k, v, alpha, beta, out, *, state_in=None, state_out=None, cu_seqlens=None, n_seqs=None,
            slots=None, kind=GDN, order=DELTA_FIRST, status=None, workspace=None, stream=None):
    """Runs every sequence from its state: S_t = A_t S_{t-1} + beta_t k_t v_t^T, out_t = S_t^T q_t.

    cu_seqlens: int32 [n + 1] on the device, or None for n_seqs (default 1) equal sequences.  state_in:
    None = zero.  state_out: None = not kept; may be state_in (in place).  slots: int32 [n], sequence
    s uses state slots[s] of state_in and state_out, -1 = skip.  status: int32 [1], bad slots and offsets
    raise flags there."""
    a = _Sequences(q, k, v, alpha, beta, out, "out", cu_seqlens, n_seqs, kind, order, status, stream)
    n_slots = None
    if slots is not None:
        S = state_in if state_in is not None else state_out
        if S is None:
            raise ValueError("slots need state_in or state_out")
        n_slots = S.shape[0]
    si, so = a.state(state_in, "state_in", n_slots), a.state(state_out, "state_out", n_slots)
    if (q.requires_grad or k.requires_grad or v.requires_grad or alpha.requires_grad or beta.requires_grad
            or (state_in is not None and state_in.requires_grad)):
        _no_graph()
    sl = _slots(slots, a.N, a.device)
    L, d = lib(), ctypes.byref(a.desc)
    ws, size, keep = a.workspace(workspace, _need(L.stepq_delta_forward_workspace,
                                                  "delta_forward_workspace", d))
    _check(L.stepq_delta_forward(d, a.q, a.k, a.v, a.alpha, a.beta, si, so, n_slots or 0, sl, a.out,
                                 ws, size, a.ptr()), "delta_forward")


def backward(q, k, v, alpha, beta, d_out, dq, dk, dv, dalpha, dbeta, *, state_in=None, d_state_out=None,
             d_state_in=None, cu_seqlens=None, n_seqs=None, order=DELTA_FIRST, status=None,
             workspace=None, stream=None):
    """Gradient of forward() for GDN gates: from d_out and d_state_out (None = zero) into dq, dk, dv
    (packed), dalpha, dbeta and d_state_in (None = not wanted), all overwritten."""
    import torch
    a = _Sequences(q, k, v, alpha, beta, d_out, "d_out", cu_seqlens, n_seqs, GDN, order, status, stream)
    dev, T, f = a.device, a.T, torch.float32
    got = [_dense(t, name, dt, shape, dev)
           for t, name, shape, dt in ((dq, "dq", (T, a.Hq, a.d), a.dtype), (dk, "dk", (T, a.Hq, a.d), a.dtype),
                                      (dv, "dv", (T, a.H, a.d), a.dtype), (dalpha, "dalpha", (T, a.H), f),
                                      (dbeta, "dbeta", (T, a.H), f))]
    si = a.state(state_in, "state_in")
    ds1, ds0 = a.state(d_state_out, "d_state_out"), a.state(d_state_in, "d_state_in")
    L, d = lib(), ctypes.byref(a.desc)
    ws, size, keep = a.workspace(workspace, _need(L.stepq_delta_backward_workspace,
                                                  "delta_backward_workspace", d))
    _check(L.stepq_delta_backward(d, a.q, a.k, a.v, a.alpha, a.beta, si, a.out, ds1, *got, ds0, ws, size,
                                  a.ptr()), "delta_backward")
