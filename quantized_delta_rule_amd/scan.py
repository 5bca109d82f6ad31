"""Python binding of libstepq's selective state space scan and its gradient (argument marshalling only; see
include/stepq.h).

    from quantized_delta_rule_amd import scan
    scan.forward(x, dt, A, B, C, out, D=D, dt_bias=bias, z=z, state_in=S0, state_out=S1, cu_seqlens=cu)    # prompts
    scan.forward(x, dt, A, B, C, out, D=D, dt_bias=bias, z=z, state_in=S, state_out=S, slots=slots, n_seqs=B)
    scan.backward(x, dt, A, B, C, d_out, dx, ddt, dA, dB, dC, D=D, dD=dD, z=z, dz=dz, state_in=S0)

x, dt, z and out are [tokens, channels], B and C [tokens, groups, states] (float32, bfloat16 or float16; the token
dimension may be strided, in multiples of 16 bytes), A [channels, states], D and dt_bias [channels] and the states [n,
channels, states] float32.  Streams, workspaces, offsets and slots are as for delta.forward; no call records an
autograd graph.
"""
from __future__ import annotations

import ctypes

import torch

from .layer import (dense, device_of, dtype_code, need, no_graph, rows, sequences, slots_of, status_of, stream_of,
                    workspace_of)
from .stepq import StepqError, _check, lib  # noqa: F401


class _ScanDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("channels", ctypes.c_int), ("n_groups", ctypes.c_int),
                ("d_state", ctypes.c_int), ("softplus", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("n_tokens", ctypes.c_int), ("device", ctypes.c_int), ("x_stride", ctypes.c_longlong),
                ("dt_stride", ctypes.c_longlong), ("z_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong),
                ("b_stride", ctypes.c_longlong), ("c_stride", ctypes.c_longlong), ("cu_seqlens", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class _Call:
    """One call's checked description and inputs."""

    def __init__(self, x, dt, A, B, C, out, out_name, D, dt_bias, softplus, z, cu_seqlens, n_seqs, status):
        self.dev = dev = device_of(x, "x", (2,))
        T, ch = x.shape
        if not isinstance(B, torch.Tensor) or B.dim() != 3:
            raise ValueError("B must be a tensor [tokens, groups, states]")
        G, n = B.shape[1], B.shape[2]
        t, f = x.dtype, torch.float32
        code = dtype_code(t)
        self.T, self.ch, self.G, self.n, self.dtype = T, ch, G, n, t
        px, xs = rows(x, "x", t, (T, ch), dev)
        pdt, ds = rows(dt, "dt", t, (T, ch), dev)
        pb, bs = rows(B, "B", t, (T, G, n), dev)
        pc, cs = rows(C, "C", t, (T, G, n), dev)
        pz, zs = (None, 0) if z is None else rows(z, "z", t, (T, ch), dev)
        self.out, os_ = rows(out, out_name, t, (T, ch), dev)
        self.inputs = (px, pdt, dense(A, "A", f, (ch, n), dev), pb, pc, dense(D, "D", f, (ch,), dev),
                       dense(dt_bias, "dt_bias", f, (ch,), dev), pz)
        if A is None:
            raise TypeError("A must be a torch tensor")
        self.N, cu = sequences(cu_seqlens, n_seqs, T, dev)
        self.desc = _ScanDesc(code, ch, G, n, 1 if softplus else 0, self.N, T, dev, xs, ds, zs, os_, bs, cs, cu,
                              status_of(status, dev))
        self.ptr = ctypes.byref(self.desc)

    def state(self, S, name, many=None):
        return dense(S, name, torch.float32, (self.N if many is None else many, self.ch, self.n), self.dev)


def forward_workspace(x, dt, A, B, C, out, *, D=None, dt_bias=None, softplus=True, z=None, cu_seqlens=None, n_seqs=None):
    """Bytes of workspace that forward() with these arguments takes."""
    a = _Call(x, dt, A, B, C, out, "out", D, dt_bias, softplus, z, cu_seqlens, n_seqs, None)
    return need(lib().stepq_scan_forward_workspace, "scan_forward_workspace", a.ptr)


def backward_workspace(x, dt, A, B, C, d_out, *, D=None, dt_bias=None, softplus=True, z=None, cu_seqlens=None,
                       n_seqs=None):
    """Bytes of workspace that backward() with these arguments takes."""
    a = _Call(x, dt, A, B, C, d_out, "d_out", D, dt_bias, softplus, z, cu_seqlens, n_seqs, None)
    return need(lib().stepq_scan_backward_workspace, "scan_backward_workspace", a.ptr)


def forward(x, dt, A, B, C, out, *, D=None, dt_bias=None, softplus=True, z=None, state_in=None, state_out=None,
            cu_seqlens=None, n_seqs=None, slots=None, status=None, workspace=None, stream=None):
    """Runs every sequence from its state: h_t = exp(step A) h_{t-1} + step B_t x_t, out_t = (C_t . h_t + D x_t) z
    sigmoid(z), step = softplus(dt + dt_bias) (softplus=False: dt + dt_bias).

    state_in: None = zero.  state_out: None = not kept; may be state_in (in place).  cu_seqlens, n_seqs, slots and
    status as for delta.forward."""
    a = _Call(x, dt, A, B, C, out, "out", D, dt_bias, softplus, z, cu_seqlens, n_seqs, status)
    sl, many = slots_of(slots, state_in, state_out, a.N, a.dev)
    si = a.state(state_in, "state_in", many)
    so = si if state_out is state_in else a.state(state_out, "state_out", many)
    no_graph("scan", x, dt, A, B, C, D, dt_bias, z, state_in)
    ws, size, keep = workspace_of(workspace, need(lib().stepq_scan_forward_workspace, "scan_forward_workspace", a.ptr),
                                  a.dev, stream)
    _check(lib().stepq_scan_forward(a.ptr, *a.inputs, si, so, many if sl else 0, sl, a.out, ws, size, stream_of(stream, a.dev)),
           "scan_forward")


def backward(x, dt, A, B, C, d_out, dx, ddt, dA, dB, dC, *, D=None, dD=None, dt_bias=None, ddt_bias=None,
             softplus=True, z=None, dz=None, state_in=None, d_state_out=None, d_state_in=None, cu_seqlens=None,
             n_seqs=None, status=None, workspace=None, stream=None):
    """Gradient of forward(): from d_out and d_state_out (None = zero) into dx, ddt, dz [tokens, channels], dB, dC
    (packed), dA, dD, ddt_bias and d_state_in (None = not wanted), all overwritten."""
    a = _Call(x, dt, A, B, C, d_out, "d_out", D, dt_bias, softplus, z, cu_seqlens, n_seqs, status)
    f, dev, t = torch.float32, a.dev, a.dtype
    for v, name in ((dx, "dx"), (ddt, "ddt"), (dA, "dA"), (dB, "dB"), (dC, "dC")):
        if v is None:
            raise TypeError(f"{name} must be a torch tensor")
    if (z is None) != (dz is None):
        raise ValueError("dz goes with z")
    wide, bc = (a.T, a.ch), (a.T, a.G, a.n)
    got = (dense(dx, "dx", t, wide, dev), dense(ddt, "ddt", t, wide, dev), dense(dA, "dA", f, (a.ch, a.n), dev),
           dense(dB, "dB", t, bc, dev), dense(dC, "dC", t, bc, dev), dense(dD, "dD", f, (a.ch,), dev),
           dense(ddt_bias, "ddt_bias", f, (a.ch,), dev), dense(dz, "dz", t, wide, dev),
           a.state(d_state_in, "d_state_in"))
    si, ds1 = a.state(state_in, "state_in"), a.state(d_state_out, "d_state_out")
    ws, size, keep = workspace_of(workspace, need(lib().stepq_scan_backward_workspace, "scan_backward_workspace", a.ptr),
                                  dev, stream)
    _check(lib().stepq_scan_backward(a.ptr, *a.inputs, si, a.out, ds1, *got, ws, size, stream_of(stream, a.dev)), "scan_backward")
