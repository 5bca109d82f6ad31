"""Python binding of libstepq's short causal convolution and its gradient (argument marshalling only; see
include/stepq.h).

    from quantized_delta_rule_amd import conv
    conv.forward(x, weight, out, bias=b, state_in=S0, state_out=S1, cu_seqlens=cu)             # prompts
    conv.forward(x, weight, out, bias=b, state_in=S, state_out=S, slots=slots, n_seqs=B)      # decode
    conv.backward(x, weight, d_out, dx, dweight, bias=b, dbias=db, state_in=S0, cu_seqlens=cu)

x, out and their gradients are [tokens, channels] (float32, bfloat16 or float16; the token dimension may be strided, in
multiples of 16 bytes), weight [channels, width] and bias [channels] of one of those types, states [n, width - 1,
channels] of x's: the last inputs, oldest first.  dweight and dbias are float32.  Streams, workspaces, offsets and
slots are as for delta.forward; no call records an autograd graph.
"""
from __future__ import annotations

import ctypes

import torch

from .layer import (any_dense, dense, device_of, dtype_code, need, no_graph, rows, sequences, slots_of, status_of,
                    stream_of, workspace_of)
from .stepq import StepqError, _check, lib  # noqa: F401

NONE, SILU = 0, 1


class _ConvDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("param_dtype", ctypes.c_int), ("channels", ctypes.c_int),
                ("width", ctypes.c_int), ("activation", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("n_tokens", ctypes.c_int), ("device", ctypes.c_int), ("x_stride", ctypes.c_longlong),
                ("out_stride", ctypes.c_longlong), ("cu_seqlens", ctypes.c_void_p), ("status", ctypes.c_void_p)]


def _describe(x, weight, bias, out, out_name, activation, cu_seqlens, n_seqs, status):
    """(description, device, x's, out's, weight's and bias's addresses, sequences, tokens, channels, width)."""
    dev = device_of(x, "x", (2,))
    T, C = x.shape
    dt = x.dtype
    code = dtype_code(dt)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [channels, width]")
    W = weight.shape[1]
    px, xs = rows(x, "x", dt, (T, C), dev)
    po, os_ = rows(out, out_name, dt, (T, C), dev)
    pw, pcode = any_dense(weight, "weight", (C, W), dev)
    pb = dense(bias, "bias", weight.dtype, (C,), dev)
    n, cu = sequences(cu_seqlens, n_seqs, T, dev)
    desc = _ConvDesc(code, pcode, C, W, int(activation), n, T, dev, xs, os_, cu, status_of(status, dev))
    return desc, dev, px, po, pw, pb, n, T, C, W


def forward(x, weight, out, *, bias=None, activation=SILU, state_in=None, state_out=None, cu_seqlens=None,
            n_seqs=None, slots=None, status=None, stream=None):
    """out_t = act(bias + sum_j weight[:, j] x_{t - (width - 1) + j}) over every sequence by itself; activation SILU
    or NONE.  state_in: inputs before the first token (None = zeros).  state_out: None = not kept; may be state_in
    (in place).  cu_seqlens, n_seqs, slots and status as for delta.forward."""
    d, dev, px, po, pw, pb, n, _, C, W = _describe(x, weight, bias, out, "out", activation, cu_seqlens, n_seqs, status)
    sl, many = slots_of(slots, state_in, state_out, n, dev)
    shape = (many, W - 1, C)
    si = dense(state_in, "state_in", x.dtype, shape, dev)
    so = si if state_out is state_in else dense(state_out, "state_out", x.dtype, shape, dev)
    no_graph("conv", x, weight, bias, state_in)
    _check(lib().stepq_conv_forward(ctypes.byref(d), px, pw, pb, si, so, many if sl else 0, sl, po, stream_of(stream, dev)),
           "conv_forward")


def backward_workspace(x, weight, d_out, *, bias=None, activation=SILU, cu_seqlens=None, n_seqs=None):
    """Bytes of workspace that backward() with these arguments takes."""
    d = _describe(x, weight, bias, d_out, "d_out", activation, cu_seqlens, n_seqs, None)[0]
    return need(lib().stepq_conv_backward_workspace, "conv_backward_workspace", ctypes.byref(d))


def backward(x, weight, d_out, dx, dweight, *, bias=None, dbias=None, activation=SILU, state_in=None,
             d_state_out=None, d_state_in=None, cu_seqlens=None, n_seqs=None, status=None, workspace=None, stream=None):
    """Gradient of forward(): from d_out and d_state_out (None = zero) into dx (packed), dweight, dbias and d_state_in
    (None = not wanted), all overwritten."""
    d, dev, px, po, pw, pb, n, T, C, W = _describe(x, weight, bias, d_out, "d_out", activation, cu_seqlens, n_seqs, status)
    dt, f = x.dtype, torch.float32
    shape = (n, W - 1, C)
    si, ds1 = dense(state_in, "state_in", dt, shape, dev), dense(d_state_out, "d_state_out", dt, shape, dev)
    ds0 = dense(d_state_in, "d_state_in", dt, shape, dev)
    gx, gw = dense(dx, "dx", dt, (T, C), dev), dense(dweight, "dweight", f, (C, W), dev)
    gb = dense(dbias, "dbias", f, (C,), dev)
    p = ctypes.byref(d)
    ws, size, keep = workspace_of(workspace, need(lib().stepq_conv_backward_workspace, "conv_backward_workspace", p),
                                  dev, stream)
    _check(lib().stepq_conv_backward(p, px, pw, pb, si, po, ds1, gx, gw, gb, ds0, ws, size, stream_of(stream, dev)),
           "conv_backward")
