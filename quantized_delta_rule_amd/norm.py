"""Python binding of libstepq's root-mean-square norm and its gradient (argument marshalling only; see
include/stepq.h).

    from quantized_delta_rule_amd import norm
    norm.forward(x, weight, out, z=z, gate=norm.SILU)                             # a layer's readout, per head
    norm.forward(x, weight, out, residual=r, residual_out=r)                      # the next block's input
    norm.forward(x, weight, codes, residual=r, residual_out=r, scale=scale)       # eight bits with scales
    norm.backward(h, weight, d_out, dx, dweight, d_residual=dr)

Rows are [tokens, d] or [tokens, heads, d] (float32, bfloat16 or float16; each head's row is normed by itself; the token
dimension may be strided, in multiples of 16 bytes); weight [d] is of one of those types.  out has x's type, or is
torch.float8_e4m3fn or torch.int8 with scale [tokens(, heads)] (group = 0) or [tokens(, heads), d / group].  Streams and
workspaces are as for delta.forward; no call records an autograd graph.
"""
from __future__ import annotations

import ctypes

import torch

from .layer import (any_dense, dense, device_of, dtype_code, need, no_graph, rows, stream_of, workspace_of)
from .stepq import StepqError, _check, lib  # noqa: F401

SILU, SIGMOID = 1, 2


class _NormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("param_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("n_rows", ctypes.c_int), ("n_heads", ctypes.c_int), ("d", ctypes.c_int), ("gate", ctypes.c_int),
                ("group", ctypes.c_int), ("eps", ctypes.c_float), ("device", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("residual_stride", ctypes.c_longlong),
                ("z_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong)]


def _shape(x):
    """(device, shape, rows, heads, d)."""
    dev = device_of(x, "x", (2, 3))
    shape = tuple(x.shape)
    if shape[0] > 0x7FFFFFFF:
        raise ValueError(f"{shape[0]} rows: at most 2^31 - 1")
    return dev, shape, shape[0], shape[1] if len(shape) == 3 else 1, shape[-1]


def forward(x, weight, out, *, eps=1e-6, residual=None, residual_out=None, z=None, gate=SILU, scale=None, group=0,
            stream=None):
    """out = h / sqrt(mean(h^2) + eps) * weight * act(z), h = x + residual; residual_out = h, rounded once.

    weight None: ones.  gate: what z goes through, SILU or SIGMOID.  8-bit out: scale = max |y| / 448 (e4m3) or
    / 127 (int8) of a row or of every `group` columns, out = y / scale to the nearest.  out and residual_out may
    each be x, residual or z, with its type and strides (in place)."""
    dev, shape, R, H, d = _shape(x)
    t = x.dtype
    code = dtype_code(t)
    px, xs = rows(x, "x", t, shape, dev)
    pw, pcode = (None, code) if weight is None else any_dense(weight, "weight", (d,), dev)
    pr, rs = (None, 0) if residual is None else rows(residual, "residual", t, shape, dev)
    pz, zs = (None, 0) if z is None else rows(z, "z", t, shape, dev)
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch tensor")
    ot = out.dtype
    ocode = code if ot is t else 3 if ot is torch.float8_e4m3fn else 4 if ot is torch.int8 else None
    if ocode is None:
        raise TypeError(f"out must be {t}, torch.float8_e4m3fn or torch.int8 (got {ot})")
    po, os_ = rows(out, "out", ot, shape, dev)
    if residual_out is None:
        ph = None
    else:
        ph, hs = rows(residual_out, "residual_out", t, shape, dev)
        if residual is None:
            rs = hs
        elif hs != rs:
            raise ValueError("residual_out must have residual's strides")
    group = int(group)
    if (ocode == code) != (scale is None):
        raise ValueError("scale goes with an 8-bit out")
    if group < 0 or (group and d % group):
        raise ValueError(f"group must divide d = {d} (got {group})")
    ps = dense(scale, "scale", torch.float32, shape[:-1] + ((d // group,) if group else ()), dev)
    no_graph("norm", x, weight, residual, z)
    desc = _NormDesc(code, pcode, ocode, R, H, d, int(gate), group, eps, dev, xs, rs, zs, os_)
    _check(lib().stepq_norm_forward(ctypes.byref(desc), px, pw, pr, pz, po, ps, ph, stream_of(stream, dev)),
           "norm_forward")


def _describe_grad(h, weight, d_out, eps, z, gate, d_residual):
    dev, shape, R, H, d = _shape(h)
    t = h.dtype
    code = dtype_code(t)
    px, xs = rows(h, "h", t, shape, dev)
    pw, pcode = (None, code) if weight is None else any_dense(weight, "weight", (d,), dev)
    pz, zs = (None, 0) if z is None else rows(z, "z", t, shape, dev)
    po, os_ = rows(d_out, "d_out", t, shape, dev)
    pr, rs = (None, 0) if d_residual is None else rows(d_residual, "d_residual", t, shape, dev)
    return (_NormDesc(code, pcode, code, R, H, d, int(gate), 0, eps, dev, xs, rs, zs, os_), dev, shape,
            (px, pw, pz, po, pr))


def backward_workspace(h, weight, d_out, *, eps=1e-6, z=None, gate=SILU, d_residual=None):
    """Bytes of workspace that backward() with these arguments and a dweight takes (without one: none)."""
    d = _describe_grad(h, weight, d_out, eps, z, gate, d_residual)[0]
    return need(lib().stepq_norm_backward_workspace, "norm_backward_workspace", ctypes.byref(d))


def backward(h, weight, d_out, dx, dweight=None, *, eps=1e-6, z=None, dz=None, gate=SILU, d_residual=None,
             workspace=None, stream=None):
    """Gradient of forward() at h (x, or x + residual as residual_out keeps it): from d_out and d_residual (the gradient
    that reaches h beside the norm; None = zero) into dx (packed; the gradient of x and of the residual alike), dz and
    dweight (float32; None = not wanted), all overwritten.  dx and dz may each be a packed h, d_out, z or d_residual."""
    desc, dev, shape, p = _describe_grad(h, weight, d_out, eps, z, gate, d_residual)
    if dx is None:
        raise TypeError("dx must be a torch tensor")
    if (z is None) != (dz is None):
        raise ValueError("dz goes with z")
    gx, gz = dense(dx, "dx", h.dtype, shape, dev), dense(dz, "dz", h.dtype, shape, dev)
    gw = dense(dweight, "dweight", torch.float32, (shape[-1],), dev)
    d = ctypes.byref(desc)
    room = 0 if dweight is None else need(lib().stepq_norm_backward_workspace, "norm_backward_workspace", d)
    ws, size, keep = workspace_of(workspace, room, dev, stream)
    _check(lib().stepq_norm_backward(d, *p, gx, gw, gz, ws, size, stream_of(stream, dev)), "norm_backward")
