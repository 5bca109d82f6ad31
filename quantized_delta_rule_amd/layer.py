"""What the bindings of the operators around the recurrence (conv, scan, norm) share: checks of tensors, the
sequences' description, streams and workspaces."""
from __future__ import annotations

import ctypes

import torch

from .delta import _dense, _tensor, dtype_code  # noqa: F401
from .stepq import _check, _dev_tensor

Tensor = torch.Tensor


def device_of(t, name, dims):
    """Device of the call: that of its first tensor."""
    if not isinstance(t, Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions (got {t.dim()})")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must live on a GPU (got {t.device})")
    return dev


def rows(t, name, dtype, shape, device):
    """(address, row stride in elements, 0 = packed) of a tensor whose rows are packed and do not overlap."""
    if type(t) is Tensor and t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr(), 0
    _tensor(t, name, dtype, shape, device)
    st, inner = t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] > 1 and st[i] != inner:
            raise ValueError(f"{name}: the elements of a row must be packed (strides {list(st)})")
        inner *= shape[i]
    if shape[0] <= 1 or inner == 0:
        return t.data_ptr(), 0
    if st[0] < inner:
        raise ValueError(f"{name}: rows must not overlap (strides {list(st)})")
    return t.data_ptr(), 0 if st[0] == inner else st[0]


def dense(t, name, dtype, shape, device):
    """Address of a contiguous tensor (None: no tensor)."""
    if t is None:
        return None
    if type(t) is Tensor and t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    return _dense(t, name, dtype, shape, device)


def any_dense(t, name, shape, device):
    """(address, dtype code) of a contiguous parameter of one of the row types."""
    if not isinstance(t, Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    return dense(t, name, t.dtype, shape, device), dtype_code(t.dtype)


def sequences(cu_seqlens, n_seqs, T, device):
    """(number of sequences, address of their offsets or None)."""
    if T > 0x7FFFFFFF:
        raise ValueError(f"{T} tokens: at most 2^31 - 1")
    if cu_seqlens is None:
        n = 1 if n_seqs is None else int(n_seqs)
        if not 0 <= n <= 0x7FFFFFFF:
            raise ValueError(f"n_seqs must be 0 .. 2^31 - 1 (got {n})")
        return n, None
    if not isinstance(cu_seqlens, Tensor):
        raise TypeError("cu_seqlens must be a torch tensor")
    n = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or n < 0:
        raise ValueError("cu_seqlens must be [n_seqs + 1]")
    if n_seqs is not None and n_seqs != n:
        raise ValueError(f"cu_seqlens holds {n} sequences, n_seqs is {n_seqs}")
    return n, dense(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), device)


def status_of(status, device):
    return None if status is None else _dev_tensor(status, "status", torch.int32, 1, device)


def slots_of(slots, state_in, state_out, n, device):
    """(address of the slots or None, how many states the states hold)."""
    if slots is None:
        return None, n
    S = state_in if state_in is not None else state_out
    if S is None:
        raise ValueError("slots need state_in or state_out")
    return dense(slots, "slots", torch.int32, (n,), device), S.shape[0]


def stream_of(stream, device):
    """Handle of the call's stream."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device)
    if stream.device.index != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{device}")
    return stream.cuda_stream


# the current stream's handle without an object around it (a quarter of a microsecond a call instead of one)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def workspace_of(given, need, device, stream):
    """(address, bytes, keep-alive) of `need` bytes on the call's stream."""
    if given is not None:
        return _dev_tensor(given, "workspace", torch.uint8, given.numel(), device), given.numel(), given
    if need == 0:
        return None, 0, None
    if stream is None:  # the allocator's block belongs to the stream that the call runs on
        given = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", device))
    else:
        with torch.cuda.stream(stream):
            given = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", device))
    return given.data_ptr(), need, given


def need(fn, what, desc):
    n = ctypes.c_size_t()
    _check(fn(desc, ctypes.byref(n)), what)
    return n.value


def no_graph(what, *tensors):
    """Says that a forward call records no graph where one is wanted."""
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            import warnings
            warnings.warn(f"{what}.forward records no graph: its outputs get no gradient (call it from a "
                          f"torch.autograd.Function, with {what}.backward as its backward, or under torch.no_grad)",
                          stacklevel=3)
            return
