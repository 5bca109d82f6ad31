"""Refusals of the sequence calls at the C boundary: every call below returns its error code and message
before it looks for a device, so all of this runs without one.  Pointers are made-up aligned numbers:
a refused call reads none of them."""
import ctypes

import pytest

INVALID, UNSUPPORTED = -1, -2
V = ctypes.c_void_p
AT = 4096  # an aligned address that nothing may read


@pytest.fixture(scope="module")
def L():
    from quantized_delta_rule_amd import stepq
    return stepq.lib()


def _desc(**kw):
    from quantized_delta_rule_amd import delta
    x = dict(kind=0, order=0, dtype=1, n_qk_heads=2, n_heads=4, d=128, n_seqs=2, n_tokens=128, device=0,
             q_stride=0, k_stride=0, v_stride=0, out_stride=0, cu_seqlens=None, status=None)
    x.update(kw)
    return delta._SeqDesc(*x.values())


def _refused(L, rc, code, text):
    msg = L.stepq_last_error().decode()
    assert rc == code and text in msg, (rc, msg)


BAD = [
    (dict(kind=2), INVALID, "kind"),
    (dict(order=-1), INVALID, "order"),
    (dict(dtype=3), INVALID, "dtype"),
    (dict(d=96), UNSUPPORTED, "d must be 64 or 128"),
    (dict(d=0), UNSUPPORTED, "d must be 64 or 128"),
    (dict(n_heads=3), INVALID, "multiple of n_qk_heads"),
    (dict(n_heads=0), INVALID, "multiple of n_qk_heads"),
    (dict(n_qk_heads=0), INVALID, "multiple of n_qk_heads"),
    (dict(n_qk_heads=-2), INVALID, "multiple of n_qk_heads"),
    (dict(n_heads=65536), INVALID, "65535"),
    (dict(n_seqs=-1), INVALID, "n_seqs"),
    (dict(n_tokens=-1), INVALID, "n_tokens"),
    (dict(n_seqs=0), INVALID, "without a sequence"),
    (dict(n_seqs=3), INVALID, "multiple of n_seqs"),
    (dict(n_seqs=2 ** 31 - 1, n_tokens=0), INVALID, "launch grid"),
    (dict(n_seqs=2 ** 21, n_tokens=0), INVALID, "launch grid"),
    (dict(n_seqs=1, n_tokens=2 ** 31 - 1), INVALID, "launch grid"),
    (dict(q_stride=248), INVALID, "q_stride"),       # tokens would overlap
    (dict(k_stride=260), INVALID, "k_stride"),       # not 16 bytes
    (dict(v_stride=516), INVALID, "v_stride"),
    (dict(dtype=0, v_stride=514), INVALID, "v_stride"),
    (dict(out_stride=-512), INVALID, "out_stride"),
    (dict(out_stride=2 ** 23), INVALID, "out_stride"),
]


@pytest.mark.parametrize("kw,code,text", BAD, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_bad_descriptions(L, kw, code, text):
    d, n = _desc(**kw), ctypes.c_size_t()
    ptr = [V(AT)] * 8
    for fn in (L.stepq_delta_forward_workspace, L.stepq_delta_backward_workspace):
        _refused(L, fn(ctypes.byref(d), ctypes.byref(n)), code, text)
    _refused(L, L.stepq_delta_forward(ctypes.byref(d), *ptr[:5], None, None, 0, None, V(AT), V(AT), 1 << 40,
                                      None), code, text)
    _refused(L, L.stepq_delta_backward(ctypes.byref(d), *ptr[:5], None, V(AT), None, *ptr[:5], None, V(AT),
                                       1 << 40, None), code, text)


def test_missing_pieces(L):
    n = ctypes.c_size_t()
    _refused(L, L.stepq_delta_forward_workspace(None, ctypes.byref(n)), INVALID, "desc is NULL")
    d = ctypes.byref(_desc())
    _refused(L, L.stepq_delta_forward_workspace(d, None), INVALID, "bytes is NULL")
    _refused(L, L.stepq_delta_backward_workspace(d, None), INVALID, "bytes is NULL")
    kda = ctypes.byref(_desc(kind=1))
    _refused(L, L.stepq_delta_backward_workspace(kda, ctypes.byref(n)), UNSUPPORTED, "STEPQ_KIND_GDN only")
    # the handle of a plan
    _refused(L, L.stepq_prefill_workspace(None, d, ctypes.byref(n)), INVALID, "plan is NULL")
    _refused(L, L.stepq_read_slots(None, V(AT), 1, V(AT), 1, V(AT), 0, None), INVALID, "plan is NULL")
    _refused(L, L.stepq_prefill_slots(None, d, V(AT), 1, *[V(AT)] * 8, 0, None), INVALID, "plan is NULL")


@pytest.mark.parametrize("i", range(7))
def test_forward_pointers(L, i):
    """NULL and misaligned q, k, v, alpha, beta, out; the workspace's size, pointer and alignment."""
    def call(p, ws=AT, size=1 << 40, S=None, n_slots=0, slots=None):
        return L.stepq_delta_forward(ctypes.byref(_desc()), *[V(x) if x else None for x in p[:5]], S, None,
                                     n_slots, slots, V(p[5]) if p[5] else None, V(ws) if ws else None, size, None)
    p = [AT] * 6
    if i < 6:
        p[i] = 0
        _refused(L, call(p), INVALID, "non-NULL")
        p[i] = AT + 2
        _refused(L, call(p), INVALID, "aligned")
        return
    _refused(L, call(p, size=0), INVALID, "workspace of 0 bytes")
    _refused(L, call(p, ws=0), INVALID, "workspace is NULL")
    _refused(L, call(p, ws=AT + 128), INVALID, "workspace must be 256-byte aligned")
    _refused(L, call(p, S=V(AT + 4)), INVALID, "S_in must be 16-byte aligned")
    _refused(L, call(p, slots=V(AT)), INVALID, "n_slots must be >= 1")


@pytest.mark.parametrize("i", range(11))
def test_backward_pointers(L, i):
    def call(p, ws=AT, size=1 << 40, S=None):
        q = [V(x) if x else None for x in p]
        return L.stepq_delta_backward(ctypes.byref(_desc()), *q[:5], S, q[5], None, *q[6:11], None, V(ws), size,
                                      None)
    p = [AT] * 11
    p[i] = 0
    _refused(L, call(p), INVALID, "non-NULL")
    p[i] = AT + 2
    _refused(L, call(p), INVALID, "aligned")
    p[i] = AT
    _refused(L, call(p, size=1024), INVALID, "workspace of 1024 bytes")
    _refused(L, call(p, S=V(AT + 8)), INVALID, "S_in must be 16-byte aligned")


def test_good_calls_fail_only_at_the_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    n = ctypes.c_size_t()
    d = ctypes.byref(_desc())
    for fn in (L.stepq_delta_forward_workspace, L.stepq_delta_backward_workspace):
        _refused(L, fn(d, ctypes.byref(n)), INVALID, "device 0 not available")
    _refused(L, L.stepq_delta_forward(d, *[V(AT)] * 5, None, None, 0, None, V(AT), V(AT), 1 << 40, None), INVALID,
             "device 0 not available")
    _refused(L, L.stepq_delta_backward(d, *[V(AT)] * 5, None, V(AT), None, *[V(AT)] * 5, None, V(AT), 1 << 40,
                                       None), INVALID, "device 0 not available")


def test_python_refusals():
    torch = pytest.importorskip("torch")
    from quantized_delta_rule_amd import delta
    x = torch.zeros(4, 2, 64)
    a = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        delta.forward(x, x, x, a, a, x)
    with pytest.raises(TypeError, match="v must be a torch tensor"):
        delta.forward(x, x, None, a, a, x)
    with pytest.raises(ValueError, match="tokens, heads, d"):
        delta.backward(x[0], x, x, a, a, x, x, x, x, a, a)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        delta.dtype_code(torch.float64)
