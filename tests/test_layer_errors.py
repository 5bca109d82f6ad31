"""Refusals of the convolution, the scan and the norm: every call below returns its error code and message before it
looks for a device, so all of this runs without one.  Pointers are made-up aligned numbers: a refused call
reads none of them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

INVALID, UNSUPPORTED = -1, -2
V = ctypes.c_void_p
AT = 4096  # an aligned address that nothing may read
MANY = [ctypes.c_void_p(AT * (i + 1)) for i in range(32)]  # .. and others, no two the same


@pytest.fixture(scope="module")
def L():
    from quantized_delta_rule_amd import stepq
    return stepq.lib()


def conv_desc(**kw):
    from quantized_delta_rule_amd import conv
    x = dict(dtype=1, param_dtype=0, channels=64, width=4, activation=1, n_seqs=2, n_tokens=128, device=0, x_stride=0,
             out_stride=0, cu_seqlens=None, status=None)
    x.update(kw)
    return conv._ConvDesc(*x.values())


def scan_desc(**kw):
    from quantized_delta_rule_amd import scan
    x = dict(dtype=1, channels=64, n_groups=2, d_state=16, softplus=1, n_seqs=2, n_tokens=128, device=0, x_stride=0,
             dt_stride=0, z_stride=0, out_stride=0, b_stride=0, c_stride=0, cu_seqlens=None, status=None)
    x.update(kw)
    return scan._ScanDesc(*x.values())


def norm_desc(**kw):
    from quantized_delta_rule_amd import norm
    x = dict(dtype=1, param_dtype=0, out_dtype=1, n_rows=16, n_heads=2, d=128, gate=1, group=0, eps=1e-6, device=0,
             x_stride=0, residual_stride=0, z_stride=0, out_stride=0)
    x.update(kw)
    return norm._NormDesc(*x.values())


def refused(L, rc, code, text):
    msg = L.stepq_last_error().decode()
    assert rc == code and text in msg, (rc, msg)


def conv_calls(L, d):
    """Every call of the convolution with this description, all pointers good."""
    n = ctypes.c_size_t()
    p, q = ctypes.byref(d), MANY
    return [L.stepq_conv_forward(p, *q[:5], 0, None, q[5], None), L.stepq_conv_backward_workspace(p, ctypes.byref(n)),
            L.stepq_conv_backward(p, *q[:11], 1 << 40, None)]


def scan_calls(L, d):
    n = ctypes.c_size_t()
    p, q = ctypes.byref(d), MANY
    return [L.stepq_scan_forward_workspace(p, ctypes.byref(n)), L.stepq_scan_backward_workspace(p, ctypes.byref(n)),
            L.stepq_scan_forward(p, *q[:10], 0, None, q[10], q[11], 1 << 40, None),
            L.stepq_scan_backward(p, *q[:21], 1 << 40, None)]


def norm_calls(L, d):
    n = ctypes.c_size_t()
    p, q = ctypes.byref(d), MANY
    return [L.stepq_norm_forward(p, *q[:7], None), L.stepq_norm_backward_workspace(p, ctypes.byref(n)),
            L.stepq_norm_backward(p, *q[:9], 1 << 40, None)]


SEQS = [
    (dict(n_seqs=-1), INVALID, "n_seqs"), (dict(n_tokens=-1), INVALID, "n_seqs"),
    (dict(n_seqs=0), INVALID, "without a sequence"), (dict(n_seqs=3), INVALID, "multiple of n_seqs"),
    (dict(n_seqs=2 ** 31 - 1, n_tokens=0), INVALID, "launch grid"),
]


@pytest.mark.parametrize("kw,code,text", SEQS + [
    (dict(dtype=3), INVALID, "dtype"), (dict(param_dtype=-1), INVALID, "param_dtype"),
    (dict(channels=0), INVALID, "channels"), (dict(channels=60), INVALID, "multiple of 8"),
    (dict(channels=2 ** 24 + 8), INVALID, "channels"), (dict(width=1), UNSUPPORTED, "width"),
    (dict(width=5), UNSUPPORTED, "width"), (dict(activation=2), INVALID, "activation"),
    (dict(n_seqs=1, n_tokens=2 ** 31 - 1, channels=8192), INVALID, "launch grid"),
    (dict(x_stride=56), INVALID, "x_stride"), (dict(x_stride=68), INVALID, "x_stride"),
    (dict(dtype=0, x_stride=66), INVALID, "x_stride"), (dict(out_stride=-64), INVALID, "out_stride"),
    (dict(out_stride=2 ** 24), INVALID, "out_stride"),
], ids=str)
def test_conv_descriptions(L, kw, code, text):
    for rc in conv_calls(L, conv_desc(**kw)):
        refused(L, rc, code, text)


@pytest.mark.parametrize("kw,code,text", SEQS + [
    (dict(dtype=4), INVALID, "dtype"), (dict(channels=72), INVALID, "8 n_groups"), (dict(channels=0), INVALID, "channels"),
    (dict(n_groups=0), INVALID, "n_groups"), (dict(n_groups=-2), INVALID, "n_groups"), (dict(d_state=4), UNSUPPORTED, "d_state"),
    (dict(d_state=128), UNSUPPORTED, "d_state"), (dict(d_state=24), UNSUPPORTED, "d_state"),
    (dict(softplus=2), INVALID, "softplus"), (dict(n_seqs=1, n_tokens=2 ** 31 - 1), INVALID, "launch grid"),
    (dict(x_stride=56), INVALID, "x_stride"), (dict(dt_stride=68), INVALID, "dt_stride"), (dict(z_stride=4), INVALID, "z_stride"),
    (dict(out_stride=1), INVALID, "out_stride"), (dict(b_stride=24), INVALID, "b_stride"), (dict(c_stride=36), INVALID, "c_stride"),
], ids=str)
def test_scan_descriptions(L, kw, code, text):
    for rc in scan_calls(L, scan_desc(**kw)):
        refused(L, rc, code, text)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=3), INVALID, "dtype"), (dict(param_dtype=4), INVALID, "param_dtype"), (dict(out_dtype=0), INVALID, "out_dtype"),
    (dict(out_dtype=5), INVALID, "out_dtype"), (dict(d=12), UNSUPPORTED, "multiple of 8"), (dict(d=0), UNSUPPORTED, "multiple of 8"),
    (dict(d=32776), UNSUPPORTED, "32768"), (dict(n_rows=-1), INVALID, "n_rows"), (dict(n_heads=0), INVALID, "n_heads"),
    (dict(n_rows=2 ** 30), INVALID, "below 2^31"), (dict(n_rows=2 ** 24, d=1024), INVALID, "launch grid"),
    (dict(n_rows=2 ** 22, n_heads=1, d=16384), INVALID, "launch grid"),
    (dict(gate=0), INVALID, "gate"), (dict(group=128), INVALID, "group"), (dict(eps=-1e-6), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(eps=float("inf")), INVALID, "eps"), (dict(x_stride=8), INVALID, "x_stride"),
    (dict(residual_stride=260), INVALID, "residual_stride"), (dict(z_stride=-256), INVALID, "z_stride"),
    (dict(out_stride=2 ** 24), INVALID, "out_stride"),
], ids=str)
def test_norm_descriptions(L, kw, code, text):
    for rc in norm_calls(L, norm_desc(**kw)):
        refused(L, rc, code, text)


def test_norm_eight_bits(L):
    q, p = V(AT), lambda **kw: ctypes.byref(norm_desc(**kw))
    for group in (32, 64 + 1, 256, -64):
        refused(L, L.stepq_norm_forward(p(out_dtype=3, group=group), *[q] * 7, None), INVALID, "group")
    refused(L, L.stepq_norm_forward(p(out_dtype=4, d=64, group=128), *[q] * 7, None), INVALID, "group")
    refused(L, L.stepq_norm_forward(p(out_dtype=3, out_stride=260), *[q] * 7, None), INVALID, "out_stride")
    refused(L, L.stepq_norm_forward(p(out_dtype=3), q, q, q, q, q, None, q, None), INVALID, "scale must be non-NULL")
    refused(L, L.stepq_norm_backward(p(out_dtype=3), *[q] * 9, 1 << 40, None), INVALID, "the gradient's out_dtype")


def _pointers(L, call, names, needed, loose=()):
    """NULL (where it is needed) and misaligned pointers, one at a time."""
    for i, name in enumerate(names):
        args = MANY[:len(names)]
        if name in needed:
            args[i] = None
            refused(L, call(args), INVALID, f"{name} must be non-NULL")
        args[i] = V(AT * 40 + 2)
        refused(L, call(args), INVALID, f"{name} must be {4 if name in loose else 16}-byte aligned")


def test_pointers(L):
    c, s, n = ctypes.byref(conv_desc()), ctypes.byref(scan_desc()), ctypes.byref(norm_desc())
    big = (V(AT), 1 << 40, None)
    _pointers(L, lambda p: L.stepq_conv_forward(c, *p[:5], 0, None, p[5], None), ["x", "weight", "bias", "S_in", "S_out", "out"],
              {"x", "weight", "out"})
    _pointers(L, lambda p: L.stepq_conv_backward(c, *p, *big),
              ["x", "weight", "bias", "S_in", "d_out", "dS_out", "dx", "dweight", "dbias", "dS_in"],
              {"x", "weight", "d_out", "dx", "dweight"}, {"dbias"})
    _pointers(L, lambda p: L.stepq_scan_forward(s, *p[:10], 0, None, p[10], *big),
              ["x", "dt", "A", "B", "C", "D", "dt_bias", "z", "S_in", "S_out", "out (d_out)"],
              {"x", "dt", "A", "B", "C", "out (d_out)"}, {"D", "dt_bias"})
    _pointers(L, lambda p: L.stepq_scan_backward(s, *p, *big),
              ["x", "dt", "A", "B", "C", "D", "dt_bias", "z", "S_in", "out (d_out)", "dS_out", "dx", "ddt", "dA", "dB", "dC", "dD",
               "ddt_bias", "dz", "dS_in"],
              {"x", "dt", "A", "B", "C", "out (d_out)", "dx", "ddt", "dA", "dB", "dC", "dz"}, {"D", "dt_bias", "dD", "ddt_bias"})
    _pointers(L, lambda p: L.stepq_norm_forward(n, *p[:5], None, p[5], None), ["x", "weight", "residual", "z", "out", "residual_out"],
              {"x", "out"})
    _pointers(L, lambda p: L.stepq_norm_backward(n, *p, *big),
              ["h", "weight", "z", "d_out", "d_residual", "dx", "dweight", "dz"], {"h", "d_out", "dx", "dz"}, {"dweight"})


def test_workspaces_slots_and_missing_pieces(L):
    q, n = V(AT), ctypes.c_size_t()
    for fn in (L.stepq_conv_backward_workspace, L.stepq_scan_forward_workspace, L.stepq_scan_backward_workspace,
               L.stepq_norm_backward_workspace):
        refused(L, fn(None, ctypes.byref(n)), INVALID, "desc is NULL")
    c, s, m = ctypes.byref(conv_desc()), ctypes.byref(scan_desc()), ctypes.byref(norm_desc())
    for fn, d in ((L.stepq_conv_backward_workspace, c), (L.stepq_scan_forward_workspace, s),
                  (L.stepq_scan_backward_workspace, s), (L.stepq_norm_backward_workspace, m)):
        refused(L, fn(d, None), INVALID, "bytes is NULL")
        assert fn(d, ctypes.byref(n)) == 0
    refused(L, L.stepq_conv_forward(c, *MANY[:5], 0, q, MANY[6], None), INVALID, "n_slots must be >= 1")
    refused(L, L.stepq_scan_forward(s, *MANY[:10], 0, q, *MANY[11:13], 1 << 40, None), INVALID, "n_slots must be >= 1")
    for call in (lambda w, b: L.stepq_conv_backward(c, *MANY[:10], w, b, None),
                 lambda w, b: L.stepq_scan_backward(s, *MANY[:20], w, b, None),
                 lambda w, b: L.stepq_norm_backward(m, *MANY[:8], w, b, None)):
        refused(L, call(q, 16), INVALID, "workspace of 16 bytes")
        refused(L, call(None, 1 << 40), INVALID, "workspace is NULL")
        refused(L, call(V(AT + 128), 1 << 40), INVALID, "workspace must be 256-byte aligned")


def test_outputs_in_the_place_of_inputs(L):
    c, s = ctypes.byref(conv_desc()), ctypes.byref(scan_desc())

    def same(a, b, n):
        p = list(MANY[:n])
        p[b] = p[a]
        return p
    p = same(0, 5, 6)
    refused(L, L.stepq_conv_forward(c, *p[:5], 0, None, p[5], None), INVALID, "out must not overlap x")
    names = ["x", "weight", "bias", "S_in", "d_out", "dS_out", "dx", "dweight", "dbias", "dS_in"]
    for a, b in (("x", "dx"), ("d_out", "dx"), ("S_in", "dS_in"), ("dS_out", "dS_in")):
        p = same(names.index(a), names.index(b), 11)
        refused(L, L.stepq_conv_backward(c, *p, 1 << 40, None), INVALID, f"{b} must not overlap {a}")
    for a, name in ((0, "x"), (1, "dt"), (7, "z")):
        p = same(a, 10, 12)
        refused(L, L.stepq_scan_forward(s, *p[:10], 0, None, *p[10:], 1 << 40, None), INVALID, f"out must not overlap {name}")
    names = ["x", "dt", "A", "B", "C", "D", "dt_bias", "z", "S_in", "d_out", "dS_out", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias",
             "dz", "dS_in"]
    for a, b in (("x", "dx"), ("d_out", "ddt"), ("z", "dz"), ("dx", "dz"), ("dt", "ddt"), ("S_in", "dS_in"), ("dS_out", "dS_in")):
        p = same(names.index(a), names.index(b), 21)
        refused(L, L.stepq_scan_backward(s, *p, 1 << 40, None), INVALID, f"{b} must not overlap {a}")


def test_norm_rows_in_the_place_of_others(L):
    """The norm works in place where a row of both has the same bytes, and is refused where workgroups would write
    rows that others still read."""
    def norm(kw, a, b):
        names = ["x", "weight", "residual", "z", "out", "scale", "residual_out"]
        p = list(MANY[:7])
        p[names.index(b)] = p[names.index(a)]
        return L.stepq_norm_forward(ctypes.byref(norm_desc(**kw)), *p, None)

    for a in ("x", "residual", "z"):
        for b, own in (("out", "out"), ("residual_out", "residual")):
            if (a, b) != ("residual", "residual_out"):
                refused(L, norm({f"{own}_stride": 512}, a, b), INVALID, f"{b} must not overlap {a}")
                refused(L, norm({f"{a}_stride": 512}, a, b), INVALID, f"{b} must not overlap {a}")
            if not torch.cuda.is_available():
                refused(L, norm({}, a, b), INVALID, "device 0 not available")
                refused(L, norm({f"{own}_stride": 512, f"{a}_stride": 512}, a, b), INVALID, "device 0 not available")
        refused(L, norm(dict(out_dtype=4), a, "out"), INVALID, f"out must not overlap {a}")
    refused(L, norm({}, "out", "residual_out"), INVALID, "residual_out must not overlap out")
    names = ["h", "weight", "z", "d_out", "d_residual", "dx", "dweight", "dz"]
    strides = dict(h="x_stride", z="z_stride", d_out="out_stride", d_residual="residual_stride")
    for b in ("dx", "dz"):
        for a, st in strides.items():
            p = list(MANY[:9])
            p[names.index(b)] = p[names.index(a)]
            refused(L, L.stepq_norm_backward(ctypes.byref(norm_desc(**{st: 512})), *p, 1 << 40, None), INVALID,
                    f"{b} must not overlap {a}")
            if not torch.cuda.is_available():
                refused(L, L.stepq_norm_backward(ctypes.byref(norm_desc()), *p, 1 << 40, None), INVALID,
                        "device 0 not available")
    p = list(MANY[:9])
    p[names.index("dz")] = p[names.index("dx")]
    refused(L, L.stepq_norm_backward(ctypes.byref(norm_desc()), *p, 1 << 40, None), INVALID, "dx must not overlap dz")


def test_good_calls_fail_only_at_the_device(L):
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    n = ctypes.c_size_t()
    for calls, d in ((conv_calls, conv_desc()), (scan_calls, scan_desc()), (norm_calls, norm_desc())):
        for rc in calls(L, d):
            if rc:
                refused(L, rc, INVALID, "device 0 not available")


def test_python_refusals():
    from quantized_delta_rule_amd import conv, norm, scan
    x, w = torch.zeros(4, 64), torch.zeros(64, 4)
    B = torch.zeros(4, 1, 16)
    for call in (lambda v: conv.forward(v, w, x), lambda v: conv.backward(v, w, x, x, w),
                 lambda v: scan.forward(v, x, x, B, B, x), lambda v: scan.backward(v, x, x, B, B, x, x, x, x, B, B),
                 lambda v: norm.forward(v, None, x), lambda v: norm.backward(v, None, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call(x)
        with pytest.raises(TypeError, match="must be a torch tensor"):
            call(None)
        with pytest.raises(ValueError, match="dimensions"):
            call(x[0])
