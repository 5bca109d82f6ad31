"""The operators around the recurrence as a program uses them: layers of several calls, prompts and then single tokens by
slot, gradients through a whole layer, captured graphs, other streams, calls at once, rows past 4 GiB, refusals.

Tolerances (relative 2-norms) are sums of the operators' own (see their tests): U = 2^-24, a result of a 16-bit type adds
half a step of it wherever it is rounded on the way."""
import warnings

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib  # noqa: E402
import layerlib as R  # noqa: E402
from layerlib import BF16, F32, HALF, U  # noqa: E402


@pytest.fixture(scope="module")
def ops():
    from quantized_delta_rule_amd import conv, delta, norm, scan
    return conv, delta, norm, scan


def cuda(x):
    return {m: None if v is None else v.cuda() for m, v in x.items()}


def offs(cu):
    return torch.tensor(cu, dtype=torch.int32).cuda()


# ---------------------------------------------------------------------------------------------
# a gated delta rule layer: convolution over queries, keys and values together, the rule, the gated norm
# ---------------------------------------------------------------------------------------------

def delta_layer(ops, p, rows, cu, conv_state, state, slots=None):
    """One call of each operator over rows of the layer's projections; states in place."""
    conv, delta, norm, _ = ops
    K, H, d = 2, 4, 64
    x = p["x"][rows]
    u = torch.empty_like(x)
    how = dict(cu_seqlens=offs(cu), slots=slots)
    conv.forward(x, p["w"], u, state_in=conv_state, state_out=conv_state, **how)
    q, k, v = (t.unflatten(1, (-1, d)) for t in u.split([K * d, K * d, H * d], 1))
    out = torch.empty(x.shape[0], H, d, dtype=x.dtype, device="cuda")
    delta.forward(q, k, v, p["alpha"][rows], p["beta"][rows], out, state_in=state, state_out=state, **how)
    y = torch.empty_like(out)
    norm.forward(out, p["nw"], y, z=p["z"][rows])
    return y


def test_delta_layer_prompts_then_tokens(ops):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    K, H, d, lens = 2, 4, 64, [70, 3, 33]
    cu = R.offsets(lens)
    T, C = cu[-1], (2 * K + H) * d
    p = dict(x=0.25 * r(T, C), w=r(C, 4) / 2, alpha=0.9 + 0.1 * torch.rand(T, H, generator=g), beta=torch.sigmoid(r(T, H)) / 4,
             nw=1 + 0.1 * r(d), z=r(T, H, d))
    S0, c0 = 0.3 * r(5, H, d, d), r(5, 3, C) / 4
    slots = [3, 0, 4]
    # binary64
    u, last = R.conv(p["x"], p["w"], None, c0[slots], cu, True)
    q, k, v = (t.unflatten(1, (-1, d)) for t in u.split([K * d, K * d, H * d], 1))
    o, S = deltalib.run(q, k, v, p["alpha"], p["beta"], S0[slots], cu)
    want = R.norm(o, p["nw"], None, p["z"], 1e-6, False)[0]
    # prompts to half of every sequence, then token by token
    dp = cuda(p)
    state, conv_state = S0.cuda(), c0.cuda()
    got = torch.empty(T, H, d).cuda()
    half = [n // 2 for n in lens]
    sl = torch.tensor(slots, dtype=torch.int32).cuda()
    rows = torch.cat([torch.arange(cu[i], cu[i] + half[i]) for i in range(3)]).cuda()
    got[rows] = delta_layer(ops, dp, rows, R.offsets(half), conv_state, state, sl)
    for t in range(max(lens)):
        some = [i for i in range(3) if half[i] + t < lens[i]]
        if some:
            rows = torch.tensor([cu[i] + half[i] + t for i in some]).cuda()
            got[rows] = delta_layer(ops, dp, rows, list(range(len(some) + 1)), conv_state, state, sl[some].contiguous())
    # convolution 32 U, rule 12 * 2^-22 (its tests), norm 64 U; the norm divides rows of any size by theirs, and a small row carries
    # what large ones beside it lost: rows differ by some tens
    assert R.rel(state[slots], S) <= 64 * 2.0 ** -22
    assert torch.equal(conv_state[slots].cpu().double(), last)
    assert R.rel(got, want) <= 256 * 2.0 ** -22
    assert torch.equal(state[[1, 2]].cpu(), S0[[1, 2]]) and torch.equal(conv_state[[1, 2]].cpu(), c0[[1, 2]])


# ---------------------------------------------------------------------------------------------
# a selective scan block with its gradients: norm with the residual's addition, convolution, scan, gated norm
# ---------------------------------------------------------------------------------------------

def functions(ops, cu):
    conv, _, norm, scan = ops
    how = dict(cu_seqlens=offs(cu))

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, res, w):
            y, h = torch.empty_like(x), torch.empty_like(x)
            norm.forward(x, w, y, residual=res, residual_out=h)
            ctx.save_for_backward(h, w)
            return y, h

        @staticmethod
        def backward(ctx, dy, dh):
            h, w = ctx.saved_tensors
            dx, dw = torch.empty_like(h), torch.empty_like(w)
            norm.backward(h, w, dy.contiguous(), dx, dw, d_residual=dh.contiguous())
            return dx, dx, dw

    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y = torch.empty_like(x)
            conv.forward(x, w, y, bias=b, **how)
            ctx.save_for_backward(x, w, b)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, b = ctx.saved_tensors
            g = [torch.empty_like(t) for t in (x, w, b)]
            conv.backward(x, w, dy.contiguous(), g[0], g[1], bias=b, dbias=g[2], **how)
            return tuple(g)

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A, B, C, D, bias, z):
            y = torch.empty_like(x)
            scan.forward(x, dt, A, B, C, y, D=D, dt_bias=bias, z=z, **how)
            ctx.save_for_backward(x, dt, A, B, C, D, bias, z)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, dt, A, B, C, D, bias, z = t = ctx.saved_tensors
            g = [torch.empty_like(v) for v in t]
            scan.backward(x, dt, A, B, C, dy.contiguous(), *g[:5], D=D, dD=g[5], dt_bias=bias, ddt_bias=g[6], z=z, dz=g[7], **how)
            return tuple(g)
    return Norm.apply, Conv.apply, Scan.apply


def test_scan_block_and_its_gradients(ops):
    cu, ch = R.offsets([45, 1, 130]), 64
    T = cu[-1]
    s = R.scan_inputs(2, T, ch, 1, 16, 3, F32)
    c = R.conv_inputs(3, T, ch, 4, 3, F32)
    g = torch.Generator().manual_seed(4)
    leaves = dict(x=s["x"], res=torch.randn(T, ch, generator=g), nw=1 + 0.1 * torch.randn(ch, generator=g), cw=c["w"], cb=c["b"],
                  dt=s["dt"], A=s["A"], B=s["B"], C=s["C"], D=s["D"], bias=s["bias"], z=s["z"])
    dy, dh = s["dy"], torch.randn(T, ch, generator=g)
    dev = {m: v.cuda().requires_grad_(True) for m, v in leaves.items()}
    Norm, Conv, Scan = functions(ops, cu)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        y, h = Norm(dev["x"], dev["res"], dev["nw"])
        out = Scan(Conv(y, dev["cw"], dev["cb"]), *(dev[m] for m in ("dt", "A", "B", "C", "D", "bias", "z")))
        got = torch.autograd.grad([out, h], list(dev.values()), [dy.cuda(), dh.cuda()])
    # binary64: the definitions one after the other, the gradients back through each
    y64, h64 = R.norm(leaves["x"], leaves["nw"], leaves["res"], None, 1e-6, False)
    u64, _ = R.conv(y64, leaves["cw"], leaves["cb"], None, cu, True)
    o64, _, gs = R.scan(u64, *(leaves[m] for m in ("dt", "A", "B", "C", "D", "bias")), True, leaves["z"], None, cu, dy)
    _, _, gc = R.conv(y64, leaves["cw"], leaves["cb"], None, cu, True, gs["x"])
    gn = R.norm(leaves["x"], leaves["nw"], leaves["res"], None, 1e-6, False, gc["x"], dh)
    want = dict(gs, x=gn["x"], res=gn["x"], nw=gn["w"], cw=gc["w"], cb=gc["b"])
    assert R.rel(out, o64) <= (128 + 32 + 64) * U
    for (m, _), v in zip(dev.items(), got):  # scan 256 U, convolution 64 U, norm 128 U, and the inputs' own errors
        assert R.rel(v, want[m]) <= 768 * U, m


def test_eight_bits_out_of_a_block(ops):
    """A readout into the next block: the residual's addition and eight bits with scales, against the same call's own
    unquantised result."""
    _, _, norm, _ = ops
    x, r = torch.randn(33, 1536).to(BF16).cuda(), torch.randn(33, 1536).to(BF16).cuda()
    y, codes, scale = torch.empty(33, 1536, dtype=BF16).cuda(), torch.empty(33, 1536, dtype=torch.float8_e4m3fn).cuda(), torch.empty(33, 12).cuda()
    h = torch.empty_like(x)
    norm.forward(x, None, y, residual=r, residual_out=h)
    norm.forward(x, None, codes, residual=r, residual_out=r, scale=scale, group=128)
    v = codes.float().unflatten(1, (12, 128)) * scale[..., None]
    assert torch.equal(h, r)
    assert R.rel(v.flatten(1), y) <= 2.0 ** -4 + HALF[BF16]


# ---------------------------------------------------------------------------------------------
# graphs, streams, calls at once
# ---------------------------------------------------------------------------------------------

def test_captured_steps_replay(ops):
    """A decode step of all three operators in a graph: replays with eager work between them give the eager bits."""
    conv, _, norm, scan = ops
    B, ch = 9, 256
    s = cuda(R.scan_inputs(5, B, ch, 1, 16, B + 2, BF16))
    c = cuda(R.conv_inputs(6, B, ch, 4, B + 2, BF16))
    slots = torch.arange(B, dtype=torch.int32).cuda() + 1
    u, y, o = (torch.empty_like(s["x"]) for _ in range(3))
    S, cs = s["S"].clone(), c["S"].clone()

    def step(S, cs):
        conv.forward(s["x"], c["w"], u, bias=c["b"], state_in=cs, state_out=cs, slots=slots, n_seqs=B)
        scan.forward(u, s["dt"], s["A"], s["B"], s["C"], y, D=s["D"], dt_bias=s["bias"], z=s["z"], state_in=S, state_out=S,
                     slots=slots, n_seqs=B)
        norm.forward(y, None, o)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(S.clone(), cs.clone())
    side.synchronize()
    S1, cs1 = S.clone(), cs.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(S1, cs1)
    S1.copy_(S)
    cs1.copy_(cs)
    S2, cs2 = S.clone(), cs.clone()
    for k in range(4):
        s["x"].copy_(torch.randn(B, ch, generator=torch.Generator().manual_seed(k)).to(BF16))
        graph.replay()
        got = o.clone()
        torch.cuda.synchronize()
        step(S2, cs2)
        assert torch.equal(got, o) and torch.equal(S1, S2) and torch.equal(cs1, cs2), k


def test_captured_gradients_replay(ops):
    conv, _, norm, scan = ops
    cu = [0, 300, 300, 420]
    x = cuda(R.scan_inputs(7, 420, 64, 1, 16, 3, F32))
    c = cuda(R.conv_inputs(8, 420, 64, 4, 3, F32))
    off, nw = offs(cu), torch.randn(64).cuda()

    def outputs():
        return {m: torch.zeros_like(v) for m, v in dict(x=x["x"], dt=x["dt"], A=x["A"], B=x["B"], C=x["C"], D=x["D"], bias=x["bias"],
                                                        z=x["z"], cx=x["x"], cw=c["w"], cb=c["b"], nx=x["x"], nw=nw, out=x["x"]).items()}

    def run(g):
        scan.forward(x["x"], x["dt"], x["A"], x["B"], x["C"], g["out"], D=x["D"], dt_bias=x["bias"], z=x["z"], cu_seqlens=off)
        scan.backward(x["x"], x["dt"], x["A"], x["B"], x["C"], x["dy"], g["x"], g["dt"], g["A"], g["B"], g["C"], D=x["D"], dD=g["D"],
                      dt_bias=x["bias"], ddt_bias=g["bias"], z=x["z"], dz=g["z"], cu_seqlens=off)
        conv.backward(x["x"], c["w"], g["x"], g["cx"], g["cw"], bias=c["b"], dbias=g["cb"], cu_seqlens=off)
        norm.backward(x["x"], nw, g["cx"], g["nx"], g["nw"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(outputs())
    side.synchronize()
    a, b = outputs(), outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(a)
    for k in range(3):
        x["dy"].copy_(torch.randn(420, 64, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(a[m], b[m]) for m in a), k


def test_other_streams_and_calls_at_once(ops):
    conv, _, norm, scan = ops
    sets = []
    for k in range(2):
        x = cuda(R.scan_inputs(9 + k, 900, 64, 1, 16, 1, BF16))
        sets.append((x, [torch.empty_like(x["x"]), torch.empty_like(x["x"]), torch.empty_like(x["x"]), torch.empty_like(x["A"])],
                     torch.cuda.Stream()))
    w = torch.randn(64, 4).cuda()

    def run(x, o, stream):
        conv.forward(x["x"], w, o[0], stream=stream)
        scan.forward(o[0], x["dt"], x["A"], x["B"], x["C"], o[1], D=x["D"], dt_bias=x["bias"], z=x["z"], stream=stream)
        g = [torch.empty_like(x[m]) for m in ("dt", "B", "C")]
        scan.backward(o[0], x["dt"], x["A"], x["B"], x["C"], x["dy"], o[2], g[0], o[3], g[1], g[2], dt_bias=x["bias"], stream=stream)
        norm.forward(o[1], None, o[0], stream=stream)
        return g
    torch.cuda.synchronize()
    keep = [run(x, o, st) for _ in range(3) for x, o, st in sets]
    torch.cuda.synchronize()
    for x, o, _ in sets:
        got = [v.clone() for v in o]
        keep.append(run(x, o, None))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, o))


def test_given_workspaces(ops):
    """The sizes that the workspace calls tell are enough, and one byte less is refused; what lies behind is left."""
    conv, _, norm, scan = ops
    x = cuda(R.scan_inputs(11, 700, 64, 1, 16, 1, F32))
    args = [x[m] for m in ("x", "dt", "A", "B", "C")]
    out, w, dw = torch.empty_like(x["x"]), torch.randn(64, 4).cuda(), torch.empty(64, 4).cuda()
    g = [torch.empty_like(t) for t in args]
    nw = torch.empty(64).cuda()
    for need, call in (
            (scan.forward_workspace(*args, out), lambda ws: scan.forward(*args, out, workspace=ws)),
            (scan.backward_workspace(*args, x["dy"]), lambda ws: scan.backward(*args, x["dy"], *g, workspace=ws)),
            (conv.backward_workspace(x["x"], w, x["dy"]), lambda ws: conv.backward(x["x"], w, x["dy"], out, dw, workspace=ws)),
            (norm.backward_workspace(x["x"], None, x["dy"]), lambda ws: norm.backward(x["x"], None, x["dy"], out, nw, workspace=ws))):
        assert need > 0
        room = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
        call(room[:need])
        torch.cuda.synchronize()
        assert bool((room[need:] == 7).all())
        with pytest.raises(RuntimeError, match="needs"):
            call(room[:need - 1])


# ---------------------------------------------------------------------------------------------
# rows and states past 4 GiB
# ---------------------------------------------------------------------------------------------

def test_rows_past_4_gib(ops):
    """The last rows of tensors of 2.2e9 elements give what they give by themselves."""
    conv, _, norm, scan = ops
    T, C, tail = 270_000, 8192, 512
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.empty(T, C, dtype=BF16, device="cuda")
    x[:] = torch.randn(1000, C, device="cuda").to(BF16).repeat(270, 1)
    out = torch.empty_like(x)
    few, last = x[-tail:].clone(), torch.empty(tail, C, dtype=BF16, device="cuda")
    off, o1 = offs([0, T - tail, T]), offs([0, tail])
    w = torch.randn(C, 4, device="cuda")
    conv.forward(x, w, out, cu_seqlens=off)
    conv.forward(few, w, last, cu_seqlens=o1)
    assert torch.equal(out[-tail:], last)
    dx, dw = torch.empty_like(x), torch.empty(C, 4, device="cuda")
    conv.backward(x, w, x, dx, dw, cu_seqlens=off)
    conv.backward(few, w, few, last, dw, cu_seqlens=o1)
    assert torch.equal(dx[-tail:], last)
    norm.forward(x, None, out)
    norm.forward(few, None, last)
    assert torch.equal(out[-tail:], last)
    norm.backward(x, None, x, dx)
    norm.backward(few, None, few, last)
    assert torch.equal(dx[-tail:], last)
    dt = torch.full_like(x, -3.0)
    A = -1 - torch.rand(C, 16, device="cuda")
    B = torch.randn(T, 1, 16, device="cuda").to(BF16)
    scan.forward(x, dt, A, B, B, out, cu_seqlens=off)
    scan.forward(few, dt[-tail:], A, B[-tail:], B[-tail:], last, cu_seqlens=o1)
    assert R.rel(out[-tail:], last) <= 2 * HALF[BF16]


def test_states_past_4_gib(ops):
    _, _, _, scan = ops
    conv = ops[0]
    n, C = 20_000, 4096  # 5.2 GB of states
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    S = torch.zeros(n, C, 16, device="cuda")
    x = cuda(R.scan_inputs(12, 3, C, 1, 16, 3, BF16))
    S[-3:] = x["S"]
    a, b, last = torch.empty_like(x["x"]), torch.empty_like(x["x"]), torch.empty_like(x["S"])
    args = [x[m] for m in ("x", "dt", "A", "B", "C")]
    scan.forward(*args, a, dt_bias=x["bias"], state_in=S, state_out=S, slots=torch.arange(n - 3, n, dtype=torch.int32).cuda(), n_seqs=3)
    scan.forward(*args, b, dt_bias=x["bias"], state_in=x["S"], state_out=last, n_seqs=3)
    assert torch.equal(a, b) and torch.equal(S[-3:], last) and float(S[:-3].abs().sum()) == 0
    cs = torch.zeros(200_000, 3, C, dtype=BF16, device="cuda")
    w = torch.randn(C, 4, device="cuda")
    conv.forward(x["x"], w, a, state_in=cs, state_out=cs, slots=torch.arange(199_997, 200_000, dtype=torch.int32).cuda(), n_seqs=3)
    assert torch.equal(cs[-3:, 2], x["x"]) and float(cs[:-3].float().abs().sum()) == 0


# ---------------------------------------------------------------------------------------------
# refusals and warnings of the bindings
# ---------------------------------------------------------------------------------------------

def test_forward_says_that_it_records_no_graph(ops):
    conv, _, norm, scan = ops
    x = cuda(R.scan_inputs(13, 20, 64, 1, 16, 1, F32))
    w, o = torch.randn(64, 4).cuda(), torch.empty_like(x["x"])
    calls = {"conv": lambda: conv.forward(x["x"], w, o), "norm": lambda: norm.forward(x["x"], None, o),
             "scan": lambda: scan.forward(x["x"], x["dt"], x["A"], x["B"], x["C"], o)}
    for name, call in calls.items():
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call()
            x["x"].requires_grad_(True)
            with torch.no_grad():
                call()
        with pytest.warns(UserWarning, match=f"{name}.forward records no graph"):
            call()
        x["x"].requires_grad_(False)


def test_binding_refuses(ops):
    conv, _, norm, scan = ops
    x, w = torch.zeros(6, 64).cuda(), torch.zeros(64, 4).cuda()
    B, A = torch.zeros(6, 1, 16).cuda(), torch.zeros(64, 16).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for err, match, call in (
            (TypeError, "out must be", lambda: conv.forward(x, w, x.bfloat16())),
            (ValueError, r"out must be \[6, 64\]", lambda: conv.forward(x, w, x[:5])),
            (ValueError, "cuda:0", lambda: conv.forward(x, w, x.cpu())),
            (ValueError, "weight", lambda: conv.forward(x, w[0], x)),
            (ValueError, r"weight must be \[64, 4\]", lambda: conv.forward(x, w[:32], x)),
            (TypeError, "bias", lambda: conv.forward(x, w, x, bias=w[:, 0].contiguous().half())),
            (ValueError, "packed", lambda: conv.forward(x.T.contiguous().T, w, x)),
            (ValueError, "overlap", lambda: conv.forward(x[:1].expand(6, 64), w, x)),
            (ValueError, "state_in must be", lambda: conv.forward(x, w, x, state_in=torch.zeros(1, 4, 64).cuda())),
            (ValueError, "slots need", lambda: conv.forward(x, w, x, slots=i32(0))),
            (ValueError, "holds 1 sequences", lambda: conv.forward(x, w, x, cu_seqlens=i32(0, 6), n_seqs=2)),
            (TypeError, "cu_seqlens must be", lambda: conv.forward(x, w, x, cu_seqlens=i32(0, 6).long())),
            (TypeError, "dtype must be", lambda: conv.forward(x.double(), w, x)),
            (RuntimeError, "multiple of 16|x_stride", lambda: conv.forward(torch.zeros(6, 66).cuda()[:, :64], w, x)),
            (RuntimeError, "16-byte aligned", lambda: conv.forward(torch.zeros(6, 72).cuda()[:, 1:65], w, x)),
            (RuntimeError, "multiple of n_seqs", lambda: conv.forward(x, w, x, n_seqs=4)),
            (TypeError, "dx must be", lambda: conv.backward(x, w, x, x.half(), w)),
            (ValueError, "B must be", lambda: scan.forward(x, x, A, B[0], B, x)),
            (ValueError, r"C must be \[6, 1, 16\]", lambda: scan.forward(x, x, A, B, B[:5], x)),
            (TypeError, "A must be", lambda: scan.forward(x, x, None, B, B, x)),
            (ValueError, r"A must be \[64, 16\]", lambda: scan.forward(x, x, A[:32], B, B, x)),
            (RuntimeError, "d_state", lambda: scan.forward(x, x, A[:, :4].contiguous(), B[..., :4].contiguous(), B[..., :4].contiguous(), x)),
            (ValueError, "dz goes with z", lambda: scan.backward(x, x, A, B, B, x, x, x, A, B, B, z=x)),
            (TypeError, "dA must be", lambda: scan.backward(x, x, A, B, B, x, x, x, None, B, B)),
            (TypeError, "out must be", lambda: norm.forward(x, None, x.bfloat16())),
            (ValueError, "scale goes with", lambda: norm.forward(x, None, x, scale=x[:, 0].contiguous())),
            (ValueError, "scale goes with", lambda: norm.forward(x, None, x.to(torch.int8))),
            (ValueError, "scale must be", lambda: norm.forward(x, None, x.to(torch.int8), scale=torch.zeros(6, 1).cuda())),
            (ValueError, "group must divide", lambda: norm.forward(x, None, x.to(torch.int8), scale=torch.zeros(6, 1).cuda(), group=48)),
            (RuntimeError, "group must be", lambda: norm.forward(x, None, x.to(torch.int8), scale=torch.zeros(6, 2).cuda(), group=32)),
            (ValueError, "strides", lambda: norm.forward(x, None, x, residual=x, residual_out=torch.zeros(6, 72).cuda()[:, :64])),
            (ValueError, "weight must be", lambda: norm.forward(x, w[:32, 0].contiguous(), x)),
            (RuntimeError, "gate", lambda: norm.forward(x, None, x, z=x, gate=7)),
            (ValueError, "dz goes with z", lambda: norm.backward(x, None, x, x, z=x)),
            (TypeError, "dx must be", lambda: norm.backward(x, None, x, None))):
        with pytest.raises(err, match=match):
            call()
    torch.cuda.synchronize()


def test_nothing_to_do(ops):
    conv, _, norm, scan = ops
    x, w, B, A = torch.zeros(0, 64).cuda(), torch.zeros(64, 4).cuda(), torch.zeros(0, 1, 16).cuda(), torch.ones(64, 16).cuda()
    S, S1 = torch.randn(2, 64, 16).cuda(), torch.zeros(2, 64, 16).cuda()
    scan.forward(x, x, A, B, B, x, state_in=S, state_out=S1, n_seqs=2)  # no tokens: states pass
    assert torch.equal(S, S1)
    dA, dS = torch.ones(64, 16).cuda(), torch.zeros_like(S)
    scan.backward(x, x, A, B, B, x, x, x, dA, B, B, state_in=S, d_state_out=S, d_state_in=dS, n_seqs=2)
    assert float(dA.abs().sum()) == 0 and torch.equal(dS, S)
    scan.forward(x, x, A, B, B, x, n_seqs=0)
    scan.backward(x, x, A, B, B, x, x, x, dA, B, B, n_seqs=0)
    norm.forward(x, None, x)
    dw = torch.ones(64).cuda()
    norm.backward(x, None, x, x, dw)
    assert float(dw.abs().sum()) == 0
    cs, c1 = torch.randn(2, 3, 64).cuda(), torch.zeros(2, 3, 64).cuda()
    conv.forward(x, w, x, state_in=cs, state_out=c1, n_seqs=2)
    assert torch.equal(cs, c1)
