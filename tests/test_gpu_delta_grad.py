"""The gradient of the gated delta rule on the GPU, against the adjoint recursion token by token in binary64,
and that recursion against differences (CPU part of the check, in binary64).

Tolerances (relative 2-norms), as for the forward pass: 12 * 2^-22 + 4 * 12 u a chain of four products,
times 2 for rows' largest elements against their norm.  The gradients chain the states before a chunk (one such
chain), the states' gradients (one more, from Y) and the products of both: three chains, 3.6e-5.  The gates'
and strengths' gradients are sums over 128 x 128 state entries and over pairs of tokens whose terms cancel
to about a fifth of their norm: times 5 would bound them, and the same 3.6e-5 is asked because rounding errors
of the terms are independent.  16-bit gradients add half a step of their type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TOL = 3.6e-5
OUT = {F32: TOL, BF16: 2.0 ** -8 + TOL, F16: 2.0 ** -11 + TOL}


@pytest.fixture(scope="module")
def delta():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from quantized_delta_rule_amd import delta
    return delta


def _backward(delta, x, cu, state=True, **kw):
    g = {m: t.cuda() for m, t in x.items()}
    nan = lambda t, dt=None: torch.full(t.shape, float("nan"), dtype=dt or t.dtype, device="cuda")  # noqa: E731
    r = dict(dq=nan(g["q"]), dk=nan(g["k"]), dv=nan(g["v"]), dalpha=nan(g["alpha"]), dbeta=nan(g["beta"]),
             dS=nan(g["S"]))
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    delta.backward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["do"], r["dq"], r["dk"], r["dv"], r["dalpha"],
                   r["dbeta"], state_in=g["S"] if state else None, d_state_out=g["dS"] if state else None,
                   d_state_in=r["dS"], cu_seqlens=c, **kw)
    return {m: t.cpu() for m, t in r.items()}


def _want(x, cu, state=True):
    S, dS = (x["S"], x["dS"]) if state else (torch.zeros_like(x["S"]), torch.zeros_like(x["dS"]))
    return R.gradient(x["q"], x["k"], x["v"], x["alpha"], x["beta"], S, cu, x["do"], dS)


def _check(got, want, cu, dtype):
    a, b = cu[0], cu[-1]
    for m in ("dq", "dk", "dv", "dalpha", "dbeta"):
        assert torch.isnan(got[m][:a]).all() and torch.isnan(got[m][b:]).all(), m
        e = R.rel(got[m][a:b], want[m][a:b])
        assert e <= (OUT[dtype] if m in ("dq", "dk", "dv") else TOL), (m, e)
    assert R.rel(got["dS"], want["dS"]) <= TOL, R.rel(got["dS"], want["dS"])


def test_reference_gradient_against_differences():
    """The adjoint recursion itself: central differences of <out, do> + <S1, dS1> in binary64."""
    cu = [0, 5, 9]
    x = {m: t.double() for m, t in R.inputs(2, 9, 1, 2, 8, 2, F32, gates="any").items()}
    g = R.gradient(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu, x["do"], x["dS"])

    def loss(y):
        out, S = R.run(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["S"], cu)
        return float((out * x["do"]).sum() + (S * x["dS"]).sum())

    names = dict(q="dq", k="dk", v="dv", alpha="dalpha", beta="dbeta", S="dS")
    gen = torch.Generator().manual_seed(0)
    for m, dm in names.items():
        for _ in range(4):
            d = torch.randn(x[m].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            num = (loss({**x, m: x[m] + h * d}) - loss({**x, m: x[m] - h * d})) / (2 * h)
            assert abs(num - float((g[dm] * d).sum())) <= 1e-7 * (1 + abs(num)), m


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[1], [64], [65], [130, 0, 1, 40], [3, 150]], ids=str)
def test_gradient(delta, d, dtype, lens):
    cu = R.offsets(lens, first=1)
    x = R.inputs(21 + cu[-1], cu[-1] + 2, 2, 6, d, len(lens), dtype)
    _check(_backward(delta, x, cu), _want(x, cu), cu, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (1, 4)])
def test_gradient_heads_without_states(delta, heads):
    cu = [0, 70]
    x = R.inputs(31, 70, heads[0], heads[1], 128, 1, F32)
    _check(_backward(delta, x, cu, state=False), _want(x, cu, False), cu, F32)


@pytest.mark.gpu
def test_gradient_of_gates_of_any_value(delta):
    cu = [0, 100, 130]
    x = R.inputs(41, 130, 1, 2, 128, 2, F32, gates="any")
    _check(_backward(delta, x, cu), _want(x, cu), cu, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-20, 1e-8, 1e8])
def test_gradients_of_any_size(delta, scale):
    """Small and large output gradients with none behind the last token; and in a chunk before a closed
    gate, with others of another size behind it."""
    cu = [0, 200]
    x = R.inputs(23, 200, 2, 2, 128, 1, F32)
    x["do"], x["dS"] = x["do"] * scale, torch.zeros_like(x["dS"])
    _check(_backward(delta, x, cu), _want(x, cu), cu, F32)
    x["do"][64:] /= scale
    x["alpha"][64] = 0.0
    got, want = _backward(delta, x, cu), _want(x, cu)
    for m in ("dq", "dk", "dv"):
        assert R.rel(got[m][:64], want[m][:64]) <= TOL and R.rel(got[m][64:], want[m][64:]) <= TOL, m
    assert R.rel(got["dS"], want["dS"]) <= TOL
