"""Sequences that remember: first states, and gradients of last states, of ordinary size (column maxima 1 to 100)
under gates near one, so that what a chunk starts from is still there chunks later, against the token-by-token
recurrence in binary64.

Tolerances as in test_gpu_delta.py and test_gpu_delta_grad.py (relative 2-norms).  The update K^T diag(L) W of a
state column is the one operand without a scale of its own: it is written in the state's units.  A term
y K has y as two binary16 planes, off by at most max(2^-22 |y|, 2^-25) units, times K's planes below 2^12: 2^-13
units a token, where the column (or what its gates leave of it) is at least 2^10 units: 2^-23 of its largest.  64
tokens that err independently, on K's elements of a third of its largest, uniformly (3^-0.5): 8 / 3 / 3^0.5 * 2^-23 =
2^-22.4, one of the 12 * 2^-22 that the tolerances count for a chain.  Errors of chunks before add up as
independent ones while gates of one keep them and the delta rule shrinks them: ten chunks are sqrt(10) * 2^-22.4 =
5.7e-7 here, well inside.  16-bit outputs add half a step of their type."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402
from test_gpu_delta import BF16, F16, F32, OUT, STATE, _forward, delta  # noqa: E402,F401
from test_gpu_delta_grad import TOL, _backward, _check, _want  # noqa: E402

# 1 - gate: up to 0.2 as a layer forgets, 0.02 and 0.002 as it remembers, exactly none
FORGET = [0.2, 0.02, 0.002, 0.0]


def _inputs(seed, cu, K, H, d, dtype, forget, size):
    x = R.inputs(seed, cu[-1], K, H, d, len(cu) - 1, dtype)
    g = torch.Generator().manual_seed(seed + 1)
    x["alpha"] = 1.0 - forget * torch.rand(x["alpha"].shape, generator=g)
    for m in ("S", "dS"):
        x[m] *= size / 0.3  # N(0, size)
    return x


@pytest.mark.parametrize("size", [0.5, 1.0, 4.0, 30.0])
@pytest.mark.parametrize("forget", FORGET)
@pytest.mark.parametrize("d,dtype", [(128, F32), (64, F32), (128, BF16)], ids=str)
def test_states_that_last(delta, d, dtype, forget, size):  # noqa: F811
    cu = R.offsets([64, 640, 17, 130])
    x = _inputs(61, cu, 2, 2, d, dtype, forget, size)
    out, S = _forward(delta, x, cu, 4)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    for n in range(4):
        assert R.rel(out[cu[n]:cu[n + 1]], want[cu[n]:cu[n + 1]]) <= OUT[dtype], n
        assert R.rel(S[n], wantS[n]) <= STATE, n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("loud", [1e2, 1e4])
def test_a_loud_chunk_that_fades(delta, d, loud):  # noqa: F811
    """Values of another size in the first chunk, forgotten little by little: every later chunk by itself."""
    cu = [0, 700]
    x = _inputs(63, cu, 1, 2, d, F32, 0.06, 1.0)
    x["v"][:64] *= loud
    out, S = _forward(delta, x, cu, 1)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    for t in range(0, 700, 64):
        assert R.rel(out[t:t + 64], want[t:t + 64]) <= OUT[F32], t
    assert R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("size", [1.0, 4.0, 30.0])
@pytest.mark.parametrize("forget", FORGET)
@pytest.mark.parametrize("d,dtype", [(128, F32), (64, F32), (128, BF16)], ids=str)
def test_gradients_that_last(delta, d, dtype, forget, size):  # noqa: F811
    cu = R.offsets([64, 330, 17])
    x = _inputs(65, cu, 1, 2, d, dtype, forget, size)
    _check(_backward(delta, x, cu), _want(x, cu), cu, dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_a_loud_last_chunk_of_gradients(delta, d):  # noqa: F811
    cu = [0, 400]
    x = _inputs(67, cu, 1, 2, d, F32, 0.06, 1.0)
    x["do"][-64:] *= 1e2
    got, want = _backward(delta, x, cu), _want(x, cu)
    for t in range(0, 400, 64):
        for m in ("dq", "dk", "dv"):
            assert R.rel(got[m][t:t + 64], want[m][t:t + 64]) <= TOL, (m, t)
    assert R.rel(got["dS"], want["dS"]) <= TOL
