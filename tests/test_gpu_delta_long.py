"""The forms that large calls take, on states that last: sequences cut into segments whose first states matter to
their outputs, and ragged batches of many heads (eight waves a state, longest sequences first), each against
the token-by-token recurrence in binary64 and, where only the batch differs, bit for bit against the same
sequences alone.

Tolerances as in test_gpu_delta.py and test_gpu_delta_grad.py.  The state behind a segment is M S + N: M's columns
are states that begin as unit vectors, each off by at most STATE of its norm of about one, so M S is off by
STATE of S a segment, independently from one segment to the next: sqrt(p) STATE more in front of segment p."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402
from test_gpu_delta import BF16, F16, F32, OUT, STATE, _forward, delta  # noqa: E402,F401
from test_gpu_delta_grad import TOL, _backward  # noqa: E402
from test_gpu_delta_grad import OUT as GRAD_OUT  # noqa: E402


def _segments(T, N, H):
    """Segments of a sequence: 256 / pairs, at most 16 and of four chunks of an average sequence or more."""
    pairs, chunks = N * H, T // (64 * N)
    return 1 if pairs > 32 or chunks < 40 else min(16, 256 // pairs, chunks // 4)


def _heads(x, heads, grp):
    """The inputs of these value heads, each with its key head."""
    y = {m: x[m][:, [h // grp for h in heads]] for m in ("q", "k")}
    return {**{m: t[:, heads] for m, t in x.items() if m not in y}, **y}


# (lengths, key heads, value heads, d); the last one with more than 128 passes over states, eight waves each
CUT = [([2700], 1, 2, 64), ([2700], 1, 2, 128), ([6000, 0, 65, 4500], 1, 2, 64), ([4096], 8, 16, 128)]


@pytest.mark.parametrize("lens,K,H,d", CUT, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("forget", [1e-4, 0.0])
def test_segments_start_from_states_that_matter(delta, lens, K, H, d, dtype, forget):  # noqa: F811
    """Gates of one or almost, weak strengths: what a segment starts from is most of what it reads out."""
    cu, N = R.offsets(lens), len(lens)
    x = R.inputs(71, cu[-1], K, H, d, N, dtype)
    x["alpha"] = 1.0 - forget * torch.rand(x["alpha"].shape, generator=torch.Generator().manual_seed(72))
    x["beta"] = 0.05 * x["beta"] + 0.02
    x["S"] *= 1 / 0.3
    P = _segments(cu[-1], N, H)
    assert P > 1
    out, S = _forward(delta, x, cu, N)
    pick = list(range(H)) if H < 4 else [0, 5, H - 1]
    y = _heads(x, pick, H // K)
    want, wantS = R.run(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["S"], cu)
    out, S = out[:, pick], S[:, pick]
    for n in range(N):
        per = -(-(-(-lens[n] // 64)) // P) * 64  # tokens of a segment
        for p, t in enumerate(range(cu[n], cu[n + 1], per or 1)):
            end = min(t + per, cu[n + 1])
            assert R.rel(out[t:end], want[t:end]) <= OUT[dtype] + p ** 0.5 * STATE, (n, p)
        assert R.rel(S[n], wantS[n]) <= max(1, P) ** 0.5 * STATE, n
        if lens[n] > 1000:  # from the zero state the second segment would read out something else
            a, b = cu[n] + per, cu[n] + 2 * per
            zero, _ = R.run(*(y[m][a:b] for m in ("q", "k", "v", "alpha", "beta")), 0 * y["S"][n:n + 1], [0, per])
            assert R.rel(zero, want[a:b]) > 0.5


# an empty sequence, a single token, two of equal length; more than 256 tokens on average
MANY, K, H = [700, 0, 1, 129, 700, 300, 64, 400], 16, 48


def _many(dtype):
    cu = R.offsets(MANY)
    assert cu[-1] >= 256 * len(MANY) and len(MANY) * H > 256
    x = R.inputs(81, cu[-1], K, H, 128, len(MANY), dtype)
    x["alpha"] = 1.0 - 0.1 * torch.rand(x["alpha"].shape, generator=torch.Generator().manual_seed(82))
    return x, cu


def _alone(x, cu, n):
    a, b = cu[n], cu[n + 1]
    return {m: t[n:n + 1] if m in ("S", "dS") else t[a:b] for m, t in x.items()}


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_ragged_batches_of_many_heads(delta, dtype):  # noqa: F811
    x, cu = _many(dtype)
    out, S = _forward(delta, x, cu, len(MANY))
    heads = [0, 1, 2, 25, H - 1]
    y = _heads(x, heads, H // K)
    want, wantS = R.run(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["S"], cu)
    for n, length in enumerate(MANY):
        a, b = cu[n], cu[n + 1]
        if length:
            assert R.rel(out[a:b][:, heads], want[a:b]) <= OUT[dtype], n
        assert R.rel(S[n][heads], wantS[n]) <= STATE, n
        if length >= 16:  # in chunks alone too
            o, s = _forward(delta, _alone(x, cu, n), [0, length], 1)
            assert torch.equal(o, out[a:b]) and torch.equal(s[0], S[n]), n


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradients_of_ragged_batches_of_many_heads(delta, dtype):  # noqa: F811
    x, cu = _many(dtype)
    got = _backward(delta, x, cu)
    g = H // K
    for k in (0, K - 1):  # whole groups: value heads add up in dq and dk
        hs = list(range(g * k, g * (k + 1)))
        y = {m: t[:, k:k + 1] if m in ("q", "k") else t[:, hs] for m, t in x.items()}
        want = R.gradient(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["S"], cu, y["do"], y["dS"])
        for m, w in want.items():
            have = got[m][:, k:k + 1] if m in ("dq", "dk") else got[m][:, hs]
            tol = GRAD_OUT[dtype] if m in ("dq", "dk", "dv") else TOL
            for n, length in enumerate(MANY):
                i = n if m == "dS" else slice(cu[n], cu[n + 1])
                if length or m == "dS":
                    assert R.rel(have[i], w[i]) <= tol, (m, n)
    for n, length in enumerate(MANY):
        if length:
            one = _backward(delta, _alone(x, cu, n), [0, length])
            for m, t in one.items():
                assert torch.equal(t[0] if m == "dS" else t, got[m][n] if m == "dS" else got[m][cu[n]:cu[n + 1]]), (m, n)
