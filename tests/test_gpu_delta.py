"""The gated delta rule over sequences on the GPU against the token-by-token recurrence in binary64.

Tolerances (relative 2-norms).  u = 2^-24; a chunked product carries its operands as pairs of binary16 under
power-of-two scales, so each operand is off by at most 2^-22 of its row's or column's largest element and
the dropped lo lo term by as much: 3 * 2^-22 a product, four products one after another (K S, T R, then P W
or K^T W, and the state they start from), and the sums' own roundings of d = 128 terms, sqrt(128) u on
average: 12 * 2^-22 + 4 * 12 u = 5.7e-6, times 2 for the rows' largest elements against their norm: 1.2e-5
bounds a binary32 result.  Token by token the roundings are binary32 alone.  A 16-bit output adds half a
step of its type (bf16 2^-9 of the power of two below, at most 2^-8 of the value; fp16 2^-11), and bf16
outputs carry single binary16 planes (2^-12 each) in their last two products: 4 * 2^-12."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
STATE = 1.2e-5
OUT = {F32: STATE, BF16: 2.0 ** -8 + 4 * 2.0 ** -12, F16: 2.0 ** -11 + STATE}


@pytest.fixture(scope="module")
def delta():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from quantized_delta_rule_amd import delta
    return delta


def _dev(x):
    return {k: v.cuda() for k, v in x.items()}


def _forward(delta, x, cu, n_seqs, **kw):
    g = _dev(x)
    out = torch.full(g["v"].shape, float("nan"), dtype=g["v"].dtype, device="cuda")
    S1 = torch.full(g["S"].shape, float("nan"), device="cuda")
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=g["S"], state_out=S1,
                  cu_seqlens=c, n_seqs=None if cu is not None else n_seqs, **kw)
    return out.cpu(), S1.cpu()


# lengths: one token, a chunk's edges, several chunks, empty sequences, rows of no sequence at both ends
LENS = [[1], [63], [64], [65], [129, 0, 1, 64], [200, 31], [17, 16, 15, 130]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gdn_sequences(delta, d, dtype, lens):
    cu = R.offsets(lens, first=2)
    T, N = cu[-1] + 3, len(lens)
    x = R.inputs(7 + T, T, 2, 6, d, N, dtype)
    out, S = _forward(delta, x, cu, N)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert torch.isnan(out[:cu[0]]).all() and torch.isnan(out[cu[-1]:]).all()
    assert R.rel(out[cu[0]:cu[-1]], want[cu[0]:cu[-1]]) <= OUT[dtype]
    assert R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("kind,order", [("gdn", 0), ("gdn", 1), ("kda", 0), ("kda", 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[1, 1, 1], [3, 0, 5]], ids=str)
def test_tokens(delta, kind, order, d, dtype, lens):
    cu = R.offsets(lens)
    x = R.inputs(3, cu[-1], 3, 3, d, len(lens), dtype, kda=kind == "kda")
    out, S = _forward(delta, x, cu, len(lens), kind=delta.KDA if kind == "kda" else delta.GDN, order=order)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu, bool(order) or kind == "gdn")
    assert R.rel(out, want) <= OUT[dtype]
    assert R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("order", [0, 1])
def test_kda_long(delta, order):
    cu = R.offsets([70, 33])
    x = R.inputs(5, cu[-1], 2, 4, 128, 2, BF16, kda=True)
    out, S = _forward(delta, x, cu, 2, kind=delta.KDA, order=order)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu, bool(order))
    assert R.rel(out, want) <= OUT[BF16] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("lens", [[150], [2, 1]], ids=str)
def test_gates_of_any_value(delta, lens):
    """Zero, one, negative, tiny and above-one gates: products of gates, never quotients."""
    cu = R.offsets(lens)
    x = R.inputs(11, cu[-1], 2, 4, 128, len(lens), F32, gates="any")
    out, S = _forward(delta, x, cu, len(lens))
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert R.rel(out, want) <= OUT[F32] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("scale", [1e-20, 1e-3, 1e4, 1e15])
def test_values_of_any_size(delta, scale):
    """The operands' power-of-two scales follow the values."""
    cu = [0, 100]
    x = R.inputs(13, 100, 2, 2, 128, 1, F32)
    x["v"], x["S"] = x["v"] * scale, x["S"] * scale
    out, S = _forward(delta, x, cu, 1)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert R.rel(out, want) <= OUT[F32] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[1100], [2700], [6000, 0, 65, 4500]], ids=str)
def test_long_sequences_cut_into_segments(delta, d, dtype, lens):
    """Few heads and many chunks: segments run at once and joined; sequences of a batch that have fewer
    chunks than segments among them.  In place, as a state that a decode loop carries."""
    cu = R.offsets(lens)
    x = R.inputs(51 + d, cu[-1], 1, 2, d, len(lens), dtype)
    g = _dev(x)
    out = torch.empty_like(g["v"])
    S = g["S"].clone()
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=S, state_out=S,
                  cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert R.rel(out, want) <= OUT[dtype] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-8, 1e15])
def test_values_of_any_size_from_the_zero_state(delta, d, scale):
    cu = [0, 200]
    x = R.inputs(15, 200, 2, 2, d, 1, F32)
    x["v"], x["S"] = x["v"] * scale, torch.zeros_like(x["S"])
    out, S = _forward(delta, x, cu, 1)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert R.rel(out, want) <= OUT[F32] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("t", [64, 128])
@pytest.mark.parametrize("gate", [0.0, 1e-30])
@pytest.mark.parametrize("scale", [1e-12, 1e-6, 1e6])
def test_values_of_another_size_behind_a_closed_gate(delta, t, gate, scale):
    """Chunks behind a closed gate owe nothing to the size of what was before it (inside a chunk a column
    has one scale); one column is zero throughout."""
    cu = [0, 250]
    x = R.inputs(19, 250, 2, 2, 128, 1, F32)
    x["alpha"][t] = gate
    x["v"][t:] *= scale
    x["v"][..., 5], x["S"][..., 5] = 0.0, 0.0
    out, S = _forward(delta, x, cu, 1)
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    assert R.rel(out[:t], want[:t]) <= OUT[F32] and R.rel(out[t:], want[t:]) <= OUT[F32]
    assert R.rel(S, wantS) <= STATE
