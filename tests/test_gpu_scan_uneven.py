"""One long sequence beside short ones, in every proportion of sequences to channels: it runs in segments (the call asks for
their workspace), the short ones whole, forward and backward, against binary64.

Tolerances as in test_gpu_scan.py and test_gpu_scan_grad.py (128 U and 256 U, with half a step of 16-bit types): segments
join a state by one decay of their steps' sum, whose argument errs no more than its terms do."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, F32, HALF  # noqa: E402
from test_gpu_scan import TOL, dev, run, scan, want as forward_want  # noqa: E402,F401
from test_gpu_scan_grad import backward, check, want  # noqa: E402

# lengths, channels, groups, states.  Groups of 8 channels take a workgroup of 32 each: many workgroups for few channels.
UNEVEN = [
    ([1, 2600], 1024, 128, 8), ([2600, 1], 1024, 128, 8), ([1] * 7 + [2300], 1024, 128, 8), ([3] * 3 + [2300], 1024, 128, 8),
    ([1] * 60 + [1500], 128, 1, 16), ([1] * 200 + [3000], 32, 1, 16), ([1] * 100 + [3100], 32, 1, 16), ([20] * 9 + [1900], 128, 16, 32),
    ([2000, 1, 1900, 3], 512, 64, 8), ([2, 0, 1700, 40, 0, 17], 256, 32, 64),
]
ids = lambda x: str(x)[:20]  # noqa: E731


def workspace(scan, x, lens):  # noqa: F811
    g = {m: dev(v) for m, v in x.items()}
    cu = torch.tensor(R.offsets(lens), dtype=torch.int32).cuda()
    return scan.forward_workspace(*[g[m] for m in ("x", "dt", "A", "B", "C")], g["x"], cu_seqlens=cu)


@pytest.mark.parametrize("lens,ch,G,n", UNEVEN, ids=ids)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_forward(scan, lens, ch, G, n, dtype):  # noqa: F811
    cu = R.offsets(lens)
    x = R.scan_inputs(61, cu[-1], ch, G, n, len(lens), dtype)
    assert workspace(scan, x, lens) > 4 * len(lens) * ch * n  # first states of every sequence, and the segments' behind them
    out, last = run(scan, x, cu)
    o, s = forward_want(x, cu)
    for i in range(len(lens)):
        assert R.rel(out[cu[i]:cu[i + 1]], o[cu[i]:cu[i + 1]]) <= TOL + HALF[dtype], i
        assert R.rel(last[i], s[i]) <= TOL, i


@pytest.mark.parametrize("lens,ch,G,n", UNEVEN, ids=ids)
def test_backward(scan, lens, ch, G, n):  # noqa: F811
    if lens == [1, 2600]:
        lens = [1] * 3 + [2600]  # the gradient's rule counts 512 workgroups
    cu = R.offsets(lens)
    x = R.scan_inputs(62, cu[-1], ch, G, n, len(lens), F32)
    got, exact = backward(scan, x, cu), want(x, cu)
    check(got, exact, F32)
    for i in range(len(lens)):
        for m in ("x", "dt", "z"):
            assert R.rel(got[m][cu[i]:cu[i + 1]], exact[m][cu[i]:cu[i + 1]]) <= 256 * R.U, (i, m)
        assert R.rel(got["S"][i], exact["S"][i]) <= 256 * R.U, i


def test_slots_gaps_and_skipped_sequences(scan):  # noqa: F811
    """A cut sequence in place in a pool, one that is skipped, rows of none: what is not theirs is left."""
    ch, cu = 1024, [6, 7, 2407, 2450, 2450, 4650]
    x = R.scan_inputs(63, 4660, ch, 128, 8, 7, F32)
    g = {m: dev(v) for m, v in x.items()}
    slots, out, pool = [4, 0, 6, 2, -1], torch.full_like(g["x"], 3.0), g["S"].clone()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    scan.forward(g["x"], g["dt"], g["A"], g["B"], g["C"], out, D=g["D"], dt_bias=g["bias"], z=g["z"], state_in=pool, state_out=pool,
                 slots=torch.tensor(slots, dtype=torch.int32).cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                 status=status)
    o, s = forward_want(dict(x, S=x["S"][slots[:4]]), cu[:5])
    assert int(status) == 0 and R.rel(out[6:2450], o[6:2450]) <= TOL and R.rel(pool[slots[:4]], s) <= TOL
    assert torch.equal(pool[[1, 3, 5]].cpu(), x["S"][[1, 3, 5]]) and torch.equal(pool[2].cpu(), x["S"][2])
    assert bool((out[:6] == 3).all()) and bool((out[2450:] == 3).all())


def test_one_graph_for_all_lengths(scan):  # noqa: F811
    """Captured calls read their offsets at each replay: even, uneven, empty and skipped sequences, against eager calls bit for bit."""
    T, N, ch = 4000, 4, 512
    x = R.scan_inputs(64, T, ch, 64, 8, N, BF16)
    g = {m: dev(v) for m, v in x.items()}
    cu = torch.tensor([0, 1000, 2000, 3000, T], dtype=torch.int32).cuda()
    args = [g[m] for m in ("x", "dt", "A", "B", "C")]

    def call(to, cu):
        scan.forward(*args, to["out"], D=g["D"], dt_bias=g["bias"], z=g["z"], state_in=g["S"], state_out=to["S1"], cu_seqlens=cu)
        scan.backward(*args, g["dy"], to["x"], to["dt"], to["A"], to["B"], to["C"], D=g["D"], dD=to["D"], dt_bias=g["bias"],
                      ddt_bias=to["bias"], z=g["z"], dz=to["z"], state_in=g["S"], d_state_out=g["dS"], d_state_in=to["S"], cu_seqlens=cu)

    def fresh():
        return {m: torch.zeros_like(g[{"out": "x", "S1": "S"}.get(m, m)]) for m in
                ("out", "S1", "x", "dt", "A", "B", "C", "D", "bias", "z", "S")}
    kept = fresh()
    call(kept, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(kept, cu)
    for lens in ([1000] * 4, [1, 3997, 1, 1], [2000, 0, 0, 2000], [3000, 17, 983, 0], [0, 0, 0, 4000], [500, 1500, 700, 1300]):
        now = torch.tensor(R.offsets(lens), dtype=torch.int32).cuda()
        cu.copy_(now)
        for v in kept.values():
            v.zero_()
        graph.replay()
        eager = fresh()
        call(eager, now)
        torch.cuda.synchronize()
        for m, v in eager.items():
            assert torch.equal(kept[m], v), (lens, m)
    o, s = forward_want(x, R.offsets([500, 1500, 700, 1300]))
    assert R.rel(kept["out"], o) <= TOL + HALF[BF16] and R.rel(kept["S1"], s) <= TOL
