"""The selective state space scan against the plain definition in binary64.

Tolerances (relative 2-norms), U = 2^-24.  A step D is right to about 12 U (an exponential, a series, a sum), which scales
D B x and, through the argument D A, a decay: over all tokens remembered that is 12 U of the arguments' sum, about one.
A decay is rounded by 1.4 U, its argument by 2 U of less than one, the update by U: 4 U a token that err independently
over the 100 tokens that these inputs remember at most: 40 U.  n products are summed (n <= 64, in four chains and six
steps over lanes: 20 U), skip and gate 20 U more: below 128 U for outputs and states.  16-bit outputs add half a step."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, F16, F32, HALF, U  # noqa: E402

TOL = 128 * U


@pytest.fixture(scope="module")
def scan():
    from quantized_delta_rule_amd import scan
    return scan


def dev(v):
    return None if v is None else v.cuda()


def run(scan, x, cu, softplus=True, D=True, z=True, state=True, equal=False, **more):
    N = len(cu) - 1
    g = {m: dev(v) for m, v in x.items()}
    out, last = torch.full_like(g["x"], 7.0), torch.full_like(g["S"], 7.0)
    how = dict(n_seqs=N) if equal else dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    scan.forward(g["x"], g["dt"], g["A"], g["B"], g["C"], out, D=g["D"] if D else None, dt_bias=g["bias"],
                 softplus=softplus, z=g["z"] if z else None, state_in=g["S"] if state else None, state_out=last, **how, **more)
    return out, last


def want(x, cu, softplus=True, D=True, z=True, state=True):
    return R.scan(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"] if D else None, x["bias"], softplus,
                  x["z"] if z else None, x["S"] if state else None, cu)


CASES = [  # lengths, channels, groups, states
    ([1], 8, 1, 16), ([0], 16, 1, 16), ([3], 64, 1, 8), ([2, 0, 1, 5], 72, 1, 16), ([37], 256, 1, 16),
    ([31, 32, 33], 160, 4, 32), ([64, 0, 96, 1, 2, 3], 200, 1, 64), ([300], 64, 2, 16), ([1] * 70, 136, 1, 16),
    ([129, 7], 512, 1, 16), ([15, 16, 17, 47, 48, 49], 48, 2, 8), ([257], 24, 3, 64), ([700, 1, 90], 40, 1, 16),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("lens,ch,G,n", CASES, ids=str)
def test_forward(scan, lens, ch, G, n, dtype):
    cu = R.offsets(lens)
    for k, flags in enumerate((dict(), dict(softplus=False, D=False, z=False, state=False))):
        x = R.scan_inputs(1 + k, cu[-1], ch, G, n, len(lens), dtype, softplus=flags.get("softplus", True))
        out, last = run(scan, x, cu, **flags)
        o, s = want(x, cu, **flags)
        assert R.rel(out, o) <= TOL + HALF[dtype]
        for i in range(len(lens)):
            assert R.rel(last[i], s[i]) <= TOL, i


@pytest.mark.parametrize("T,ch,N", [(3000, 16, 1), (2048, 64, 1), (1200, 24, 3), (640, 512, 1), (4100, 8, 1)])
def test_long_sequences(scan, T, ch, N):
    """Few channels and long sequences; equal lengths without offsets."""
    x = R.scan_inputs(11, T, ch, 1, 16, N, F32)
    cu = R.offsets([T // N] * N)
    out, last = run(scan, x, cu, equal=True)
    o, s = want(x, cu)
    assert R.rel(out, o) <= TOL and R.rel(last, s) <= TOL
    for a in range(0, T, 500):
        assert R.rel(out[a:a + 500], o[a:a + 500]) <= TOL


MIXED = [  # single tokens beside a prompt: lengths, channels
    ([1] * 40 + [300] + [1] * 20, 64), ([2, 0, 1, 15, 16, 17, 1, 1, 1, 1, 1, 1, 1, 1, 160], 40), ([1] * 64 + [1500], 1024),
    ([3] * 30 + [1100] + [20] * 9 + [900], 512), ([1] * 9 + [700, 650], 4096),
]


@pytest.mark.parametrize("lens,ch", MIXED, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_short_and_long_in_one_call(scan, lens, ch, dtype):
    """Each sequence takes its path, long ones in segments; states by slot and in place."""
    cu = R.offsets(lens)
    x = R.scan_inputs(21, cu[-1], ch, 1, 16, len(lens), dtype)
    g = {m: dev(v) for m, v in x.items()}
    slots = torch.randperm(len(lens), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    pool = torch.empty_like(g["S"])
    pool[slots.long().cuda()] = g["S"]
    out = torch.empty_like(g["x"])
    scan.forward(g["x"], g["dt"], g["A"], g["B"], g["C"], out, D=g["D"], dt_bias=g["bias"], z=g["z"], state_in=pool, state_out=pool,
                 slots=slots.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    o, s = want(x, cu)
    last = pool[slots.long().cuda()]
    for i in range(len(lens)):
        assert R.rel(out[cu[i]:cu[i + 1]], o[cu[i]:cu[i + 1]]) <= TOL + HALF[dtype], i
        assert R.rel(last[i], s[i]) <= TOL, i


@pytest.mark.parametrize("slow", [1e-3, 1e-4])
def test_states_that_last(scan, slow):
    """Steps so small that a state remembers all of 3,000 tokens: roundings of the decays add up.  They err
    independently, 1.2 U each (rms), over 3,000 tokens: 66 U; a mean error of a tenth of U a token would be 300 U."""
    x = R.scan_inputs(12, 3000, 32, 1, 16, 1, F32, slow=slow)
    x["x"] = x["x"].abs()  # sums that grow, so that what was lost early shows
    x["B"] = x["B"].abs()
    out, last = run(scan, x, [0, 3000])
    o, s = want(x, [0, 3000])
    assert R.rel(last, s) <= TOL and R.rel(out[2000:], o[2000:]) <= TOL


def test_no_steps_leave_the_state(scan):
    """dt = -inf (softplus) and steps of zero (plain): the state keeps its bits, outputs read it."""
    for softplus in (True, False):
        x = R.scan_inputs(13, 40, 64, 1, 16, 2, F32, softplus=softplus)
        x["dt"][:20] = -float("inf") if softplus else 0.0
        out, last = run(scan, x, [0, 20, 40], softplus=softplus)
        assert torch.equal(last[0].cpu(), x["S"][0])
        o, s = want(x, [0, 20, 40], softplus=softplus) if not softplus else (None, None)
        assert bool(torch.isfinite(out).all())
        if o is not None:
            assert R.rel(out, o) <= TOL and R.rel(last, s) <= TOL


def test_extreme_steps(scan):
    """Steps so large that every decay is zero, and raw values far to both sides of softplus."""
    x = R.scan_inputs(14, 50, 64, 1, 16, 1, F32)
    x["dt"] = x["dt"] * 60
    out, last = run(scan, x, [0, 50])
    o, s = want(x, [0, 50])
    assert R.rel(out, o) <= TOL and R.rel(last, s) <= TOL


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("n,G", [(16, 1), (32, 2), (64, 1), (8, 1)])
def test_slots_in_place_and_token_by_token(scan, dtype, n, G):
    """Prompts and then tokens one by one, states by slot and in place, against the whole prompts."""
    lens, ch = [9, 2, 90, 1], 80
    cu = R.offsets(lens)
    x = R.scan_inputs(15, cu[-1], ch, G, n, 6, dtype)
    g = {m: dev(v) for m, v in x.items()}
    pool, slots = g["S"].clone(), [4, 0, 5, 2]
    out = torch.empty_like(g["x"])

    def part(rows, sl, offsets):
        some = {m: g[m][rows] for m in ("x", "dt", "B", "C", "z")}
        o = torch.empty_like(some["x"])
        how = dict(n_seqs=len(sl)) if offsets is None else dict(cu_seqlens=torch.tensor(offsets, dtype=torch.int32).cuda())
        scan.forward(some["x"], some["dt"], g["A"], some["B"], some["C"], o, D=g["D"], dt_bias=g["bias"], z=some["z"],
                     state_in=pool, state_out=pool, slots=torch.tensor(sl, dtype=torch.int32).cuda(), **how)
        out[rows] = o
    half = [m // 2 for m in lens]
    part(torch.cat([torch.arange(cu[i], cu[i] + half[i]) for i in range(4)]).cuda(), slots, R.offsets(half))
    for k in range(max(lens)):
        some = [i for i in range(4) if half[i] + k < lens[i]]
        if some:
            part(torch.tensor([cu[i] + half[i] + k for i in some]).cuda(), [slots[i] for i in some], None)
    x["S"] = x["S"][slots]
    o, s = want(x, cu)
    assert R.rel(out, o) <= TOL + HALF[dtype]
    assert R.rel(pool[slots], s) <= TOL
    assert torch.equal(pool[[1, 3]], g["S"][[1, 3]])


@pytest.mark.parametrize("T", [40, 900])
def test_gaps_bad_offsets_and_slots(scan, T):
    """Rows and states of no sequence are left as they were; bad offsets and slots raise their flags."""
    x = R.scan_inputs(16, T + 10, 64, 1, 16, 3, F32)
    g = {m: dev(v) for m, v in x.items()}
    status = torch.zeros(1, dtype=torch.int32).cuda()

    def call(cu, slots, pool):
        out = torch.full_like(g["x"], 3.0)
        status.zero_()
        scan.forward(g["x"], g["dt"], g["A"], g["B"], g["C"], out, D=g["D"], dt_bias=g["bias"], z=g["z"], state_in=pool,
                     state_out=pool, status=status, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                     slots=None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda())
        return out
    pool = g["S"].clone()
    out = call([5, T // 2, T], [2, -1], pool)
    x2 = dict(x, S=x["S"][2:3])
    o, s = want(x2, [5, T // 2])
    assert R.rel(out[5:T // 2], o[5:T // 2]) <= TOL and R.rel(pool[2:], s) <= TOL
    assert bool((out[:5] == 3).all()) and bool((out[T // 2:] == 3).all())
    assert torch.equal(pool[:2], g["S"][:2]) and int(status) == 0
    call([5, T // 2, T], [3, -2], pool)
    assert int(status) == 8
    out = call([0, 20, T, T + 20], None, g["S"].clone())
    assert int(status) == 16 and bool((out[T:] == 3).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("lens", [[33, 20], [400, 171], [1] * 53], ids=str)
def test_strided_rows(scan, dtype, lens):
    """Every row a part of wider rows: the bits of packed ones."""
    cu = R.offsets(lens)
    x = R.scan_inputs(17, cu[-1], 72, 1, 16, len(lens), dtype)
    out, last = run(scan, x, cu)
    g = {m: dev(v) for m, v in x.items()}

    def wide(t):
        flat = t.reshape(t.shape[0], -1)
        w = torch.full((t.shape[0], flat.shape[1] + 24), 5.0, dtype=dtype, device="cuda")
        w[:, 16:16 + flat.shape[1]] = flat
        return w[:, 16:16 + flat.shape[1]].unflatten(1, t.shape[1:])
    o = wide(torch.zeros_like(g["x"]))
    last2 = torch.empty_like(last)
    scan.forward(wide(g["x"]), wide(g["dt"]), g["A"], wide(g["B"]), wide(g["C"]), o, D=g["D"], dt_bias=g["bias"],
                 z=wide(g["z"]), state_in=g["S"], state_out=last2, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    assert torch.equal(o, out) and torch.equal(last2, last)


@pytest.mark.parametrize("T", [40, 600])
def test_non_finite_inputs_stay_in_their_channel(scan, T):
    x = R.scan_inputs(18, T, 64, 1, 16, 1, F32)
    x["x"][10, 5], x["dt"][20, 6], x["S"][0, 9, 3] = float("nan"), float("nan"), float("inf")
    out, last = run(scan, x, [0, T])
    bad = ~torch.isfinite(out.cpu())
    keep = torch.ones(64, dtype=torch.bool)
    keep[[5, 6, 9]] = False
    assert not bool(bad[:, keep].any())
    assert bool(bad[10:, 5].all()) and not bool(bad[:10, 5].any())
    assert bool(bad[20:, 6].all()) and not bool(bad[:20, 6].any())
    assert bool(torch.isfinite(last.cpu()[0, keep]).all())


def test_same_call_same_bits(scan):
    x = R.scan_inputs(19, 900, 256, 1, 16, 4, BF16)
    cu = [0, 500, 501, 501, 900]
    a = run(scan, x, cu)
    for _ in range(3):
        b = run(scan, x, cu)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
