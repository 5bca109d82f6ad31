"""The scan's gradient against the definition's in binary64 (autograd), and against differences.

Tolerances (relative 2-norms), U = 2^-24: states and adjoints are each a chain as the forward pass is (128 U, see
test_gpu_scan.py), and a gradient is a sum of their products: 256 U; dA, dD, ddt_bias sum over tokens, dB and dC over
channels, terms that err independently: no more.  16-bit results add half a step of their type."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, F16, F32, HALF, U  # noqa: E402
from test_gpu_scan import CASES, dev, scan  # noqa: E402,F401

TOL = 256 * U
WIDE = ("A", "D", "bias", "S")


def backward(scan, x, cu, softplus=True, D=True, z=True, state=True, equal=False, fill=None, **more):  # noqa: F811
    g = {m: dev(v) for m, v in x.items()}
    N = len(cu) - 1
    got = {m: torch.empty_like(g[m]) for m in ("x", "dt", "A", "B", "C")}
    got.update({m: torch.empty_like(g[m]) for m, on in (("D", D), ("bias", g["bias"] is not None), ("z", z), ("S", state)) if on})
    if fill is not None:
        for v in got.values():
            v.fill_(fill)
    how = dict(n_seqs=N) if equal else dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    scan.backward(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], got["x"], got["dt"], got["A"], got["B"], got["C"],
                  D=g["D"] if D else None, dD=got.get("D"), dt_bias=g["bias"], ddt_bias=got.get("bias"),
                  softplus=softplus, z=g["z"] if z else None, dz=got.get("z"), state_in=g["S"] if state else None,
                  d_state_out=g["dS"] if state else None, d_state_in=got.get("S"), **how, **more)
    return got


def want(x, cu, softplus=True, D=True, z=True, state=True):
    return R.scan(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"] if D else None, x["bias"], softplus,
                  x["z"] if z else None, x["S"] if state else None, cu, x["dy"], x["dS"] if state else None)[2]


def check(got, exact, dtype):
    for m, v in got.items():
        assert R.rel(v, exact[m]) <= TOL + (0.0 if m in WIDE else HALF[dtype]), m


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("lens,ch,G,n", CASES, ids=str)
def test_backward(scan, lens, ch, G, n, dtype):  # noqa: F811
    cu = R.offsets(lens)
    for k, flags in enumerate((dict(), dict(softplus=False, D=False, z=False, state=False))):
        x = R.scan_inputs(31 + k, cu[-1], ch, G, n, len(lens), dtype, softplus=flags.get("softplus", True))
        check(backward(scan, x, cu, **flags), want(x, cu, **flags), dtype)


@pytest.mark.parametrize("T,ch,N", [(2000, 16, 1), (1500, 64, 1), (1200, 24, 3), (640, 256, 1)])
def test_long_sequences(scan, T, ch, N):  # noqa: F811
    x = R.scan_inputs(33, T, ch, 1, 16, N, F32)
    cu = R.offsets([T // N] * N)
    check(backward(scan, x, cu, equal=True), want(x, cu), F32)


@pytest.mark.parametrize("lens,ch", [([1] * 20 + [900], 1024), ([5] * 9 + [700, 0, 640], 2048)], ids=lambda x: str(x)[:16])
def test_one_long_beside_short(scan, lens, ch):  # noqa: F811
    """Enough workgroups, but one sequence many times the mean: it runs in segments."""
    x = R.scan_inputs(42, sum(lens), ch, 1, 16, len(lens), F32)
    check(backward(scan, x, R.offsets(lens)), want(x, R.offsets(lens)), F32)


def test_states_that_last(scan):  # noqa: F811
    x = R.scan_inputs(34, 1500, 32, 1, 16, 1, F32, slow=1e-3)
    check(backward(scan, x, [0, 1500]), want(x, [0, 1500]), F32)


def test_gradient_is_the_difference(scan):  # noqa: F811
    """Central differences of a scalar of the definition in binary64 (step 1e-4: the cubic term is below 1e-7)."""
    cu = R.offsets([50, 1, 23])
    x = R.scan_inputs(35, cu[-1], 32, 2, 16, 3, F32)
    got = backward(scan, x, cu)
    r = torch.Generator().manual_seed(36)
    for m, v in got.items():
        way = torch.randn(x[m].shape, generator=r, dtype=torch.float64)

        def at(e):
            y = dict(x, **{m: x[m].double() + e * way})
            out, last = R.scan(y["x"], y["dt"], y["A"], y["B"], y["C"], y["D"], y["bias"], True, y["z"], y["S"], cu)
            return float((out * x["dy"]).sum() + (last * x["dS"]).sum())
        diff = (at(1e-4) - at(-1e-4)) / 2e-4
        assert abs(float((v.double().cpu() * way).sum()) - diff) <= 1e-5 * float(v.double().cpu().norm() * way.norm()), m


def test_gaps_and_bad_offsets(scan):  # noqa: F811
    x = R.scan_inputs(37, 120, 64, 1, 16, 2, F32)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    got = backward(scan, x, [7, 50, 100], fill=3.0, status=status)
    exact = want(x, [7, 50, 100])
    for m in ("x", "dt", "B", "C", "z"):
        assert bool((got[m][:7] == 3).all()) and bool((got[m][100:] == 3).all()), m
        got[m], exact[m] = got[m][7:100], exact[m][7:100]
    check(got, exact, F32)
    assert int(status) == 0
    got = backward(scan, x, [0, 50, 130], status=status, fill=3.0)  # the second sequence is skipped
    assert int(status) == 16
    y = dict(x, S=x["S"][:1], dS=x["dS"][:1])
    exact = want(y, [0, 50])
    for m in ("A", "D", "bias"):
        assert R.rel(got[m], exact[m]) <= TOL, m
    for m in ("x", "dt", "B", "C", "z"):
        assert bool((got[m][50:] == 3).all()), m
        assert R.rel(got[m][:50], exact[m][:50]) <= TOL, m


def test_zero_steps_and_masks(scan):  # noqa: F811
    """Steps of zero: states and adjoints pass as they are; gradients stay finite where softplus is at its end."""
    x = R.scan_inputs(38, 90, 64, 1, 16, 1, F32, softplus=False)
    x["dt"][10:40] = 0.0
    check(backward(scan, x, [0, 90], softplus=False), want(x, [0, 90], softplus=False), F32)
    x = R.scan_inputs(39, 90, 64, 1, 16, 1, F32)
    x["dt"][10:40] = -float("inf")
    got = backward(scan, x, [0, 90])
    for m, v in got.items():
        assert bool(torch.isfinite(v).all()), m
    assert float(got["dt"][10:40].abs().sum()) == 0


def test_same_call_same_bits(scan):  # noqa: F811
    x = R.scan_inputs(40, 700, 200, 1, 16, 3, BF16)
    cu = [0, 400, 401, 700]
    a = backward(scan, x, cu)
    for _ in range(2):
        b = backward(scan, x, cu)
        assert all(torch.equal(a[m], b[m]) for m in a)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_strided_rows(scan, dtype):  # noqa: F811
    cu = [0, 100, 171]
    x = R.scan_inputs(41, 171, 72, 1, 16, 2, dtype)
    a = backward(scan, x, cu)
    y = dict(x)
    for m in ("x", "dt", "B", "C", "z", "dy"):
        flat = x[m].reshape(171, -1)
        w = torch.zeros(171, flat.shape[1] + 24, dtype=dtype).cuda()
        w[:, 8:8 + flat.shape[1]] = flat.cuda()
        y[m] = w[:, 8:8 + flat.shape[1]].unflatten(1, x[m].shape[1:])
    got = {m: torch.empty_like(x[m].cuda()) for m in a}
    scan.backward(y["x"], y["dt"], x["A"].cuda(), y["B"], y["C"], y["dy"], got["x"], got["dt"], got["A"], got["B"], got["C"],
                  D=x["D"].cuda(), dD=got["D"], dt_bias=x["bias"].cuda(), ddt_bias=got["bias"], z=y["z"], dz=got["z"],
                  state_in=x["S"].cuda(), d_state_out=x["dS"].cuda(), d_state_in=got["S"],
                  cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    assert all(torch.equal(a[m], got[m]) for m in a)
