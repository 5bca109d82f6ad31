"""The short causal convolution and its gradient against the plain definition in binary64.

Tolerances (relative 2-norms), U = 2^-24.  A pre-activation is W + 1 roundings; sigmoid(u) has an exponent argument
rounded at |u| < 6 (9 U on the small outputs of negative u), exp2 and the reciprocal within 2 U each, a sum and a product:
under 16 U of an output, doubled for sums that cancel: FWD = 32 U.  dx sums W such terms with its own
roundings: 64 U.  dw and db are sums over tokens: a piece of 32 tokens, four of them, then sums of those: terms
that err independently lose sqrt(n / 2) U in a chain of n, below 64 U at these lengths, and 64 U of the terms
themselves: 128 U.  Results of 16-bit types add half a step of theirs.  States are copies: equal bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, F16, F32, HALF, U  # noqa: E402

FWD, DX, DW = 32 * U, 64 * U, 128 * U


@pytest.fixture(scope="module")
def conv():
    from quantized_delta_rule_amd import conv
    return conv


def dev(v):
    return None if v is None else v.cuda()


def run(conv, x, cu, silu=True, bias=True, state=True, equal=False):
    N = len(cu) - 1
    out = torch.full_like(x["x"], 7.0).cuda()
    last = torch.empty_like(x["S"]).cuda()
    how = dict(n_seqs=N) if equal else dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    conv.forward(x["x"].cuda(), x["w"].cuda(), out, bias=dev(x["b"]) if bias else None,
                 activation=conv.SILU if silu else conv.NONE, state_in=dev(x["S"]) if state else None, state_out=last, **how)
    return out, last


CASES = [  # lengths, channels, width
    ([1], 8, 4), ([0], 64, 4), ([3], 64, 4), ([2, 0, 1, 5], 72, 4), ([37], 512, 3), ([31, 32, 33], 520, 2),
    ([64, 0, 96, 1, 2, 3], 1000, 4), ([300], 64, 4), ([1] * 70, 1032, 4), ([129, 7], 2048, 3),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("lens,C,W", CASES, ids=str)
def test_forward(conv, lens, C, W, dtype):
    cu = R.offsets(lens)
    x = R.conv_inputs(1, cu[-1], C, W, len(lens), dtype, params=dtype if C % 64 else None)
    for silu, bias, state in ((True, True, True), (False, False, False)):
        out, last = run(conv, x, cu, silu, bias, state)
        want, wl = R.conv(x["x"], x["w"], x["b"] if bias else None, x["S"] if state else None, cu, silu)
        assert R.rel(out, want) <= FWD + HALF[dtype]
        assert torch.equal(last.cpu().double(), wl)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("lens,C,W", CASES, ids=str)
def test_backward(conv, lens, C, W, dtype):
    cu = R.offsets(lens)
    x = R.conv_inputs(2, cu[-1], C, W, len(lens), dtype, params=dtype if C % 64 else None)
    g = {m: v.cuda() for m, v in x.items()}
    dx, dw, db, dS = torch.empty_like(g["x"]), torch.empty(C, W).cuda(), torch.empty(C).cuda(), torch.empty_like(g["S"])
    conv.backward(g["x"], g["w"], g["dy"], dx, dw, bias=g["b"], dbias=db, state_in=g["S"], d_state_out=g["dS"],
                  d_state_in=dS, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    _, _, want = R.conv(x["x"], x["w"], x["b"], x["S"], cu, True, x["dy"], x["dS"])
    assert R.rel(dx, want["x"]) <= DX + HALF[dtype]
    assert R.rel(dS, want["S"]) <= DX + HALF[dtype]
    assert R.rel(dw, want["w"]) <= DW
    assert R.rel(db, want["b"]) <= DW
    # without bias, activation and states; equal lengths
    if cu[-1] % len(lens) == 0:
        each = cu[-1] // len(lens)
        cu = R.offsets([each] * len(lens))
        conv.backward(g["x"], g["w"], g["dy"], dx, dw, activation=conv.NONE, n_seqs=len(lens))
        _, _, want = R.conv(x["x"], x["w"], None, None, cu, False, x["dy"])
        assert R.rel(dx, want["x"]) <= DX + HALF[dtype]
        assert R.rel(dw, want["w"]) <= DW


def test_gradient_is_the_difference(conv):
    """The directional derivative of a scalar of the definition, by central differences in binary64 (step 1e-4: the
    cubic term is below 1e-7), against the gradient's product with the direction."""
    cu = R.offsets([40, 3, 25])
    x = R.conv_inputs(3, cu[-1], 64, 4, 3, F32)
    g = {m: v.cuda() for m, v in x.items()}
    dx, dw, db, dS = torch.empty_like(g["x"]), torch.empty(64, 4).cuda(), torch.empty(64).cuda(), torch.empty_like(g["S"])
    conv.backward(g["x"], g["w"], g["dy"], dx, dw, bias=g["b"], dbias=db, state_in=g["S"], d_state_out=g["dS"],
                  d_state_in=dS, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    r = torch.Generator().manual_seed(4)
    for m, got in (("x", dx), ("w", dw), ("b", db), ("S", dS)):
        way = torch.randn(x[m].shape, generator=r, dtype=torch.float64)

        def at(e):
            y = dict(x, **{m: x[m].double() + e * way})
            out, last = R.conv(y["x"], y["w"], y["b"], y["S"], cu, True)
            return float((out * x["dy"]).sum() + (last * x["dS"]).sum())
        diff = (at(1e-4) - at(-1e-4)) / 2e-4
        scale = float(got.double().cpu().norm() * way.norm())
        assert abs(float((got.double().cpu() * way).sum()) - diff) <= 1e-6 * scale, m


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_slots_in_place_and_token_by_token(conv, dtype):
    """A prompt and then tokens one by one, states by slot and in place, give the bits of the whole prompt."""
    lens, C, W = [9, 2, 41, 1], 264, 4
    cu = R.offsets(lens)
    x = R.conv_inputs(5, cu[-1], C, W, 6, dtype)
    pool = x["S"].cuda()
    before = pool.clone()
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32).cuda()
    xs, w, b = x["x"].cuda(), x["w"].cuda(), x["b"].cuda()
    whole, last = torch.empty_like(xs), torch.empty_like(pool[:4])
    conv.forward(xs, w, whole, bias=b, state_in=before[slots.long()], state_out=last,
                 cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    out = torch.empty_like(xs)
    half = [n // 2 for n in lens]
    rows = torch.cat([torch.arange(cu[i], cu[i] + half[i]) for i in range(4)]).cuda()
    part = torch.empty_like(xs[rows])
    conv.forward(xs[rows], w, part, bias=b, state_in=pool, state_out=pool, slots=slots,
                 cu_seqlens=torch.tensor(R.offsets(half), dtype=torch.int32).cuda())
    out[rows] = part
    for k in range(max(lens)):
        some = [i for i in range(4) if half[i] + k < lens[i]]
        if not some:
            break
        at = torch.tensor([cu[i] + half[i] + k for i in some]).cuda()
        one = torch.empty_like(xs[at])
        conv.forward(xs[at], w, one, bias=b, state_in=pool, state_out=pool,
                     slots=torch.tensor([int(slots[i]) for i in some], dtype=torch.int32).cuda(), n_seqs=len(some))
        out[at] = one
    assert torch.equal(out, whole)
    assert torch.equal(pool[slots.long()], last)
    assert torch.equal(pool[[1, 3]], before[[1, 3]])


def test_gaps_bad_offsets_and_slots(conv):
    """Rows and states of no sequence are left as they were; bad offsets and slots raise their flags."""
    C = 64
    x = R.conv_inputs(6, 50, C, 4, 3, F32)
    xs, w = x["x"].cuda(), x["w"].cuda()
    out, pool = torch.full_like(xs, 3.0), x["S"].cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    conv.forward(xs, w, out, state_in=pool, state_out=pool, status=status, slots=torch.tensor([2, -1], dtype=torch.int32).cuda(),
                 cu_seqlens=torch.tensor([5, 20, 40], dtype=torch.int32).cuda())
    want, last = R.conv(x["x"], x["w"], None, x["S"][2:3], [5, 20], True)
    assert R.rel(out[5:20], want[5:20]) <= FWD
    assert bool((out[:5] == 3).all()) and bool((out[20:] == 3).all())
    assert torch.equal(pool[:2].cpu(), x["S"][:2]) and torch.equal(pool[2:].cpu().double(), last)
    assert int(status) == 0
    conv.forward(xs, w, out, state_in=pool, state_out=pool, status=status, slots=torch.tensor([3, -2], dtype=torch.int32).cuda(),
                 cu_seqlens=torch.tensor([5, 20, 40], dtype=torch.int32).cuda())
    assert int(status) == 8
    status.zero_()
    out.fill_(3.0)
    conv.forward(xs, w, out, state_out=pool, status=status, cu_seqlens=torch.tensor([0, 20, 40, 60], dtype=torch.int32).cuda())
    assert int(status) == 16
    assert bool((out[40:] == 3).all())
    dx, dw = torch.full_like(xs, 3.0), torch.empty(C, 4).cuda()
    conv.backward(xs, w, xs, dx, dw, status=status, cu_seqlens=torch.tensor([5, 20, 40], dtype=torch.int32).cuda())
    assert bool((dx[:5] == 3).all()) and bool((dx[40:] == 3).all()) and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_strided_rows(conv, dtype):
    """Columns of a wider projection, in and out."""
    cu = R.offsets([33, 20])
    x = R.conv_inputs(7, cu[-1], 72, 4, 2, dtype)
    wide, wide_out = torch.randn(53, 200).to(dtype).cuda(), torch.zeros(53, 160, dtype=dtype).cuda()
    wide[:, 64:136] = x["x"].cuda()
    off = torch.tensor(cu, dtype=torch.int32).cuda()
    a, _ = run(conv, x, cu)
    conv.forward(wide[:, 64:136], x["w"].cuda(), wide_out[:, 8:80], bias=x["b"].cuda(), state_in=x["S"].cuda(), cu_seqlens=off)
    assert torch.equal(wide_out[:, 8:80], a)
    assert float(wide_out[:, :8].abs().sum() + wide_out[:, 80:].abs().sum()) == 0


def test_non_finite_inputs_stay_in_their_window(conv):
    x = R.conv_inputs(8, 40, 64, 4, 1, F32)
    x["x"][10, 5], x["x"][20, 6], x["x"][30, 7] = float("nan"), float("inf"), -float("inf")
    out, _ = run(conv, x, [0, 40])
    bad = ~torch.isfinite(out.cpu())
    assert bool(bad[10:14, 5].all()) and int(bad[:, 5].sum()) == 4
    keep = torch.ones(64, dtype=torch.bool)
    keep[5:8] = False
    assert not bool(bad[:, keep].any())
    assert not bool(bad[:20, 6].any()) and not bool(bad[24:, 6].any())


def test_no_sequence(conv):
    x = torch.zeros(0, 64).cuda()
    w, dw = torch.ones(64, 4).cuda(), torch.ones(64, 4).cuda()
    conv.forward(x, w, torch.zeros(0, 64).cuda(), n_seqs=0)
    conv.backward(x, w, x, torch.zeros(0, 64).cuda(), dw, n_seqs=0)
    assert float(dw.abs().sum()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_long_pieces(conv, dtype):
    """Calls of so many waves that pieces are long: offsets around their ends, against shifted products in binary64."""
    lens, C, W = [31, 33, 64, 0, 65, 1, 2, 127, 4000, 129, 4100], 4096, 4
    cu = R.offsets(lens)
    x = {m: v.cuda() for m, v in R.conv_inputs(9, cu[-1], C, W, len(lens), dtype).items()}
    leaf = {m: x[m].double().requires_grad_(True) for m in ("x", "w", "b", "S")}
    outs, lasts = [], []
    for n in range(len(lens)):
        every = torch.cat([leaf["S"][n], leaf["x"][cu[n]:cu[n + 1]]])
        u = leaf["b"] + sum(leaf["w"][:, j] * every[j:j + lens[n]] for j in range(W))
        outs.append(u * torch.sigmoid(u))
        lasts.append(every[lens[n]:])
    want, wl = torch.cat(outs), torch.stack(lasts)
    grads = torch.autograd.grad([want, wl], list(leaf.values()), [x["dy"].double(), x["dS"].double()])
    off = torch.tensor(cu, dtype=torch.int32).cuda()
    out, last = torch.empty_like(x["x"]), torch.empty_like(x["S"])
    conv.forward(x["x"], x["w"], out, bias=x["b"], state_in=x["S"], state_out=last, cu_seqlens=off)
    assert R.rel(out, want) <= FWD + HALF[dtype] and torch.equal(last.double(), wl.detach())
    dx, dw, db, dS = torch.empty_like(x["x"]), torch.empty(C, W).cuda(), torch.empty(C).cuda(), torch.empty_like(x["S"])
    conv.backward(x["x"], x["w"], x["dy"], dx, dw, bias=x["b"], dbias=db, state_in=x["S"], d_state_out=x["dS"], d_state_in=dS,
                  cu_seqlens=off)
    # sums of 8,552 tokens: pieces of 64, four of them, 34 rows: the chains are no longer than the tolerance counts
    for got, g, tol in zip((dx, dw, db, dS), grads, (DX + HALF[dtype], DW, DW, DX + HALF[dtype])):
        assert R.rel(got, g) <= tol
    for n in range(len(lens)):
        assert R.rel(dx[cu[n]:cu[n + 1]], grads[0][cu[n]:cu[n + 1]]) <= DX + HALF[dtype], n
