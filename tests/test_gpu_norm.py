"""The root-mean-square norm and its gradient against the plain definition in binary64.

Tolerances (relative 2-norms), U = 2^-24.  The sum of squares is a chain of at most 32 in a lane, six steps over lanes and
sixteen waves: 54 U of a sum of positive terms, 27 U of its root; square root, quotient, sum with eps and three products 8 U;
the gate 16 U (see the convolution's): under 64 U.  The gradient subtracts a mean product from each term, both with such
errors: 128 U; dweight sums rows that err independently: 128 U.  Results of 16-bit types add half a step of theirs.
Eight bits: half a step of e4m3 is 2^-4 of the value, or 2^-10 of the scale below its normal numbers (2^-6); of int8 half
the scale; 64 U of y and of the scale beside them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, F16, F32, HALF, U  # noqa: E402

FWD, BWD = 64 * U, 128 * U
SIZES = [8, 64, 72, 128, 256, 264, 512, 520, 1000, 2048, 2056, 4096, 8192, 8200, 16384, 20000, 32768]


@pytest.fixture(scope="module")
def norm():
    from quantized_delta_rule_amd import norm
    return norm


def inputs(seed, shape, dtype, params=F32):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    loud = 1 + 15.0 * (torch.rand(shape[-1], generator=g) < 0.02)
    return dict(x=(r(*shape) * loud).to(dtype), res=r(*shape).to(dtype), z=r(*shape).to(dtype),
                w=(1 + 0.1 * r(shape[-1])).to(params), dy=r(*shape).to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("d", SIZES)
def test_forward(norm, d, dtype):
    x = inputs(d, (5, d), dtype, params=dtype)
    g = {m: v.cuda() for m, v in x.items()}
    out, h = torch.empty_like(g["x"]), torch.empty_like(g["x"])
    norm.forward(g["x"], g["w"], out, eps=1e-5)
    assert R.rel(out, R.norm(x["x"], x["w"], None, None, 1e-5, False)[0]) <= FWD + HALF[dtype]
    norm.forward(g["x"], g["w"], out, residual=g["res"], residual_out=h)
    assert R.rel(out, R.norm(x["x"], x["w"], x["res"], None, 1e-6, False)[0]) <= FWD + HALF[dtype]
    assert torch.equal(h, (g["x"].float() + g["res"].float()).to(dtype))
    for gate in (norm.SILU, norm.SIGMOID):
        norm.forward(g["x"], None, out, z=g["z"], gate=gate)
        assert R.rel(out, R.norm(x["x"], None, None, x["z"], 1e-6, gate == norm.SIGMOID)[0]) <= FWD + HALF[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("d", SIZES)
def test_backward(norm, d, dtype):
    x = inputs(d + 1, (7, d), dtype)
    g = {m: v.cuda() for m, v in x.items()}
    dx, dw, dz = torch.empty_like(g["x"]), torch.empty(d).cuda(), torch.empty_like(g["x"])
    norm.backward(g["x"], g["w"], g["dy"], dx, dw, d_residual=g["res"])
    want = R.norm(x["x"], x["w"], None, None, 1e-6, False, x["dy"], x["res"])
    assert R.rel(dx, want["x"]) <= BWD + HALF[dtype] and R.rel(dw, want["w"]) <= BWD
    for gate in (norm.SILU, norm.SIGMOID):
        norm.backward(g["x"], g["w"], g["dy"], dx, dw, z=g["z"], dz=dz, gate=gate)
        want = R.norm(x["x"], x["w"], None, x["z"], 1e-6, gate == norm.SIGMOID, x["dy"])
        assert R.rel(dx, want["x"]) <= BWD + HALF[dtype] and R.rel(dw, want["w"]) <= BWD
        assert R.rel(dz, want["z"]) <= BWD + HALF[dtype]
    norm.backward(g["x"], None, g["dy"], dx)
    assert R.rel(dx, R.norm(x["x"], None, None, None, 1e-6, False, x["dy"])["x"]) <= BWD + HALF[dtype]


@pytest.mark.parametrize("rows", [0, 1, 3, 63, 700, 5000])
@pytest.mark.parametrize("shape", [(48, 128), (5, 64), (3, 200), (1200,)], ids=str)
def test_rows_and_heads(norm, rows, shape):
    x = inputs(rows + 11, (rows,) + shape, BF16)
    g = {m: v.cuda() for m, v in x.items()}
    out = torch.empty_like(g["x"])
    norm.forward(g["x"], g["w"], out, z=g["z"])
    assert R.rel(out, R.norm(x["x"], x["w"], None, x["z"], 1e-6, False)[0]) <= FWD + HALF[BF16]
    dx, dw, dz = torch.empty_like(g["x"]), torch.empty(shape[-1]).cuda(), torch.empty_like(g["x"])
    norm.backward(g["x"], g["w"], g["dy"], dx, dw, z=g["z"], dz=dz)
    want = R.norm(x["x"], x["w"], None, x["z"], 1e-6, False, x["dy"])
    assert R.rel(dx, want["x"]) <= BWD + HALF[BF16] and R.rel(dw, want["w"]) <= BWD
    assert R.rel(dz, want["z"]) <= BWD + HALF[BF16]


def test_gradient_is_the_difference(norm):
    """As for the convolution: central differences of a scalar of the definition in binary64."""
    x = inputs(21, (6, 72), F32)
    g = {m: v.cuda() for m, v in x.items()}
    dx, dw, dz = torch.empty_like(g["x"]), torch.empty(72).cuda(), torch.empty_like(g["x"])
    norm.backward(g["x"], g["w"], g["dy"], dx, dw, z=g["z"], dz=dz)
    r = torch.Generator().manual_seed(22)
    for m, got in (("x", dx), ("w", dw), ("z", dz)):
        way = torch.randn(x[m].shape, generator=r, dtype=torch.float64)

        def at(e):
            y = dict(x, **{m: x[m].double() + e * way})
            return float((R.norm(y["x"], y["w"], None, y["z"], 1e-6, False)[0] * x["dy"]).sum())
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(float((got.double().cpu() * way).sum()) - diff) <= 1e-6 * float(got.double().cpu().norm() * way.norm()), m


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("shape,group", [((9, 64), 0), ((9, 64), 64), ((5, 3, 128), 0), ((5, 3, 128), 128), ((4, 1000), 0),
                                         ((4, 1024), 64), ((4, 640), 128), ((70, 4096), 128), ((3, 8192), 0),
                                         ((2, 20480), 128), ((2, 32768), 0)], ids=str)
def test_eight_bits(norm, shape, group, dtype, kind):
    x = inputs(31, shape, dtype)
    g = {m: v.cuda() for m, v in x.items()}
    d = shape[-1]
    x["x"][0], x["res"][0] = 0, 0   # a row of zeros
    g["x"][0], g["res"][0] = 0, 0
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.int8, device="cuda")
    scale = torch.empty(shape[:-1] + ((d // group,) if group else ()), device="cuda")
    h = torch.empty_like(g["x"])
    norm.forward(g["x"], g["w"], codes, residual=g["res"], residual_out=h, scale=scale, group=group)
    y = R.norm(x["x"], x["w"], x["res"], None, 1e-6, False)[0].unflatten(-1, (-1, group or d))
    top = y.abs().amax(-1)
    most = 448.0 if kind == "e4m3" else 127.0
    want = torch.where(top > 0, top / most, torch.ones_like(top))
    s = scale.double().cpu().reshape(want.shape)
    assert float(((s - want).abs() / want).max()) <= 2 * FWD
    c = codes.float().double().cpu().unflatten(-1, (-1, group or d))
    got = c * s[..., None]
    half = 2.0 ** -4 * y.abs() if kind == "e4m3" else 0.5 * s[..., None]
    least = 2.0 ** -10 * s[..., None] if kind == "e4m3" else 0.0
    assert bool(((got - y).abs() <= torch.maximum(half, torch.as_tensor(least).expand_as(half)) + 4 * FWD * top[..., None]).all())
    some = top > 0
    assert bool((c.abs().amax(-1)[some] == most).all())  # the largest is the largest code
    assert bool((c[~some] == 0).all()) and bool((s[~some] == 1).all())


def test_eight_bits_of_known_rows(norm):
    """Codes are h / max |h| * top whatever the norm: values that are codes come back as they are, others go to a
    neighbour at most a step away (ties may fall either way behind the norm's roundings)."""
    d = 64
    h = torch.zeros(2, d)
    h[0, :9] = torch.tensor([448.0, 208.0, -17.0, 0.0009765625, 0.0029296875, 1.0625, 1.1875, 300.0, -2.0 ** -6])
    h[1, :6] = torch.tensor([127.0, 0.5, 1.5, -2.5, 63.5, -126.0])
    for row, kind, exact in ((0, torch.float8_e4m3fn, [0, 1, 8]), (1, torch.int8, [0, 5])):
        codes, scale = torch.empty(1, d, dtype=kind, device="cuda"), torch.empty(1, device="cuda")
        norm.forward(h[row:row + 1].cuda(), None, codes, eps=0.0, scale=scale)
        got, want = codes.float().cpu()[0], h[row]
        assert bool((got[exact] == want[exact]).all()) and bool((got[9:] == 0).all())
        step = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) if row == 0 else torch.tensor(0.5)
        assert bool(((got - want).abs() <= step * (1 + 2.0 ** -18)).all())
        rms = float(torch.sqrt((h[row].double() ** 2).mean()))
        assert abs(float(scale) * rms - 1.0) <= 64 * U


def test_in_place(norm):
    x = inputs(41, (33, 4096), BF16)
    g = {m: v.cuda() for m, v in x.items()}
    out, h = torch.empty_like(g["x"]), torch.empty_like(g["x"])
    norm.forward(g["x"], g["w"], out, residual=g["res"], residual_out=h)
    a, b = g["x"].clone(), g["res"].clone()
    norm.forward(a, g["w"], a, residual=b, residual_out=b)
    assert torch.equal(a, out) and torch.equal(b, h)
    c = g["x"].clone()
    norm.forward(c, g["w"], out, residual=g["res"], residual_out=c)
    assert torch.equal(c, h) and torch.equal(a, out)


@pytest.mark.parametrize("rows,d", [(3000, 72), (1500, 520), (1100, 4096), (1100, 8192), (600, 16384), (600, 20000)])
def test_in_the_place_of_any_input(norm, rows, d):
    """The same bits, whichever rows are overwritten: more rows than workgroups, so that rows are read ahead."""
    g = {m: v.cuda() for m, v in inputs(d + 43, (rows, d), BF16).items()}
    out, h, dx, dz = (torch.empty_like(g["x"]) for _ in range(4))
    dw, dw1 = torch.empty(d).cuda(), torch.empty(d).cuda()
    norm.forward(g["x"], g["w"], out, residual=g["res"], residual_out=h, z=g["z"])
    norm.backward(h, g["w"], g["dy"], dx, dw, z=g["z"], dz=dz, d_residual=g["x"])
    for a, b in (("x", "z"), ("res", "x"), ("z", "res")):
        c = {m: g[m].clone() for m in ("x", "res", "z")}
        norm.forward(c["x"], g["w"], c[a], residual=c["res"], residual_out=c[b], z=c["z"])
        assert torch.equal(c[a], out) and torch.equal(c[b], h), (a, b)
    for a, b in (("h", "dy"), ("dy", "h"), ("z", "x"), ("x", "z")):
        c = {m: v.clone() for m, v in dict(g, h=h).items()}
        norm.backward(c["h"], g["w"], c["dy"], c[a], dw1, z=c["z"], dz=c[b], d_residual=c["x"])
        assert torch.equal(c[a], dx) and torch.equal(c[b], dz) and torch.equal(dw1, dw), (a, b)


def test_strided_rows(norm):
    wide = torch.randn(40, 3, 256).to(BF16).cuda()
    x, z = wide[:, 0, :], wide[:, 2, :]
    w = torch.randn(256).cuda()
    target = torch.zeros(40, 600, dtype=BF16).cuda()
    norm.forward(x, w, target[:, 8:264], z=z)
    out = torch.empty(40, 256, dtype=BF16).cuda()
    norm.forward(x.contiguous(), w, out, z=z.contiguous())
    assert torch.equal(target[:, 8:264], out) and float(target[:, 264:].abs().sum()) == 0
    heads = torch.randn(40, 5, 64).to(BF16).cuda()
    big = torch.randn(40, 8, 64).to(BF16).cuda()
    big[:, :5] = heads
    a, b = torch.empty_like(heads), torch.empty_like(heads)
    norm.forward(heads, None, a)
    norm.forward(big[:, :5], None, b)
    assert torch.equal(a, b)
    dy = torch.randn(40, 5, 64).to(BF16).cuda()
    da, db, wa, wb = torch.empty_like(heads), torch.empty_like(heads), torch.empty(64).cuda(), torch.empty(64).cuda()
    norm.backward(heads, None, dy, da, wa)
    norm.backward(big[:, :5], None, dy, db, wb)
    assert torch.equal(da, db) and torch.equal(wa, wb)


def test_strided_eight_bits(norm):
    """Codes into a part of wider rows (strides of eight)."""
    x = torch.randn(21, 264).to(BF16).cuda()
    a, b = torch.zeros(21, 600, dtype=torch.int8).cuda(), torch.empty(21, 264, dtype=torch.int8).cuda()
    sa, sb = torch.empty(21).cuda(), torch.empty(21).cuda()
    norm.forward(x, None, a[:, 8:272], scale=sa)
    norm.forward(x, None, b, scale=sb)
    assert torch.equal(a[:, 8:272], b) and torch.equal(sa, sb)
    assert int(a[:, :8].abs().max()) == 0 and int(a[:, 272:].abs().max()) == 0


def test_non_finite_rows_keep_to_themselves(norm):
    x = inputs(51, (6, 640), F32)
    x["x"][1, 3], x["x"][3, 7] = float("nan"), float("inf")
    for kind in (F32, torch.float8_e4m3fn, torch.int8):
        out = torch.empty(6, 640, dtype=kind, device="cuda")
        scale = None if kind == F32 else torch.empty(6, device="cuda")
        norm.forward(x["x"].cuda(), x["w"].cuda(), out, scale=scale)
        fine = [0, 2, 4, 5]
        ok = R.norm(x["x"][fine], x["w"], None, None, 1e-6, False)[0]
        if kind == F32:
            assert R.rel(out[fine], ok) <= FWD
            assert bool(torch.isnan(out[1]).all())
        else:
            assert bool(torch.isfinite(scale).all())
            v = out.float()[fine].cpu().double() * scale.cpu().double()[fine][:, None]
            assert R.rel(v, ok) <= 2.0 ** -4
            if kind == torch.int8:
                assert int(out[1].abs().max()) == 0
            else:
                assert bool(torch.isnan(out[1].float()).all())


def test_tiny_and_huge_rows(norm):
    """Squares of 1e15 and 1e-15 stay within binary32; eps rules where rows vanish; scales stay normal."""
    d = 256
    x = torch.randn(4, d, generator=torch.Generator().manual_seed(61))
    x[0] *= 1e15
    x[1] *= 1e-15
    out = torch.empty(4, d).cuda()
    norm.forward(x.cuda(), None, out, eps=0.0)
    assert R.rel(out, R.norm(x, None, None, None, 0.0, False)[0]) <= FWD
    scale = torch.empty(4, device="cuda")
    codes = torch.empty(4, d, dtype=torch.int8, device="cuda")
    norm.forward(x.cuda(), torch.full((d,), 1e-36).cuda(), codes, scale=scale)
    assert bool((scale >= 2.0 ** -126).all()) and bool(torch.isfinite(scale).all())
