"""The norm's eight-bit codes are the quotients y / scale, rounded to binary32 and then to the nearest code (ties to even), to
the bit: y is what the same call gives as binary32, the scale what the call writes."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

KINDS = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


@pytest.fixture(scope="module")
def norm():
    from quantized_delta_rule_amd import norm
    return norm


def codes_of(y, scale, group, kind):
    """On the CPU, whose binary32 quotient is correctly rounded."""
    v = (y.unflatten(-1, (-1, group or y.shape[-1])) / scale.reshape(*y.shape[:-1], -1, 1)).flatten(-2)
    return v.to(kind) if kind == torch.float8_e4m3fn else v.round().to(kind)


def check(norm, kind, x, w, group=0, **more):
    y, codes = torch.empty(x.shape, device="cuda"), torch.empty(x.shape, dtype=kind, device="cuda")
    scale = torch.empty(x.shape[:-1] + ((x.shape[-1] // group,) if group else ()), device="cuda")
    norm.forward(x, w, y, **more)
    norm.forward(x, w, codes, scale=scale, group=group, **more)
    top = y.cpu().unflatten(-1, (-1, group or x.shape[-1])).abs().amax(-1).reshape(scale.shape)
    least = torch.tensor(2.0 ** -126)  # of a scale
    assert torch.equal(scale.cpu(), torch.where(top > 0, torch.maximum(top / KINDS[kind], least), torch.ones_like(top)))
    want = codes_of(y.cpu(), scale.cpu(), group, kind)
    assert int((codes.cpu().view(torch.int8) != want.view(torch.int8)).sum()) == 0


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_quotients_at_ties(norm, kind):
    """Rows whose every element is half-way between two codes, but for the norm's roundings."""
    if kind == torch.int8:
        ties = torch.arange(-126, 126).float() + 0.5
    else:
        ties = torch.tensor([(8 + m + 0.5) * 2.0 ** (e - 3) for e in range(-6, 8) for m in range(8)])
        ties = torch.cat([ties, -ties])
    d = 512
    loud = 2.0 ** (8 * torch.rand(4000, 1, generator=torch.Generator().manual_seed(1)) - 4)
    row = torch.zeros(d)
    row[:len(ties)], row[-1] = ties, KINDS[kind]
    check(norm, kind, (row * loud).cuda(), None, eps=1e-5)


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("rows,d,group", [(1000, 4096, 0), (1000, 4096, 128), (400, 1000, 0), (37, 8192, 64), (9, 20480, 0)])
def test_quotients(norm, kind, rows, d, group):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, r, w = (torch.randn(*s, generator=g, device="cuda") for s in ((rows, d), (rows, d), (d,)))
    check(norm, kind, x, w, group, residual=r)
    check(norm, kind, x, None, group, z=r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("d", [64, 640, 4096])
def test_rows_with_an_infinity(norm, d, dtype):
    """1 / sqrt(inf) is zero: so are the finite columns, and the infinite ones NaN (zero in int8); scales are one."""
    x, w = torch.randn(5, d, generator=torch.Generator().manual_seed(3)).to(dtype).cuda(), torch.ones(d).cuda()
    x[1, 7], x[3, 0], x[3, d - 1] = float("inf"), -float("inf"), float("inf")
    at = {1: [7], 3: [0, d - 1]}
    for kind in (dtype, torch.float8_e4m3fn, torch.int8):
        out, scale = torch.empty(5, d, dtype=kind, device="cuda"), None if kind == dtype else torch.empty(5, device="cuda")
        norm.forward(x, w, out, scale=scale)
        got = out.float().cpu()
        for row, cols in at.items():
            assert scale is None or float(scale[row]) == 1.0
            bad = torch.zeros(d, dtype=torch.bool)
            bad[cols] = True
            assert bool((got[row][~bad] == 0).all())
            assert bool((got[row][bad] == 0).all() if kind == torch.int8 else torch.isnan(got[row][bad]).all())
        assert bool(torch.isfinite(got[[0, 2, 4]]).all()) and bool((got[[0, 2, 4]].abs().amax(-1) > 0).all())


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_quotients_by_scales_of_every_size(norm, kind):
    """Rows whose scales go from the smallest normal binary32 to its largest, and an infinite one."""
    d = 512
    x = torch.randn(2000, d, generator=torch.Generator().manual_seed(4)).cuda()
    w = torch.ones(d, device="cuda")
    for power in (-126, -120, -100, -95, -91, -88, -60, 60, 100, 118):
        check(norm, kind, x, w * 2.0 ** power)
    w[5] = float("inf")  # finite values over an infinite scale are zero, infinite ones NaN (zero in int8)
    codes, scale = torch.empty(2000, d, dtype=kind, device="cuda"), torch.empty(2000, device="cuda")
    norm.forward(x, w, codes, scale=scale)
    got = codes.float().cpu()
    assert bool(torch.isinf(scale).all()) and float(got[:, :5].abs().max()) == 0 and float(got[:, 6:].abs().max()) == 0
    assert bool((got[:, 5] == 0).all() if kind == torch.int8 else torch.isnan(got[:, 5]).all())
