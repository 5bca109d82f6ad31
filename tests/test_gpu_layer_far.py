"""The scan's gradient of rows past 4 GiB: the last sequence's gradients are what they are by itself."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layerlib as R  # noqa: E402
from layerlib import BF16, HALF  # noqa: E402


def test_gradient_past_4_gib():
    from quantized_delta_rule_amd import scan
    T, C, n, tail = 270_000, 8192, 16, 512
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(*shape):
        x = torch.empty(T, *shape, dtype=BF16, device="cuda")
        x.copy_(torch.randn(1000, *shape, generator=g, device="cuda").to(BF16).repeat(270, *[1] * len(shape)))
        return x
    x, z, dy, B, Cm = rows(C), rows(C), rows(C), rows(1, n), rows(1, n)
    dt = torch.full_like(x, -3.0)
    A = -1 - torch.rand(C, n, generator=g, device="cuda")

    def back(first, cu):
        part = [v[first:] for v in (x, dt, B, Cm, z, dy)]
        to = {m: torch.full_like(v, 7.0) for m, v in zip(("x", "dt", "B", "C", "z"), part)}
        dA = torch.empty_like(A)
        scan.backward(part[0], part[1], A, part[2], part[3], part[5], to["x"], to["dt"], dA, to["B"], to["C"], z=part[4], dz=to["z"],
                      cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        assert bool(torch.isfinite(dA).all()) and float(dA.abs().max()) > 0
        return to
    alone = back(T - tail, [0, tail])
    whole = back(0, [0, 40, T - tail, T])
    for m, v in alone.items():
        assert R.rel(whole[m][T - tail:], v) <= 2 * HALF[BF16], m
    few = {m: v[:40].clone() for m, v in whole.items()}
    del whole
    x, dt, B, Cm, z, dy = (v[:40].contiguous() for v in (x, dt, B, Cm, z, dy))
    alone = back(0, [0, 40])
    for m, v in alone.items():
        assert R.rel(few[m], v) <= 2 * HALF[BF16], m
