"""The layer calls' exponentials on binary32 rows, element by element against binary64: sigmoid (the convolution's SiLU, the
norm's and the scan's gates) and softplus (the scan's step).

Bounds, U = 2^-24: exp(-|v|) is right to 3 U (the hardware's exponential 2, its correction 1) and 0.05 |v| U (ln 2 rounded to
1.9e-9, times |v| / ln 2).  A sigmoid adds the sum's U, the reciprocal's 2 and a product's U, SiLU one more product: 8 U.
log(1 + e) adds 3.4 U (its series, 2e-7), the sum with max(v, 0) U, the scan's two products with one nothing: 8 U."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24


def values():
    g = torch.Generator().manual_seed(1)
    return torch.cat([160 * torch.rand(30000, generator=g) - 80, 8 * torch.randn(30000, generator=g),
                      torch.tensor([0.0, -0.0, 1e-30, -1e-30, 80.0, -80.0])]).clamp(-80, 80)


def errors(got, want, v):
    return float(((got.double().cpu() - want).abs() / want.abs() / U / (8 + 0.05 * v.double().abs())).nan_to_num(0.0).max())


def test_silu():
    from quantized_delta_rule_amd import conv
    v = values()
    x = v[:len(v) // 8 * 8].reshape(-1, 8).cuda()
    w, out = torch.tensor([[0.0, 1.0]] * 8).cuda(), torch.empty_like(x)
    conv.forward(x, w, out)  # the last of two inputs, times one
    d = x.double().cpu()
    assert errors(out, d * torch.sigmoid(d), d) <= 1


def test_gate():
    from quantized_delta_rule_amd import norm
    v = values()
    z = v[:len(v) // 8 * 8].reshape(-1, 8).cuda()
    one, out = torch.ones_like(z), torch.empty_like(z)
    norm.forward(one, None, out, eps=0.0, z=z, gate=norm.SIGMOID)  # the norm of ones is ones
    d = z.double().cpu()
    assert errors(out, torch.sigmoid(d), d) <= 1


def test_step():
    from quantized_delta_rule_amd import scan
    v = values()
    dt = v[:len(v) // 8 * 8].reshape(1, -1).cuda()
    C = dt.shape[1]
    one, A, B = torch.ones_like(dt), torch.zeros(C, 8).cuda(), torch.ones(1, 1, 8).cuda()
    out, S = torch.empty_like(dt), torch.empty(1, C, 8).cuda()
    scan.forward(one, dt, A, B, B, out, state_out=S)  # the state is the step
    d = dt.double().cpu()
    want = torch.log1p(torch.exp(-d.abs())) + d.clamp(min=0)
    assert errors(S[..., 0], want, d) <= 1
    long = dt.expand(40, C).contiguous()  # and in blocks of tokens: 40 steps of one value
    out, one, B = torch.empty_like(long), torch.ones_like(long), torch.ones(40, 1, 8).cuda()
    scan.forward(one, long, A, B, B, out, state_out=S)
    assert float((S[..., 0].double().cpu() / want / 40 - 1).abs().nan_to_num(0.0).max()) <= (8 + 0.05 * 80 + 20) * U  # 40 sums


def test_ends():
    """Infinities and NaN pass as the formulas say, in binary32 as in bfloat16."""
    from quantized_delta_rule_amd import norm, scan
    inf, nan = float("inf"), float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.tensor([[inf, -inf, nan, 0.0, 500.0, -500.0, 100.0, -200.0]], dtype=dtype).cuda()
        out = torch.empty_like(z)
        norm.forward(torch.ones_like(z), None, out, eps=0.0, z=z, gate=norm.SIGMOID)
        got = out.float().cpu()[0].tolist()
        assert got[:2] == [1.0, 0.0] and got[2] != got[2] and got[3:] == [0.5, 1.0, 0.0, 1.0, 0.0]
        A, B, S = torch.zeros(8, 8).cuda(), torch.ones(1, 1, 8, dtype=dtype).cuda(), torch.empty(1, 8, 8).cuda()
        scan.forward(torch.ones_like(z), z, A, B, B, out, state_out=S)
        got = S[0, :, 0].cpu().tolist()
        assert got[0] != got[0] and got[1] == 0 and got[2] != got[2] and got[4:] == [500.0, 0.0, 100.0, 0.0]
