"""Row strides of the layer calls' tensors: packed rows are packed whatever kind of tensor holds them (a Parameter, a view)."""
import pytest

torch = pytest.importorskip("torch")


class Named(torch.Tensor):
    """A subclass, as programs use them."""


def kinds(t):
    wide = torch.zeros(2 * t.shape[0], *t.shape[1:], dtype=t.dtype, device=t.device)
    wide[:t.shape[0]] = t
    return {"plain": t, "parameter": torch.nn.Parameter(t.clone(), requires_grad=False), "subclass": t.clone().as_subclass(Named),
            "view": wide[:t.shape[0]]}


@pytest.mark.parametrize("shape", [(4, 64), (4, 3, 64), (4, 1, 64), (1, 64), (0, 64)], ids=str)
def test_packed_rows(shape):
    from quantized_delta_rule_amd import layer
    for kind, t in kinds(torch.zeros(shape)).items():
        assert layer.rows(t, "x", torch.float32, shape, -1) == (t.data_ptr(), 0), kind
    wide = torch.zeros(4, 96)
    assert layer.rows(wide[:, 16:80], "x", torch.float32, (4, 64), -1) == (wide.data_ptr() + 64, 96)
    assert layer.rows(torch.nn.Parameter(wide)[:, :64], "x", torch.float32, (4, 64), -1)[1] == 96


@pytest.mark.gpu
def test_residual_of_any_kind():
    """The residual may be a Parameter beside a plain residual_out, and the other way round."""
    from quantized_delta_rule_amd import norm
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(5, 256, generator=g).cuda() for _ in range(2))
    want, h = torch.empty_like(x), torch.empty_like(x)
    norm.forward(x, None, want, residual=r, residual_out=h)
    assert torch.equal(h, x + r)
    for a, left in kinds(r).items():
        for b, right in kinds(torch.zeros_like(r)).items():
            out = torch.empty_like(x)
            norm.forward(x, None, out, residual=left, residual_out=right)
            assert torch.equal(out, want) and torch.equal(right.as_subclass(torch.Tensor), h), (a, b)


def odd(t, dtype=torch.float32):
    """t's rows as a part of wider ones, 16 bytes past a multiple of 32 in every other row."""
    wide = torch.zeros(t.shape[0], t.shape[1] + 12, dtype=dtype, device=t.device)
    part = wide[:, 4:4 + t.shape[1]]
    assert (part.data_ptr() + part.stride(0) * 4) % 32 in (0, 16) and part.stride(0) * 4 % 32 == 16
    part.copy_(t)
    return part


@pytest.mark.gpu
def test_binary32_rows_aligned_to_16_bytes_only():
    from quantized_delta_rule_amd import conv, norm, scan
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, z, dy = (torch.randn(50, 520, generator=g, device="cuda") for _ in range(4))
    w, b = torch.randn(520, 4, generator=g, device="cuda"), torch.randn(520, generator=g, device="cuda")
    new = torch.empty_like
    cu = torch.tensor([0, 1, 20, 50], dtype=torch.int32, device="cuda")
    one, two = new(x), odd(x)
    conv.forward(x, w, one, bias=b, cu_seqlens=cu)
    conv.forward(odd(x), w, two, bias=b, cu_seqlens=cu)
    assert torch.equal(one, two)
    got = [(new(x), new(w), new(b)) for _ in range(2)]
    conv.backward(x, w, dy, got[0][0], got[0][1], bias=b, dbias=got[0][2], cu_seqlens=cu)
    conv.backward(odd(x), w, odd(dy), got[1][0], got[1][1], bias=b, dbias=got[1][2], cu_seqlens=cu)
    assert all(torch.equal(p, q) for p, q in zip(*got))
    h = (new(x), odd(x))
    norm.forward(x, b, one, residual=r, residual_out=h[0], z=z)
    norm.forward(odd(x), b, two, residual=odd(r), residual_out=h[1], z=odd(z))
    assert torch.equal(one, two) and torch.equal(*h)
    got = [(new(x), new(b), new(x)) for _ in range(2)]
    norm.backward(x, b, dy, got[0][0], got[0][1], z=z, dz=got[0][2], d_residual=r)
    norm.backward(odd(x), b, odd(dy), got[1][0], got[1][1], z=odd(z), dz=got[1][2], d_residual=odd(r))
    assert all(torch.equal(p, q) for p, q in zip(*got))
    A, B = -torch.rand(520, 16, generator=g, device="cuda"), torch.randn(50, 16, generator=g, device="cuda")
    scan.forward(x, z, A, B.unflatten(1, (1, 16)), B.unflatten(1, (1, 16)), one, z=r, cu_seqlens=cu)
    scan.forward(odd(x), odd(z), A, odd(B).unflatten(1, (1, 16)), odd(B).unflatten(1, (1, 16)), two, z=odd(r), cu_seqlens=cu)
    assert torch.equal(one, two)
