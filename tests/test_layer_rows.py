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
