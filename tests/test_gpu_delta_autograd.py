"""The sequence calls beside torch's autograd: forward() says that it records no graph where one is wanted, and is
silent inside the autograd function that a program wires from forward() and backward()."""
import warnings

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402
from test_gpu_delta import F32, OUT, delta  # noqa: E402,F401
from test_gpu_delta_grad import TOL  # noqa: E402

NAMES = ("q", "k", "v", "alpha", "beta", "S")


def _inputs():
    x = R.inputs(5, 90, 1, 2, 64, 1, F32)
    return x, {m: x[m].cuda() for m in NAMES}


@pytest.mark.parametrize("leaf", NAMES)
def test_forward_says_that_it_records_no_graph(delta, leaf):  # noqa: F811
    _, g = _inputs()
    g[leaf].requires_grad_(True)
    call = lambda out: delta.forward(*(g[m] for m in NAMES[:5]), out, state_in=g["S"])  # noqa: E731
    a, b = torch.empty_like(g["v"].detach()), torch.empty_like(g["v"].detach())
    with pytest.warns(UserWarning, match="records no graph"):
        call(a)
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        call(b)
    assert torch.equal(a, b)


def test_wired_as_an_autograd_function(delta):  # noqa: F811
    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, alpha, beta, S):
            out, S1 = torch.empty_like(v), torch.empty_like(S)
            delta.forward(q, k, v, alpha, beta, out, state_in=S, state_out=S1)
            ctx.save_for_backward(q, k, v, alpha, beta, S)
            return out, S1

        @staticmethod
        def backward(ctx, d_out, dS1):
            x = ctx.saved_tensors
            g = [torch.empty_like(t) for t in x]
            delta.backward(*x[:5], d_out.contiguous(), *g[:5], state_in=x[5], d_state_out=dS1.contiguous(),
                           d_state_in=g[5])
            return tuple(g)

    x, g = _inputs()
    leaves = [g[m].requires_grad_(True) for m in NAMES]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        out, S1 = Rule.apply(*leaves)
        got = torch.autograd.grad([out, S1], leaves, [x["do"].cuda(), x["dS"].cuda()])
    want, _ = R.run(*(x[m] for m in NAMES), [0, 90])
    assert R.rel(out.detach(), want) <= OUT[F32]
    grads = R.gradient(*(x[m] for m in NAMES), [0, 90], x["do"], x["dS"])
    for m, t in zip(("dq", "dk", "dv", "dalpha", "dbeta", "dS"), got):
        assert R.rel(t, grads[m]) <= TOL, m
