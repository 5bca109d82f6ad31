"""The convolution, the scan and the norm in binary64, for the tests of their kernels: plain loops over sequences and
tokens on the CPU, written from

    u_t = b + sum_j w_j x_{t-(W-1)+j},  y = u or u sigmoid(u)
    h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,  y_t = (C_t . h_t + D x_t) z sigmoid(z),  D_t = softplus(dt_t + bias)
    y = h / sqrt(mean h^2 + eps) w act(z),  h = x + residual

with gradients by autograd in binary64.  No code is shared with the library."""
import torch

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24                                            # half a step of binary32, relative
HALF = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}       # half a step of a result's type (binary32: in U)


def rel(x, y):
    """||x - y|| / ||y|| (the absolute norm where y is zero)."""
    x, y = x.detach().double().cpu(), y.detach().double().cpu()
    assert x.shape == y.shape, (x.shape, y.shape)
    if x.numel() == 0:
        return 0.0
    n = float(y.norm())
    return float((x - y).norm()) / (n if n else 1.0)


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _leaf(x):
    return None if x is None else x.detach().double().cpu().requires_grad_(True)


def conv(x, w, b, S, cu, silu, dy=None, dS1=None):
    """out [T, C] (zero in rows of no sequence), last states [N, W - 1, C]; with dy also the gradients of
    x, w, b, S for dy and dS1 (None: zero)."""
    x, w, b, S = _leaf(x), _leaf(w), _leaf(b), _leaf(S)
    W, C = w.shape[1], x.shape[1]
    out, last = torch.zeros_like(x), []
    rows = []
    for n in range(len(cu) - 1):
        old = S[n] if S is not None else torch.zeros(W - 1, C, dtype=torch.float64)
        every = torch.cat([old, x[cu[n]:cu[n + 1]]])
        for t in range(cu[n], cu[n + 1]):
            u = (w.T * every[t - cu[n]:t - cu[n] + W]).sum(0)
            if b is not None:
                u = u + b
            rows.append((t, u * torch.sigmoid(u) if silu else u))
        last.append(every[len(every) - (W - 1):])
    if rows:
        out = torch.zeros_like(x).index_copy(0, torch.tensor([t for t, _ in rows]), torch.stack([y for _, y in rows]))
    last = torch.stack(last) if last else torch.zeros(0, W - 1, C, dtype=torch.float64)
    if dy is None:
        return out.detach(), last.detach()
    loss = (out * dy.double().cpu()).sum()
    if dS1 is not None:
        loss = loss + (last * dS1.double().cpu()).sum()
    return out.detach(), last.detach(), _grads(loss, dict(x=x, w=w, b=b, S=S))


def _grads(loss, leaves):
    names = [m for m, v in leaves.items() if v is not None]
    got = torch.autograd.grad(loss, [leaves[m] for m in names], allow_unused=True) if loss.requires_grad else [None] * len(names)
    return {m: torch.zeros_like(leaves[m]) if g is None else g for m, g in zip(names, got)}


def scan(x, dt, A, B, C, D, bias, softplus, z, S, cu, dy=None, dS1=None):
    """out [T, ch] (zero in rows of no sequence), last states [N, ch, n]; with dy also the gradients."""
    leaves = dict(x=_leaf(x), dt=_leaf(dt), A=_leaf(A), B=_leaf(B), C=_leaf(C), D=_leaf(D), bias=_leaf(bias),
                  z=_leaf(z), S=_leaf(S))
    x, dt, A, B, C, D, bias, z, S = leaves.values()
    T, ch = x.shape
    per = ch // B.shape[1]
    step = dt if bias is None else dt + bias
    if softplus:
        step = torch.logaddexp(step, torch.zeros_like(step))
    ts, ys, last = [], [], []
    for n in range(len(cu) - 1):
        h = S[n] if S is not None else torch.zeros_like(A)
        for t in range(cu[n], cu[n + 1]):
            d = step[t][:, None]
            h = torch.exp(d * A) * h + d * B[t].repeat_interleave(per, 0) * x[t][:, None]
            y = (C[t].repeat_interleave(per, 0) * h).sum(-1)
            if D is not None:
                y = y + D * x[t]
            if z is not None:
                y = y * z[t] * torch.sigmoid(z[t])
            ts.append(t)
            ys.append(y)
        last.append(h)
    out = torch.zeros(T, ch, dtype=torch.float64)
    if ts:
        out = out.index_copy(0, torch.tensor(ts), torch.stack(ys))
    last = torch.stack(last) if last else torch.zeros(0, *A.shape, dtype=torch.float64)
    if dy is None:
        return out.detach(), last.detach()
    loss = (out * dy.double().cpu()).sum()
    if dS1 is not None:
        loss = loss + (last * dS1.double().cpu()).sum()
    return out.detach(), last.detach(), _grads(loss, leaves)


def norm(x, w, res, z, eps, sigmoid, dy=None, dres=None):
    """y, and h = x + residual; with dy the gradients at h (x where there is no residual), w and z instead."""
    h = x.double().cpu() if res is None else x.double().cpu() + res.double().cpu()
    h, w, z = _leaf(h), _leaf(w), _leaf(z)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w
    if z is not None:
        y = y * torch.sigmoid(z) * (1.0 if sigmoid else z)
    if dy is None:
        return y.detach(), h.detach()
    g = _grads((y * dy.double().cpu()).sum(), dict(x=h, w=w, z=z))
    if dres is not None:
        g["x"] = g["x"] + dres.double().cpu()
    return g


def conv_inputs(seed, T, C, W, N, dtype, params=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = params or F32
    return dict(x=r(T, C).to(dtype), w=(r(C, W) / W ** 0.5).to(p), b=(0.2 * r(C)).to(p), S=r(N, W - 1, C).to(dtype),
                dy=r(T, C).to(dtype), dS=r(N, W - 1, C).to(dtype))


def scan_inputs(seed, T, ch, G, n, N, dtype, softplus=True, slow=0.05):
    """Steps of about `slow` to ten times that, decay rates of 0.2 to some per unit step: at most about
    1 / (0.2 slow) tokens are remembered (100 by default)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    step = slow * 10 ** torch.rand(ch, generator=g)
    x = dict(x=r(T, ch).to(dtype), A=-(0.2 + 4.0 * torch.rand(ch, n, generator=g)), B=r(T, G, n).to(dtype),
             C=r(T, G, n).to(dtype), D=r(ch), z=r(T, ch).to(dtype), S=r(N, ch, n), dy=r(T, ch).to(dtype),
             dS=0.3 * r(N, ch, n))
    if softplus:
        x["bias"], x["dt"] = torch.log(torch.expm1(step)), (0.3 * r(T, ch)).to(dtype)
    else:
        x["bias"], x["dt"] = None, (step * torch.exp(0.3 * r(T, ch))).to(dtype)
    return x
