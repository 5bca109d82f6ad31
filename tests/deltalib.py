"""The gated delta rule and its gradient in binary64, token by token, for the tests of the sequence
kernels: a plain loop over sequences, heads and tokens on the CPU, written from

    S_t = A_t S_{t-1} + beta_t k_t v_t^T,  o_t = S_t^T q_t,
    A_t = (I - beta_t k_t k_t^T) Diag(a_t)  or, delta first, Diag(a_t) (I - beta_t k_t k_t^T).

No code is shared with the library."""
import torch


def run(q, k, v, alpha, beta, S0, cu, decay_first=True):
    """q, k [T, K, d], v [T, H, d], alpha [T, H] or [T, H, d], beta [T, H], S0 [N, H, d, d], cu list.
    Returns out [T, H, d] (zero in rows of no sequence) and last states, in binary64."""
    q, k, v, alpha, beta, S0 = (x.double() for x in (q, k, v, alpha, beta, S0))
    T, H, d = v.shape
    grp = H // q.shape[1]
    out, S = torch.zeros_like(v), S0.clone()
    q, k = q.repeat_interleave(grp, 1), k.repeat_interleave(grp, 1)
    if alpha.dim() == 2:
        alpha = alpha[..., None].expand(T, H, d)
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            kk, a, b = k[t][:, :, None], alpha[t][:, :, None], beta[t][:, None, None]
            if decay_first:
                X = a * S[n]
                S[n] = X - b * kk * (kk * X).sum(1, keepdim=True)
            else:
                S[n] = a * (S[n] - b * kk * (kk * S[n]).sum(1, keepdim=True))
            S[n] += b * kk * v[t][:, None, :]
            out[t] = (S[n] * q[t][:, :, None]).sum(1)
    return out, S


def gradient(q, k, v, alpha, beta, S0, cu, d_out, dS1):
    """Gradient of run() (scalar gates) by the adjoint recursion, token by token, in binary64: with
    G_t the gradient of S_t, u = S_{t-1}^T k, e = v - a u, de = beta G^T k:
      dq = S_t do;  dbeta = k.(G e);  dv = de;  dk = beta G e - a S_{t-1} de;
      da = <G, S_{t-1}> - de.u;  G_{t-1} = a G - a k de^T."""
    q, k, v, alpha, beta, S0, d_out, dS1 = (x.double() for x in (q, k, v, alpha, beta, S0, d_out, dS1))
    T, H, d = v.shape
    K = q.shape[1]
    grp = H // K
    g = dict(dq=torch.zeros(T, H, d, dtype=torch.float64), dk=torch.zeros(T, H, d, dtype=torch.float64),
             dv=torch.zeros(T, H, d, dtype=torch.float64), dalpha=torch.zeros(T, H, dtype=torch.float64),
             dbeta=torch.zeros(T, H, dtype=torch.float64), dS=torch.zeros_like(S0))
    for n in range(len(cu) - 1):
        for h in range(H):
            qs, ks, vs = q[:, h // grp], k[:, h // grp], v[:, h]
            S, was = S0[n, h].clone(), []
            for t in range(cu[n], cu[n + 1]):
                was.append(S)
                e = vs[t] - alpha[t, h] * (S.T @ ks[t])
                S = alpha[t, h] * S + beta[t, h] * torch.outer(ks[t], e)
            G = dS1[n, h].clone()
            for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
                P, a, b, kt, do = was.pop(), alpha[t, h], beta[t, h], ks[t], d_out[t, h]
                u = P.T @ kt
                e = vs[t] - a * u
                S = a * P + b * torch.outer(kt, e)
                g["dq"][t, h] = S @ do
                G = G + torch.outer(qs[t], do)
                Ge, de = G @ e, b * (G.T @ kt)
                g["dbeta"][t, h] = kt @ Ge
                g["dv"][t, h] = de
                g["dk"][t, h] = b * Ge - a * (P @ de)
                g["dalpha"][t, h] = (G * P).sum() - de @ u
                G = a * (G - torch.outer(kt, de))
            g["dS"][n, h] = G
    for m in ("dq", "dk"):
        g[m] = g[m].reshape(T, K, grp, d).sum(2)
    return g


def rel(x, y):
    """||x - y|| / ||y|| (the absolute norm where y is zero)."""
    x, y = x.double().cpu(), y.double().cpu()
    n = float(y.norm())
    return float((x - y).norm()) / (n if n else 1.0)


def inputs(seed, T, K, H, d, N, dtype, kda=False, gates="usual"):
    """Unit queries and keys with a common direction, values, gates and strengths, states; CPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(r(T, K, d)).to(dtype), unit(r(T, K, d) + 0.4 * r(1, K, d)).to(dtype)
    v, beta = r(T, H, d).to(dtype), torch.sigmoid(r(T, H))
    alpha = 0.8 + 0.2 * torch.rand(*((T, H, d) if kda else (T, H)), generator=g)
    if gates == "any":  # zeros, ones, sign changes and a gate above one
        pick = torch.randint(0, 8, alpha.shape, generator=g)
        for i, x in enumerate((0.0, 1.0, -0.7, 1.05, 1e-30)):
            alpha[pick == i] = x
    return dict(q=q, k=k, v=v, alpha=alpha, beta=beta, S=0.3 * r(N, H, d, d), do=r(T, H, d).to(dtype),
                dS=0.3 * r(N, H, d, d))


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu
