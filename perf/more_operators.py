"""The operators of a layer around its recurrence, as cases that can be measured: the short causal
convolution in front of it, the selective state space scan (the recurrence whose states decay by
themselves), and the root-mean-square norm behind it (gated) or before the next block (with the
residual's addition, 8 bits out); with their gradients and their forms for single tokens.

    convolution   u_t = b + sum_j w_j x_{t-(W-1)+j},  y = u or u sigmoid(u)
    scan          h_t = exp(D_t A) h_{t-1} + D_t B_t x_t,  y_t = (C_t . h_t + skip x_t) z sigmoid(z),
                  D_t = softplus(dt_t + bias), per channel and state; channels share B, C in equal groups
    norm          h = x + residual,  y = h / sqrt(mean h^2 + eps) w act(z),  scale = max |y| / top,
                  codes = y / scale

Where `own` is false everything is elementary torch operations in 32 bits; the scan's recurrence is a
loop over the tokens of a chunk, all chunks at once, and over the chunks.
"""
import random

import torch

own = False

L = 64  # tokens of a chunk in the plain form of the scan
EPS = 1e-6
_F = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "i8": 1}
_TOP = {"e4m3": 448.0, "i8": 127.0}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _case(name, op, dtype, **more):
    c = dict(op=op, dtype=dtype, **more)
    return dict(name=name, **c) if name else c


def _conv(name, op, dtype, seqs, tokens, ch, width=4, silu=True, bias=True, params="f32", ragged=True, state=True):
    return _case(name, op, dtype, seqs=seqs, tokens=tokens, ch=ch, width=width, silu=silu, bias=bias,
                 params=params, ragged=ragged, state=state)


def _scan(name, op, dtype, seqs, tokens, ch, n=16, groups=1, z=True, softplus=True, ragged=True, state=True):
    return _case(name, op, dtype, seqs=seqs, tokens=tokens, ch=ch, n=n, groups=groups, z=z, softplus=softplus,
                 ragged=ragged, state=state)


def _norm(name, op, dtype, rows, heads, d, residual=False, gate="", out="", group=0, params="f32"):
    return _case(name, op, dtype, rows=rows, heads=heads, d=d, residual=residual, gate=gate, out=out or dtype,
                 group=group, params=params)


def listed():
    return [
        # eight prompts of about 2,048 tokens: queries, keys and values of 16, 16 and 48 heads together
        _conv("conv-prefill", "conv", "bf16", 8, 16381, 10240, params="bf16"),
        # 70 requests of a batch that decodes, the last inputs in the slots of a pool
        _conv("conv-decode", "conv-step", "bf16", 70, 70, 10240, params="bf16"),
        # a training step's layer: four sequences of 2,048 tokens, 16, 16 and 32 heads
        _conv("conv-train", "conv-back", "bf16", 4, 8192, 8192, ragged=False, state=False),
        # two short turns on a small layer: launches are all there is
        _scan("scan-tiny", "scan", "f32", 2, 37, 256),
        # eight prompts of about 2,048 tokens: the ordinary prefill
        _scan("scan-prefill", "scan", "bf16", 8, 16381, 4096),
        # one long document from an empty state, few channels: few rows, a long axis
        _scan("scan-long", "scan", "bf16", 1, 16384, 2048, state=False),
        # 70 requests of a batch that decodes, states in the slots of a pool
        _scan("scan-decode", "scan-step", "bf16", 70, 70, 6144),
        # a training step's layer: four sequences of 2,048 tokens
        _scan("scan-train", "scan-back", "bf16", 4, 8192, 4096, ragged=False, state=False),
        # packed documents of odd lengths with a carried state, four groups, more states a channel
        _scan("scan-back-ragged", "scan-back", "f16", 6, 3001, 1536, n=32, groups=4),
        # the readouts of a prefill, 48 heads of 128, gated
        _norm("norm-readout", "norm", "bf16", 16381, 48, 128, gate="silu"),
        # the next block's input of a batch that decodes: residual added, 8 bits out
        _norm("norm-decode-e4m3", "norm", "bf16", 70, 1, 4096, residual=True, out="e4m3", params="bf16"),
        # a training step's norm of 4 x 2,048 tokens, with the residual's gradient
        _norm("norm-train", "norm-back", "bf16", 8192, 1, 4096, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["conv", "conv-step", "conv-back", "scan", "scan-step", "scan-back", "norm", "norm-back"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    params = rng.choice(["f32", dtype])
    if op.startswith("norm"):
        heads = rng.choice([1, 1, 4, 12, 32, 48])
        d = 8 * _log_int(rng, 8, 1024) if heads == 1 else rng.choice([64, 128])
        rows = _log_int(rng, 1, max(2, 20_000_000 // (heads * d)))
        residual, gate = rng.choice([(True, ""), (False, "silu"), (False, "sigmoid"), (False, "")])
        out, group = "", 0
        if op == "norm" and rng.random() < 0.5:
            out = rng.choice(["e4m3", "e4m3", "i8"])
            group = rng.choice([0, 128]) if d % 128 == 0 else 0
        return _norm(None, op, dtype, rows, heads, d, residual, gate, out, group, params)
    ragged, state = rng.random() < 0.75, rng.random() < 0.7
    if op.endswith("step"):
        ch, n = 8 * _log_int(rng, 8, 1280), rng.choice([8, 16, 16, 32, 64])
        seqs = _log_int(rng, 1, min(256, 60_000_000 // (ch * n)))
        each = rng.choice([1, 1, 1, 2, 4, 7])
        if op == "conv-step":
            return _conv(None, op, dtype, seqs, seqs * each, ch, rng.choice([2, 3, 4, 4]), rng.random() < 0.8,
                         rng.random() < 0.5, params, ragged and each > 1)
        return _scan(None, op, dtype, seqs, seqs * each, ch, n, 1,
                     rng.random() < 0.7, rng.random() < 0.8, ragged and each > 1)
    most = {"conv": 60_000_000, "conv-back": 40_000_000, "scan": 300_000_000, "scan-back": 150_000_000}[op]
    if op.startswith("conv"):
        ch = 8 * _log_int(rng, 8, 1280)
        tokens = _log_int(rng, 5, max(64, min(16000, most // ch)))
    else:
        n = rng.choice([8, 16, 16, 16, 32, 64])
        groups = rng.choice([1, 1, 2, 4])
        ch = 8 * groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        tokens = _log_int(rng, 5, max(64, min(16000, most // (ch * n))))
    seqs = min(_log_int(rng, 1, 48), tokens)
    if not ragged:
        tokens = max(1, tokens // seqs) * seqs
    if op.startswith("conv"):
        return _conv(None, op, dtype, seqs, tokens, ch, rng.choice([2, 3, 4, 4]), rng.random() < 0.8,
                     rng.random() < 0.5, params, ragged, state)
    return _scan(None, op, dtype, seqs, tokens, ch, n, groups, rng.random() < 0.7, rng.random() < 0.8, ragged, state)


def _lengths(case):
    """Lengths of the sequences: equal, or spread about the mean with an empty one and a single token
    among them where there are enough."""
    n, total = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [total // n] * n
    r = random.Random(n * 1000003 + total)
    w = [r.uniform(0.5, 1.5) for _ in range(n)]
    if n >= 4 and total >= 8 * n:
        w[1], w[2] = 0.0, 0.0
    left = total - (1 if n >= 4 and w[2] == 0.0 else 0)
    cut, acc, s = [0], 0.0, sum(w)
    for x in w:
        acc += x
        cut.append(int(round(left * acc / s)))
    got = [b - a for a, b in zip(cut, cut[1:])]
    got[2 if n >= 4 else 0] += total - sum(got)
    return got


def work(case):
    e, op = _SIZE[case["dtype"]], case["op"]
    if op.startswith("norm"):
        R, n = case["rows"] * case["heads"], case["rows"] * case["heads"] * case["d"]
        w = case["d"] * _SIZE[case["params"]]
        z = n * e if case["gate"] else 0
        if op == "norm-back":  # input, output's gradient (residual's, gate) in; gradients out
            return {"bytes": 3 * n * e + (n * e if case["residual"] else 0) + 2 * z + w + 4 * case["d"], "flops": 16 * n}
        q = R * 4 * (case["d"] // case["group"] if case["group"] else 1) if case["out"] in _TOP else 0
        return {"bytes": n * (e + _SIZE[case["out"]]) + (2 * n * e if case["residual"] else 0) + z + w + q,
                "flops": 8 * n}
    T, ch, n = case["tokens"], case["ch"], case["seqs"]
    if op.startswith("conv"):
        W = case["width"]
        p = ch * (W + case["bias"]) * _SIZE[case["params"]]
        S = n * (W - 1) * ch * e
        if op == "conv-back":
            return {"bytes": 3 * T * ch * e + p + 4 * ch * (W + case["bias"]) + (3 * S if case["state"] else 0),
                    "flops": (6 * W + 10) * T * ch}
        return {"bytes": 2 * T * ch * e + p + (2 * S if case["state"] else S), "flops": (2 * W + 5) * T * ch}
    N, z = case["n"], T * ch * e if case["z"] else 0
    bc, par, S = 2 * T * case["groups"] * N * e, ch * (N + 2) * 4, n * ch * N * 4
    if op == "scan-back":  # x, dt, z, the output's gradient in; their gradients out
        return {"bytes": 5 * T * ch * e + 2 * z + 2 * bc + 2 * par + (3 * S if case["state"] else 0),
                "flops": 20 * T * ch * N}
    return {"bytes": 3 * T * ch * e + z + bc + par + (2 * S if case["state"] else S), "flops": 7 * T * ch * N}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    """Projections of unit size.  The scan's as a layer has them: inputs behind the convolution, steps
    of 0.001 to 0.1, state n of a channel decaying about n + 1 times as fast as the first.  The norm's
    with a few loud columns."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    dt, op = _F[case["dtype"]], case["op"]
    st = {"case": dict(case)}
    if op.startswith("norm"):
        R, H, d = case["rows"], case["heads"], case["d"]
        shape = (R, H, d) if H > 1 else (R, d)
        loud = 1.0 + 15.0 * (uni(d) < 0.01)
        st["x"] = (rnd(*shape) * loud).to(dt)
        st["w"] = (1.0 + 0.1 * rnd(d)).to(_F[case["params"]])
        st["z"] = rnd(*shape).to(dt) if case["gate"] else None
        st["r"] = (rnd(*shape) * loud).to(dt) if case["residual"] else None
        if op == "norm-back":
            st["dy"] = rnd(*shape).to(dt)
        return st
    T, ch, n = case["tokens"], case["ch"], case["seqs"]
    lens = _lengths(case)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["lens"] = lens
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if case["ragged"] else None
    slots = n + 1 + n // 8 if op.endswith("step") else n
    if op.endswith("step"):
        st["slots"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
    if op.startswith("conv"):
        W = case["width"]
        st["x"] = rnd(T, ch).to(dt)
        st["w"] = (rnd(ch, W) / W ** 0.5).to(_F[case["params"]])
        st["b"] = (0.2 * rnd(ch)).to(_F[case["params"]]) if case["bias"] else None
        st["S"] = rnd(slots, W - 1, ch).to(dt) if case["state"] else None
        if op == "conv-back":
            st["dy"] = rnd(T, ch).to(dt)
            st["dS"] = rnd(n, W - 1, ch).to(dt) if case["state"] else None
        return st
    N, G = case["n"], case["groups"]
    u = rnd(T, ch)
    st["x"] = (u * torch.sigmoid(u)).to(dt)
    step = torch.exp(-6.9 + 4.6 * uni(ch))
    if case["softplus"]:
        st["bias"] = step + torch.log(-torch.expm1(-step))
        st["dt"] = (0.5 * rnd(T, ch)).to(dt)
    else:
        st["bias"] = None
        st["dt"] = (step * torch.exp(0.5 * rnd(T, ch))).to(dt)
    st["A"] = -(1.0 + torch.arange(N, device=dev)) * torch.exp(0.1 * rnd(ch, N))
    st["B"], st["C"] = rnd(T, G, N).to(dt), rnd(T, G, N).to(dt)
    st["D"] = 1.0 + 0.1 * rnd(ch)
    st["z"] = rnd(T, ch).to(dt) if case["z"] else None
    st["S"] = 0.3 * rnd(slots, ch, N) if case["state"] else None
    if op == "scan-back":
        st["dy"] = rnd(T, ch).to(dt)
        st["dS"] = 0.3 * rnd(n, ch, N) if case["state"] else None
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------

def _rows_of(st):
    """Sequence, place in it and length of it for every row; first rows and lengths of the sequences."""
    dev = st["x"].device
    ln = torch.tensor(st["lens"], device=dev)
    seq = torch.repeat_interleave(torch.arange(len(ln), device=dev), ln)
    start = torch.cumsum(ln, 0) - ln
    return seq, torch.arange(len(seq), device=dev) - start[seq], ln[seq], start, ln


def _conv_sum(st, S):
    """u, and the W inputs that each of its rows reads."""
    x, w = st["x"].float(), st["w"].float()
    W = w.shape[1]
    seq, pos, _, _, _ = _rows_of(st)
    row = torch.arange(len(seq), device=x.device)
    taps = []
    for j in range(W):
        back = W - 1 - j
        v = x[(row - back).clamp(min=0)]
        if S is None:
            before = torch.zeros(1, 1, device=x.device)
        else:
            before = S[seq, (pos + j).clamp(max=W - 2)]
        taps.append(torch.where((pos >= back)[:, None], v, before))
    u = torch.zeros_like(x) if st["b"] is None else st["b"].float().expand_as(x).clone()
    for j in range(W):
        u += taps[j] * w[:, j]
    return u, taps


def _conv_last(st, S):
    """The last W - 1 rows of state and inputs together, per sequence."""
    x, W = st["x"].float(), st["w"].shape[1]
    _, _, _, start, ln = _rows_of(st)
    at = ln[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
    v = x[(start[:, None] + at).clamp(0, len(x) - 1)]
    old = torch.zeros_like(v) if S is None else S.gather(1, (at + W - 1).clamp(max=W - 2)[..., None].expand_as(v))
    return torch.where((at >= 0)[..., None], v, old)


def _plain_conv(st):
    case, dt = st["case"], st["x"].dtype
    S = None if st["S"] is None else st["S"].float()
    if S is not None and "slots" in st:
        S = S[st["slots"].long()]
    u, _ = _conv_sum(st, S)
    out = (u * torch.sigmoid(u) if case["silu"] else u).to(dt)
    last = _conv_last(st, S).to(dt)
    if "slots" not in st:
        return {"out": out, "state": last}
    st["S"][st["slots"].long()] = last
    return {"out": out, "states": st["S"]}


def _plain_conv_back(st):
    case, x, w = st["case"], st["x"].float(), st["w"].float()
    dt, W, n = st["x"].dtype, w.shape[1], len(st["lens"])
    S = None if st["S"] is None else st["S"].float()
    u, taps = _conv_sum(st, S)
    du = st["dy"].float()
    if case["silu"]:
        s = torch.sigmoid(u)
        du = du * (s * (1 + u * (1 - s)))
    seq, pos, ln, start, each = _rows_of(st)
    row = torch.arange(len(seq), device=x.device)
    dx = torch.zeros_like(x)
    for j in range(W):
        ahead = W - 1 - j
        dx += torch.where((pos + ahead < ln)[:, None], du[(row + ahead).clamp(max=len(x) - 1)], torch.zeros_like(du[:1])) * w[:, j]
    got = {"dw": torch.stack([(du * t).sum(0) for t in taps], 1)}
    if case["bias"]:
        got["db"] = du.sum(0)
    if S is not None:
        dS1 = st["dS"].float()
        at = pos - ln + W - 1
        dx += torch.where((at >= 0)[:, None], dS1[seq, at.clamp(min=0)], torch.zeros_like(dx[:1]))
        dS = torch.zeros_like(dS1)
        for r in range(W - 1):
            for j in range(r + 1):
                ok = r - j < each
                dS[:, r] += torch.where(ok[:, None], du[(start + r - j).clamp(max=len(x) - 1)], torch.zeros_like(du[:1])) * w[:, j]
            back = r - each  # the old row that is still the last ones' row `back`
            dS[:, r] += torch.where((back >= 0)[:, None], dS1[torch.arange(n, device=x.device), back.clamp(min=0)], torch.zeros_like(du[:1]))
        got["dS"] = dS.to(dt)
    return dict(got, dx=dx.to(dt))


def _chunks(st):
    """Every row's place in chunks of L rows that no two sequences share; per sequence its first chunk
    and how many there are."""
    seq, pos, _, _, ln = _rows_of(st)
    many = (ln + L - 1) // L
    first = torch.cumsum(many, 0) - many
    host = [-(-x // L) for x in st["lens"]]
    return first[seq] * L + pos, first, many, sum(host), max(host)


def _in_chunks(x, place, M):
    y = torch.zeros((M * L,) + tuple(x.shape[1:]), dtype=x.dtype, device=x.device)
    return y.index_copy(0, place, x).reshape((M, L) + tuple(x.shape[1:]))


def _scan_sum(st, x, delta, A, B, C, S):
    """sum_n C h of every row, and the last states; from states S [n, ch, N]."""
    T, ch = x.shape
    N, G = B.shape[2], B.shape[1]
    place, first, many, M, most = _chunks(st)
    xd, d = _in_chunks(x * delta, place, M), _in_chunks(delta, place, M)
    Bc, Cc = _in_chunks(B, place, M), _in_chunks(C, place, M)
    A = A.reshape(G, ch // G, N)
    wide = lambda v: v.reshape(M, G, ch // G, 1)  # noqa: E731

    def one(h, t):
        return torch.exp(wide(d[:, t]) * A) * h + wide(xd[:, t]) * Bc[:, t, :, None, :]

    h = torch.zeros(M, G, ch // G, N, device=x.device)
    for t in range(L):
        h = one(h, t)
    decay = torch.exp(wide(d.sum(1)) * A)
    begin = torch.zeros(M, dtype=torch.long, device=x.device)
    H, kept = S.reshape(len(many), G, ch // G, N), []
    for i in range(most):  # states before chunk i of every sequence that has one
        kept.append(H)
        at = (first + i).clamp(max=M - 1)
        some = (i < many)[:, None, None, None]
        H = torch.where(some, decay[at] * H + h[at], H)
        begin = torch.where((torch.arange(M, device=x.device)[:, None] == (first + i)) & (i < many), i * len(many) + torch.arange(len(many), device=x.device), 0).sum(1) + begin
    h = torch.cat(kept)[begin]
    out = []
    for t in range(L):
        h = one(h, t)
        out.append((Cc[:, t, :, None, :] * h).sum(-1).reshape(M, ch))
    return torch.stack(out, 1).reshape(M * L, ch)[place], H.reshape(len(many), ch, N)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan_all(st, x, dt, A, B, C, D, bias, z, S):
    delta = _softplus(dt + bias) if bias is not None else dt
    y, last = _scan_sum(st, x, delta, A, B, C, S)
    y = y + D * x
    return (y * (z * torch.sigmoid(z)) if z is not None else y), last


def _first_states(st):
    if st["S"] is not None:
        return st["S"] if "slots" not in st else st["S"][st["slots"].long()]
    case = st["case"]
    return torch.zeros(case["seqs"], case["ch"], case["n"], device=st["x"].device)


def _plain_scan(st):
    f = lambda v: None if v is None else v.float()  # noqa: E731
    y, last = _plain_scan_all(st, *(f(st[m]) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z")), _first_states(st))
    if "slots" not in st:
        return {"out": y.to(st["x"].dtype), "state": last}
    st["S"][st["slots"].long()] = last
    return {"out": y.to(st["x"].dtype), "states": st["S"]}


_LEAVES = ("x", "dt", "A", "B", "C", "D", "bias", "z")


def _plain_scan_back(st):
    leaf = {m: st[m].float().detach().clone().requires_grad_(True) for m in _LEAVES if st[m] is not None}
    S = _first_states(st).clone().requires_grad_(st["S"] is not None)
    y, last = _plain_scan_all(st, *(leaf.get(m) for m in _LEAVES), S)
    ends, ups = [y], [st["dy"].float()]
    if st["S"] is not None:
        leaf["S"] = S
        ends.append(last)
        ups.append(st["dS"])
    got = torch.autograd.grad(ends, list(leaf.values()), ups)
    wide = ("A", "D", "bias", "S")
    return {"d" + m: v if m in wide else v.to(st["x"].dtype) for m, v in zip(leaf, got)}


def _gate(case, z):
    s = torch.sigmoid(z)
    return z * s if case["gate"] == "silu" else s


def _plain_norm(st):
    case, x = st["case"], st["x"].float()
    h = x if st["r"] is None else x + st["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["w"].float()
    if st["z"] is not None:
        y = y * _gate(case, st["z"].float())
    got = {} if st["r"] is None else {"h": h.to(st["x"].dtype)}
    if case["out"] not in _TOP:
        return dict(got, out=y.to(st["x"].dtype))
    y = y.unflatten(-1, (-1, case["group"] or case["d"]))
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / _TOP[case["out"]], torch.ones_like(top))
    v = (y / scale).flatten(-2)
    codes = v.to(torch.float8_e4m3fn) if case["out"] == "e4m3" else v.round().to(torch.int8)
    return dict(got, out=_held(case, codes, scale[..., 0]), scale=scale[..., 0] if case["group"] else scale[..., 0, 0])


def _held(case, codes, scale):
    """Eight bits as the values they stand for: e4m3 as it is, beside its scales; integers times theirs."""
    if case["out"] == "e4m3":
        return codes
    v = codes.float().unflatten(-1, (-1, case["group"] or case["d"])) * scale[..., None]
    return v.flatten(-2).to(torch.bfloat16)


def _plain_norm_back(st):
    case, h, dy, w = st["case"], st["x"].float(), st["dy"].float(), st["w"].float()
    dt = st["x"].dtype
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hat, got = h * r, {}
    if st["z"] is not None:
        z = st["z"].float()
        s = torch.sigmoid(z)
        slope = s * (1 + z * (1 - s)) if case["gate"] == "silu" else s * (1 - s)
        got["dz"] = (dy * hat * w * slope).to(dt)
        dy = dy * _gate(case, z)
    got["dw"] = (dy * hat).reshape(-1, case["d"]).sum(0)
    p = dy * w
    dx = r * (p - hat * (p * hat).mean(-1, keepdim=True))
    if st["r"] is not None:
        dx = dx + st["r"].float()
    return dict(got, dx=dx.to(dt))


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

_PLAIN = {"conv": _plain_conv, "conv-step": _plain_conv, "conv-back": _plain_conv_back, "scan": _plain_scan,
          "scan-step": _plain_scan, "scan-back": _plain_scan_back, "norm": _plain_norm, "norm-back": _plain_norm_back}


def run(st):
    case = st["case"]
    if not own:
        return _PLAIN[case["op"]](st)
    return _OWN[case["op"].split("-")[0]](st, case, case["op"])


def _own_conv(st, case, op):
    from quantized_delta_rule_amd import conv
    x, w, b = st["x"], st["w"], st["b"]
    how = dict(bias=b, activation=conv.SILU if case["silu"] else conv.NONE)
    how.update(dict(cu_seqlens=st["cu"]) if st["cu"] is not None else dict(n_seqs=case["seqs"]))
    if op == "conv-back":
        g = {"dx": torch.empty_like(x), "dw": torch.empty_like(w, dtype=torch.float32)}
        if b is not None:
            g["db"] = torch.empty_like(b, dtype=torch.float32)
        if st["S"] is not None:
            g["dS"] = torch.empty_like(st["S"])
        conv.backward(x, w, st["dy"], g["dx"], g["dw"], dbias=g.get("db"), state_in=st["S"], d_state_out=st["dS"],
                      d_state_in=g.get("dS"), **how)
        return g
    out = torch.empty_like(x)
    if op == "conv-step":
        conv.forward(x, w, out, state_in=st["S"], state_out=st["S"], slots=st["slots"], **how)
        return {"out": out, "states": st["S"]}
    last = torch.empty(case["seqs"], case["width"] - 1, case["ch"], dtype=x.dtype, device=x.device)
    conv.forward(x, w, out, state_in=st["S"], state_out=last, **how)
    return {"out": out, "state": last}


def _own_scan(st, case, op):
    from quantized_delta_rule_amd import scan
    args = [st[m] for m in ("x", "dt", "A", "B", "C")]
    how = dict(D=st["D"], dt_bias=st["bias"], softplus=case["softplus"], z=st["z"])
    how.update(dict(cu_seqlens=st["cu"]) if st["cu"] is not None else dict(n_seqs=case["seqs"]))
    if op == "scan-back":
        g = {"d" + m: torch.empty_like(st[m]) for m in _LEAVES + ("S",) if st[m] is not None}
        scan.backward(*args, st["dy"], g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], dD=g["dD"],
                      ddt_bias=g.get("dbias"), dz=g.get("dz"), state_in=st["S"], d_state_out=st["dS"],
                      d_state_in=g.get("dS"), **how)
        return g
    out = torch.empty_like(st["x"])
    if op == "scan-step":
        scan.forward(*args, out, state_in=st["S"], state_out=st["S"], slots=st["slots"], **how)
        return {"out": out, "states": st["S"]}
    last = torch.empty(case["seqs"], case["ch"], case["n"], device=out.device)
    scan.forward(*args, out, state_in=st["S"], state_out=last, **how)
    return {"out": out, "state": last}


def _own_norm(st, case, op):
    from quantized_delta_rule_amd import norm
    x, w = st["x"], st["w"]
    how = dict(eps=EPS, z=st["z"], gate=norm.SIGMOID if case["gate"] == "sigmoid" else norm.SILU)
    if op == "norm-back":
        g = {"dx": torch.empty_like(x), "dw": torch.empty(case["d"], device=x.device)}
        if st["z"] is not None:
            g["dz"] = torch.empty_like(x)
        norm.backward(x, w, st["dy"], g["dx"], g["dw"], dz=g.get("dz"), d_residual=st["r"], **how)
        return g
    got = {} if st["r"] is None else {"h": torch.empty_like(x)}
    if case["out"] not in _TOP:
        got["out"] = torch.empty_like(x)
        norm.forward(x, w, got["out"], residual=st["r"], residual_out=got.get("h"), **how)
        return got
    codes = torch.empty_like(x, dtype=torch.float8_e4m3fn if case["out"] == "e4m3" else torch.int8)
    lead = tuple(x.shape[:-1])
    got["scale"] = torch.empty(lead + ((case["d"] // case["group"],) if case["group"] else ()), device=x.device)
    norm.forward(x, w, codes, residual=st["r"], residual_out=got.get("h"), scale=got["scale"], group=case["group"], **how)
    got["out"] = _held(case, codes, got["scale"] if case["group"] else got["scale"][..., None])
    return got


_OWN = {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"].split("-")[0]](st, case)


def _exact_conv(st, case):
    back, W = case["op"] == "conv-back", case["width"]
    x, w = st["x"].double(), st["w"].double().requires_grad_(back)
    b = torch.zeros(case["ch"], dtype=torch.float64, device=x.device) if st["b"] is None else st["b"].double()
    b.requires_grad_(back)
    S = None if st["S"] is None else st["S"].double()
    outs, lasts, at, dx, dS, dw, db = [], [], 0, [], [], 0, 0
    for s, ln in enumerate(st["lens"]):
        old = torch.zeros(W - 1, case["ch"], dtype=torch.float64, device=x.device) if S is None else S[int(st["slots"][s]) if "slots" in st else s]
        every = torch.cat([old, x[at:at + ln]]).requires_grad_(back)
        u = b + sum(w[:, j] * every[j:j + ln] for j in range(W))
        y = u / (1 + torch.exp(-u)) if case["silu"] else u
        if back:
            ends, ups = [y], [st["dy"][at:at + ln].double()]
            if S is not None:
                ends.append(every[ln:])
                ups.append(st["dS"][s].double())
            g = torch.autograd.grad(ends, [every, w, b], ups)
            dS.append(g[0][:W - 1])
            dx.append(g[0][W - 1:])
            dw, db = dw + g[1], db + g[2]
        else:
            outs.append(y)
            lasts.append(every[ln:])
        at += ln
    if back:
        r = {"dx": torch.cat(dx), "dw": dw}
        if st["b"] is not None:
            r["db"] = db
        if S is not None:
            r["dS"] = torch.stack(dS)
        return r
    last = torch.stack(lasts)
    if "slots" not in st:
        return {"out": torch.cat(outs), "state": last}
    S = S.clone()
    S[st["slots"].long()] = last
    return {"out": torch.cat(outs), "states": S}


def _padded(v, lens, fill=0.0):
    y = torch.full((len(lens), max(lens)) + tuple(v.shape[1:]), fill, dtype=torch.float64, device=v.device)
    for s, part in enumerate(torch.split(v, lens)):
        y[s, :len(part)] = part
    return y


def _exact_scan(st, case):
    n, ch, N, G, lens = case["seqs"], case["ch"], case["n"], case["groups"], st["lens"]
    most = max(lens)
    back = case["op"] == "scan-back"
    if most * n * ch * N * 8 > (6e10 if back else 1e12):
        return None
    x, raw = st["x"].double(), st["dt"].double()
    if st["bias"] is not None:
        raw = raw + st["bias"].double()
        delta = torch.logaddexp(raw, torch.zeros_like(raw))
    else:
        delta = raw
    A, D = st["A"].double(), st["D"].double()
    xs, ds = _padded(x, lens), _padded(delta, lens)
    Bs, Cs = _padded(st["B"], lens), _padded(st["C"], lens)
    per = lambda v: v.repeat_interleave(ch // G, 1)  # noqa: E731
    S = _first_states(st).double()
    hs, ys = [], []
    for t in range(most):
        if back:
            hs.append(S)
        d = ds[:, t, :, None]
        S = torch.exp(d * A) * S + d * per(Bs[:, t]) * xs[:, t, :, None]
        ys.append((per(Cs[:, t]) * S).sum(-1))
    pick = lambda v: torch.cat([v[s, :ln] for s, ln in enumerate(lens)])  # noqa: E731
    inner = pick(torch.stack(ys, 1)) + D * x
    del ys
    if st["z"] is not None:
        z = st["z"].double()
        sg = 1 / (1 + torch.exp(-z))
    if not back:
        out = inner * z * sg if st["z"] is not None else inner
        if "slots" not in st:
            return {"out": out, "state": S}
        every = st["S"].double()
        every[st["slots"].long()] = S
        return {"out": out, "states": every}
    dy, r = st["dy"].double(), {}
    if st["z"] is not None:
        r["dz"] = dy * inner * sg * (1 + z * (1 - sg))
        dy = dy * z * sg
    up = _padded(dy, lens)
    g = st["dS"].double() if st["dS"] is not None else torch.zeros_like(S)
    dA = torch.zeros_like(A)
    dxs, dds, dBs, dCs = [], [], [], []
    for t in range(most - 1, -1, -1):
        was, d = hs.pop(), ds[:, t, :, None]
        a = torch.exp(d * A)
        b, xt = per(Bs[:, t]), xs[:, t, :, None]
        now = a * was + d * b * xt
        e = up[:, t, :, None]
        # a padded row has no output and no step: it leaves g as it was
        dCs.append((e * now).reshape(n, G, ch // G, N).sum(2))
        g = g + per(Cs[:, t]) * e
        dBs.append((g * d * xt).reshape(n, G, ch // G, N).sum(2))
        dxs.append((g * d * b).sum(-1))
        dds.append((g * (A * a * was + b * xt)).sum(-1))
        dA += (g * d * a * was).sum(0)
        g = g * a
    flip = lambda v: pick(torch.stack(v[::-1], 1))  # noqa: E731
    r["dx"] = flip(dxs) + D * dy
    dd = flip(dds)
    if st["bias"] is not None:
        dd = dd / (1 + torch.exp(-raw))
        r["dbias"] = dd.sum(0)
    r.update(ddt=dd, dB=flip(dBs), dC=flip(dCs), dA=dA, dD=(dy * x).sum(0))
    if st["S"] is not None:
        r["dS"] = g
    return r


def _exact_norm(st, case):
    d = case["d"]
    if case["op"] == "norm":
        h = st["x"].double()
        if st["r"] is not None:
            h = h + st["r"].double()
        y = st["w"].double() * h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / d + EPS)
        if st["z"] is not None:
            z = st["z"].double()
            y = y * (z if case["gate"] == "silu" else 1.0) / (1 + torch.exp(-z))
        r = {} if st["r"] is None else {"h": h}
        if case["out"] not in _TOP:
            return dict(r, out=y)
        parts = y.unflatten(-1, (-1, case["group"] or d))
        scale = parts.abs().max(-1).values / _TOP[case["out"]]
        # e4m3 before its rounding, as other types; integers' values with theirs, since a step is wide of its type
        y = parts / scale[..., None]
        y = (y if case["out"] == "e4m3" else torch.round(y) * scale[..., None]).flatten(-2)
        return dict(r, out=y, scale=scale if case["group"] else scale[..., 0])
    h = st["x"].double().requires_grad_(True)
    w = st["w"].double().requires_grad_(True)
    leaves = {"dx": h, "dw": w}
    y = w * h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / d + EPS)
    if st["z"] is not None:
        z = leaves["dz"] = st["z"].double().requires_grad_(True)
        y = y * (z if case["gate"] == "silu" else 1.0) / (1 + torch.exp(-z))
    r = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), st["dy"].double())))
    if st["r"] is not None:
        r["dx"] = r["dx"] + st["r"].double()
    return r


_EXACT = {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}
