"""The Delta-rule operators beside the packed decode step, as cases that can be measured: the gated
delta rule over whole sequences (chunked) and over a token or a few (recurrent), its gradient, and
prompts that enter and leave a packed state pool.

Per value head, with state S [d, d] (key rows, value columns), gate a, strength b:

    e_t = v_t - S_{t-1}^T Diag(a_t) k_t      S_t = Diag(a_t) S_{t-1} + b_t k_t e_t^T      o_t = S_t^T q_t

GDN has one gate a head and token.  KDA has one a key row; in its delta-first order
S_t = Diag(a_t) (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T instead.  Value heads share key heads in
equal groups.  Where `own` is false everything is elementary torch operations in 32 bits (gates'
logarithms, inverses and quantiser decisions in 64); a recurrence over chunks or tokens is a loop.
"""
import random

import torch

own = False

C = 64  # tokens of a chunk in the plain form
_F = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _case(name, op, dtype, seqs, tokens, heads, qk_heads, d, **more):
    c = dict(op=op, dtype=dtype, seqs=seqs, tokens=tokens, heads=heads, qk_heads=qk_heads, d=d,
             ragged=True, state=True)
    c.update(more)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # two short turns on a four-head layer of 64-wide states: launches are all there is
        _case("forward-tiny", "forward", "f32", 2, 37, 4, 4, 64),
        # 70 prompts of about 128 tokens on a 48-head layer, an empty one and a single token among them
        _case("forward-prompts", "forward", "f16", 70, 8960, 48, 16, 128),
        # eight prompts of about 2,048 tokens: the ordinary prefill
        _case("forward-prefill", "forward", "bf16", 8, 16381, 48, 16, 128),
        # one long document from an empty state: few rows, a long axis
        _case("forward-long", "forward", "bf16", 1, 16384, 32, 32, 128, state=False),
        # gradients of a small layer
        _case("backward-tiny", "backward", "f32", 3, 97, 4, 2, 64),
        # a training step's layer: four sequences of 2,048 tokens
        _case("backward-train", "backward", "bf16", 4, 8192, 32, 16, 128, ragged=False, state=False),
        # packed documents of odd lengths with a carried state
        _case("backward-ragged", "backward", "f16", 6, 3001, 12, 4, 128),
        # one request, one token: latency
        _case("step-one", "step", "bf16", 1, 1, 48, 16, 128, kind="gdn"),
        # 70 requests of a batch that decodes, states in the slots of a pool
        _case("step-batch", "step", "bf16", 70, 70, 48, 16, 128, kind="gdn"),
        # four tokens of each of 64 requests (drafted tokens that are checked at once), per-row gates
        _case("step-draft-rows", "step", "f32", 64, 256, 32, 32, 128, kind="kda", ragged=False),
        # 16 prompts of about 128 tokens continue from 6-bit slots
        _case("packed-prompts", "packed", "bf16", 16, 2053, 48, 16, 128, bits=6),
        # a 2,048-token piece of each of four long prompts, 8-bit slots
        _case("packed-piece", "packed", "f16", 4, 8192, 48, 16, 128, bits=8, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["forward", "backward", "step", "packed"])
    d = rng.choice([64, 128, 128, 128])
    group = rng.choice([1, 2, 3, 4])
    qk = rng.choice([1, 2, 4, 8, 12, 16])
    heads = qk * group
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    ragged = rng.random() < 0.75
    state = rng.random() < 0.7
    if op == "step":
        kind = rng.choice(["gdn", "gdn", "kda", "kda-decay"])
        if kind != "gdn":
            heads = qk  # per-row gates come with a key head of their own
        seqs = _log_int(rng, 1, 96)
        each = rng.choice([1, 1, 1, 2, 4, 7])
        return _case(None, op, dtype, seqs, seqs * each, heads, qk, d, kind=kind,
                     ragged=ragged and each > 1)
    most = {"forward": 6000, "backward": 3000, "packed": 4000}[op]
    tokens = _log_int(rng, 5, max(64, most * 32 // heads // (2 if dtype == "f32" else 1)))
    seqs = min(_log_int(rng, 1, 48), tokens)
    if not ragged:
        tokens = max(1, tokens // seqs) * seqs
    if op == "packed":
        return _case(None, op, dtype, seqs, tokens, heads, qk, d, bits=rng.choice([6, 8]),
                     ragged=ragged)
    return _case(None, op, dtype, seqs, tokens, heads, qk, d, ragged=ragged, state=state)


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
    d, T, H, K, n = case["d"], case["tokens"], case["heads"], case["qk_heads"], case["seqs"]
    e = _SIZE[case["dtype"]]
    rows = d if str(case.get("kind", "")).startswith("kda") else 1
    q, v = T * K * d * e, T * H * d * e
    gates = T * H * 4 * (rows + 1)
    S = n * H * d * d * 4
    if case["op"] == "backward":
        # q, k, v, the output's gradient and the gates in; their gradients out; states where carried
        byt = 2 * (2 * q + v + gates) + v + (3 * S if case["state"] else 0)
        return {"bytes": byt, "flops": 18 * T * H * d * d}
    io = 2 * q + 2 * v + gates
    if case["op"] == "packed":
        seg = H * (d * d * case["bits"] // 8 + 4 * d)
        return {"bytes": io + n * (2 * seg + seg + H * d * d * e), "flops": 6 * T * H * d * d}
    return {"bytes": io + (2 * S if case["state"] else S), "flops": 6 * T * H * d * d}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    """Queries and keys of unit length (keys about a direction of their head), values of unit size,
    strengths sigmoid(N(0, 1)), gates with a half-life of tens of tokens (GDN) or U(0.8, 1) a row
    (KDA), states as a layer holds them after some tens of tokens."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    d, T, H, K, n = case["d"], case["tokens"], case["heads"], case["qk_heads"], case["seqs"]
    dt = _F[case["dtype"]]
    lens = _lengths(case)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st = {"case": dict(case), "lens": lens}
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if case["ragged"] else None
    st["q"] = _unit(rnd(T, K, d)).to(dt)
    st["k"] = _unit(rnd(T, K, d) + 0.5 * rnd(1, K, d)).to(dt)
    st["v"] = rnd(T, H, d).to(dt)
    st["beta"] = torch.sigmoid(rnd(T, H))
    if str(case.get("kind", "")).startswith("kda"):
        st["alpha"] = 0.8 + 0.2 * torch.rand(T, H, d, generator=g, device=dev)
    else:
        st["alpha"] = torch.exp(-torch.nn.functional.softplus(-4.0 + 0.5 * rnd(T, H)))
    if case["op"] == "step":
        slots = n + 1 + n // 8
        st["slots"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
        st["S"] = 0.25 * rnd(slots, H, d, d)
    elif case["op"] == "packed":
        slots = n + 1 + n // 8
        st["slots"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
        st["omega"] = 0.5 + torch.rand(H, d, generator=g, device=dev)
        qmax = 2 ** (case["bits"] - 1) - 1
        z = (rnd(slots, H, d, d) * (qmax / 4.5)).round().clamp(-qmax, qmax)
        r = (0.1 + 0.05 * torch.rand(slots, H, d, generator=g, device=dev)).half()
        c = ((1.5 + 0.5 * torch.rand(slots, H, d, generator=g, device=dev)) * 6.0 / qmax).half()
        st["pool"] = _pack(z, r, c, case["bits"])
        if own:  # the layer's plan, which a serving process makes once
            import numpy as np
            from quantized_delta_rule_amd import stepq
            bits = np.full((H, d), case["bits"], np.int8)
            st["plan"] = stepq.Plan(stepq.GDN, bits, np.zeros((H, d), np.uint8),
                                    st["omega"].cpu().numpy(), device=torch.cuda.current_device())
    else:
        st["S"] = 0.25 * rnd(n, H, d, d) if case["state"] else None
        if case["op"] == "backward":
            st["d_out"] = rnd(T, H, d).to(dt)
            st["d_state"] = 0.1 * rnd(n, H, d, d) if case["state"] else None
    return st


# ---------------------------------------------------------------------------------------------
# the packed pool: per request and head 64 lane streams of b-bit codes (lane L holds columns
# G L .. G L + G - 1 row by row, word w of lane L at word 64 w + L), then binary16 row factors and
# binary16 column factors, padded to 256 bytes
# ---------------------------------------------------------------------------------------------

def _pack(z, r, c, b):
    n, H, d, _ = z.shape
    codes = z.to(torch.int32).reshape(n, H, d, 64, d // 64).permute(0, 1, 3, 2, 4).reshape(n, H, 64, d * d // 64, 1)
    bit = (codes >> torch.arange(b, dtype=torch.int32, device=z.device)) & 1
    bit = bit.reshape(n, H, 64, -1, 32).to(torch.int64)
    words = (bit << torch.arange(32, device=z.device)).sum(-1).to(torch.int32)
    words = words.transpose(-1, -2).contiguous().view(torch.uint8).reshape(n, H, -1)
    seg = torch.cat([words, r.contiguous().view(torch.uint8), c.contiguous().view(torch.uint8)], -1)
    size = -(-seg.shape[-1] // 256) * 256
    pool = torch.zeros(n, H, size, dtype=torch.uint8, device=z.device)
    pool[..., :seg.shape[-1]] = seg
    return pool.reshape(-1)


def _unpack(pool, n, H, d, b):
    """(z, r, c) of a pool of n requests."""
    words = 2 * b * (d // 64) * (d // 64)
    seg = pool.reshape(n, H, -1)
    w = seg[..., :256 * words].contiguous().view(torch.int32).reshape(n, H, words, 64).transpose(-1, -2)
    bit = (w[..., None] >> torch.arange(32, dtype=torch.int32, device=pool.device)) & 1
    bit = bit.reshape(n, H, 64, d * d // 64, b)
    z = (bit << torch.arange(b, dtype=torch.int32, device=pool.device)).sum(-1)
    z = torch.where(z >= 2 ** (b - 1), z - 2 ** b, z)
    z = z.reshape(n, H, 64, d, d // 64).permute(0, 1, 3, 2, 4).reshape(n, H, d, d)
    f = seg[..., 256 * words:256 * words + 4 * d].contiguous().view(torch.float16)
    return z, f[..., :d], f[..., d:]


def _requantise(S, omega, b):
    """Codes and factors of states S [.., d, d]: r_i = (mean_j |S_ij| + 1e-8) / (1 + w_i / mean w) and
    c_j by a weighted least-squares fit to codes of a first fit by the column maximum, both binary16."""
    qmax = 2 ** (b - 1) - 1
    S, om = S.double(), omega.double()
    r = ((S.abs().mean(-1) + 1e-8) / (1 + om / om.mean(-1, keepdim=True))).half()
    rd = r.double()
    y = S * torch.where(rd > 0, 1 / rd, torch.zeros_like(rd))[..., None]
    c0 = y.abs().amax(-2) / qmax
    inv = torch.where(c0 > 0, 1 / c0, torch.zeros_like(c0))
    z0 = (y * inv[..., None, :]).round().clamp(-qmax, qmax)
    wt = (om * rd * rd)[..., None]
    num, den = (wt * z0 * y).sum(-2), (wt * z0 * z0).sum(-2)
    c = torch.where(den > 0, num / den, c0).half()
    cd = c.double()
    z = (y * torch.where(cd > 0, 1 / cd, torch.zeros_like(cd))[..., None, :]).round().clamp(-qmax, qmax)
    return z, r, c


def _values(z, r, c):
    return (r.float()[..., None] * c.float()[..., None, :]) * z.float()


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------

def _grid(st, unit):
    """How many places a sequence gets (a multiple of `unit`) and each token's place."""
    lens, n = st["lens"], len(st["lens"])
    size = max(unit, -(-max(lens) // unit) * unit)
    dev = st["q"].device
    ln = torch.tensor(lens, device=dev)
    seq = torch.repeat_interleave(torch.arange(n, device=dev), ln)
    start = torch.cumsum(ln, 0) - ln
    return size, seq * size + torch.arange(len(seq), device=dev) - start[seq]


def _spread(x, size, place, n, fill=0.0):
    """[tokens, H, ..] -> [n, H, size, ..] with `fill` in the empty places."""
    y = torch.full((n * size,) + tuple(x.shape[1:]), fill, dtype=x.dtype, device=x.device)
    y = y.index_copy(0, place, x)
    return y.reshape((n, size) + tuple(x.shape[1:])).transpose(1, 2)


def _gather(y, size, place):
    y = y.transpose(1, 2)
    return y.reshape((-1,) + tuple(y.shape[2:]))[place]


def _chunked(q, k, v, alpha, beta, S, lens):
    """q, k, v [n, H, size, d], alpha, beta [n, H, size], S [n, H, d, d]: outputs and last states."""
    n, H, size, d = v.shape
    m = size // C
    q, k, v = (x.reshape(n, H, m, C, d) for x in (q, k, v))
    g = alpha.reshape(n, H, m, C).double().log().cumsum(-1)
    beta = beta.reshape(n, H, m, C, 1)
    low = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    decay = torch.where(low, g[..., :, None] - g[..., None, :], -torch.inf).exp().float()
    A = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1).double()
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) .. (I + A^32), since A^64 = 0
    eye = torch.eye(C, dtype=torch.float64, device=v.device)
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    A16 = A8 @ A8
    inv = ((eye - A) @ (eye + A2) @ (eye + A4) @ (eye + A8) @ (eye + A16) @ (eye + A16 @ A16)).float()
    P = (q @ k.transpose(-1, -2)) * decay
    gam, last = g.exp().float()[..., None], (g[..., -1:] - g).exp().float()[..., None]
    kt = (k * last).transpose(-1, -2)
    outs = []
    for c in range(m):
        R = beta[:, :, c] * (v[:, :, c] - gam[:, :, c] * (k[:, :, c] @ S))
        W = inv[:, :, c] @ R
        outs.append(gam[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ W)
        S = gam[:, :, c, -1:] * S + kt[:, :, c] @ W
    return torch.stack(outs, 2).reshape(n, H, size, d), S


def _plain_forward(st, q, k, v, alpha, beta, S):
    case = st["case"]
    n, H, d, grp = case["seqs"], case["heads"], case["d"], case["heads"] // case["qk_heads"]
    size, place = _grid(st, C)
    q = _spread(q.repeat_interleave(grp, 1), size, place, n)
    k = _spread(k.repeat_interleave(grp, 1), size, place, n)
    v = _spread(v, size, place, n)
    alpha, beta = _spread(alpha, size, place, n, 1.0), _spread(beta, size, place, n)
    if S is None:
        S = torch.zeros(n, H, d, d, device=v.device)
    out, S = _chunked(q, k, v, alpha, beta, S, st["lens"])
    return _gather(out, size, place), S


def _plain_backward(st):
    dt = st["q"].dtype
    leaves = [st[x].float().detach().requires_grad_(True) for x in ("q", "k", "v", "alpha", "beta")]
    S0 = st["S"].detach().requires_grad_(True) if st["S"] is not None else None
    out, S1 = _plain_forward(st, *leaves, S0)
    ends, grads = [out], [st["d_out"].float()]
    if st["d_state"] is not None:
        ends.append(S1)
        grads.append(st["d_state"])
    got = torch.autograd.grad(ends, leaves + ([S0] if S0 is not None else []), grads)
    r = dict(zip(("dq", "dk", "dv"), (x.to(dt) for x in got[:3])), dalpha=got[3], dbeta=got[4])
    if S0 is not None:
        r["dstate"] = got[5]
    return r


def _plain_step(st):
    case = st["case"]
    n, grp = case["seqs"], case["heads"] // case["qk_heads"]
    size, place = _grid(st, 1)
    at = st["slots"].long()
    q = _spread(st["q"].float().repeat_interleave(grp, 1), size, place, n)
    k = _spread(st["k"].float().repeat_interleave(grp, 1), size, place, n)
    v = _spread(st["v"].float(), size, place, n)
    a, b = _spread(st["alpha"], size, place, n, 1.0), _spread(st["beta"], size, place, n)
    S = st["S"][at]
    outs = []
    for t in range(size):
        kt, at_, bt = k[:, :, t, :, None], a[:, :, t], b[:, :, t, None, None]
        at_ = at_[..., None] if at_.dim() == 3 else at_[..., None, None]
        if case["kind"] == "kda":
            u = (S * kt).sum(-2, keepdim=True)
            S = at_ * (S - bt * kt * u) + bt * kt * v[:, :, t, None]
        else:
            S = at_ * S
            S = S + bt * kt * (v[:, :, t, None] - (S * kt).sum(-2, keepdim=True))
        outs.append((S * q[:, :, t, :, None]).sum(-2))
    st["S"][at] = S
    out = _gather(torch.stack(outs, 2), size, place).to(st["q"].dtype)
    return {"out": out, "states": st["S"]}


def _plain_packed(st):
    case = st["case"]
    H, d, b = case["heads"], case["d"], case["bits"]
    slots = st["slots"].long()
    total = st["pool"].numel() // (H * (-(-(d * d * b // 8 + 4 * d) // 256) * 256))
    seg = st["pool"].reshape(total, -1)
    S = _values(*_unpack(seg[slots], len(slots), H, d, b))
    out, S = _plain_forward(st, *(st[x].float() for x in ("q", "k", "v", "alpha", "beta")), S)
    z, r, c = _requantise(S, st["omega"], b)
    # a sequence without tokens leaves its slot as it was
    some = torch.tensor([x > 0 for x in st["lens"]], device=slots.device)
    new = _pack(z, r, c, b).reshape(len(slots), -1)
    seg[slots] = torch.where(some[:, None], new, seg[slots])
    back = _values(*_unpack(seg[slots], len(slots), H, d, b))
    return {"out": out.to(st["q"].dtype), "states": back.to(st["q"].dtype if b <= 8 and st["q"].dtype != torch.float32 else torch.bfloat16)}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    op, n, H, d = case["op"], case["seqs"], case["heads"], case["d"]
    if not own:
        if op == "forward":
            out, S = _plain_forward(st, *(st[x].float() for x in ("q", "k", "v")), st["alpha"], st["beta"], st["S"])
            return {"out": out.to(st["q"].dtype), "state": S}
        return {"backward": _plain_backward, "step": _plain_step, "packed": _plain_packed}[op](st)
    from quantized_delta_rule_amd import delta
    args = [st[x] for x in ("q", "k", "v", "alpha", "beta")]
    how = dict(cu_seqlens=st["cu"]) if st["cu"] is not None else dict(n_seqs=n)
    empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=st["q"].device)  # noqa: E731
    if op == "forward":
        out, state = torch.empty_like(st["v"]), empty(n, H, d, d)
        delta.forward(*args, out, state_in=st["S"], state_out=state, **how)
        return {"out": out, "state": state}
    if op == "backward":
        g = {"d" + x: torch.empty_like(st[x]) for x in ("q", "k", "v", "alpha", "beta")}
        if st["S"] is not None:
            g["dstate"] = torch.empty_like(st["S"])
        delta.backward(*args, st["d_out"], g["dq"], g["dk"], g["dv"], g["dalpha"], g["dbeta"],
                       state_in=st["S"], d_state_out=st["d_state"], d_state_in=g.get("dstate"), **how)
        return g
    out = torch.empty_like(st["v"])
    if op == "step":
        kind = delta.GDN if case["kind"] == "gdn" else delta.KDA
        order = delta.DELTA_FIRST if case["kind"] == "kda" else delta.DECAY_FIRST
        delta.forward(*args, out, state_in=st["S"], state_out=st["S"], slots=st["slots"], kind=kind,
                      order=order, **how)
        return {"out": out, "states": st["S"]}
    plan, total = st["plan"], st["pool"].numel() // st["plan"].bytes_per_request
    plan.prefill_slots(st["pool"], total, st["slots"], *args, out, **how)
    back = empty(n, H, d, d, dtype=torch.bfloat16 if out.dtype == torch.float32 else out.dtype)
    plan.read_slots(st["pool"], total, st["slots"], n, back)
    return {"out": out, "states": back}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, token by token
# ---------------------------------------------------------------------------------------------

def _one(S, q, k, v, a, b, delta_first):
    """One token of every sequence and head: S [.., d, d], q, k, v [.., d], a [.., d or 1], b [..]."""
    if delta_first:
        u = torch.matmul(k[..., None, :], S)
        S = a[..., None] * (S - b[..., None, None] * k[..., None] * u) + b[..., None, None] * k[..., None] * v[..., None, :]
    else:
        S = a[..., None] * S
        e = v - torch.matmul(k[..., None, :], S)[..., 0, :]
        S = S + (b[..., None] * k)[..., None] * e[..., None, :]
    return S, torch.matmul(q[..., None, :], S)[..., 0, :]


def _whole(st):
    """Every input as [n, H, longest, ..] in 64 bits."""
    case, lens = st["case"], st["lens"]
    n, grp, most = case["seqs"], case["heads"] // case["qk_heads"], max(lens)
    dev = st["q"].device
    got = {}
    for name in ("q", "k", "v", "alpha", "beta", "d_out"):
        if name not in st:
            continue
        x = st[name].double()
        if name in ("q", "k"):
            x = x.repeat_interleave(grp, 1)
        y = torch.full((n, most) + tuple(x.shape[1:]), 1.0 if name == "alpha" else 0.0, dtype=torch.float64, device=dev)
        at = 0
        for i, ln in enumerate(lens):
            y[i, :ln] = x[at:at + ln]
            at += ln
        got[name] = y.transpose(1, 2)
    if got["alpha"].dim() == 3:
        got["alpha"] = got["alpha"][..., None]
    return got, most


def _tokens(y, lens):
    return torch.cat([y[i, :, :ln].transpose(0, 1) for i, ln in enumerate(lens)])


def exact(case, seed):
    st = prepare(case, seed)
    x, most = _whole(st)
    n, H, d, lens = case["seqs"], case["heads"], case["d"], st["lens"]
    first = case.get("kind") == "kda"
    if most * n * H * d * d * 8 * (60 if case["op"] == "backward" else 12) > 4e13:
        return None  # too long token by token
    tok = lambda t: [x[m][:, :, t] for m in ("q", "k", "v", "alpha", "beta")]  # noqa: E731
    if case["op"] == "step":
        S = st["S"].double()[st["slots"].long()]
    elif case["op"] == "packed":
        b = case["bits"]
        total = len(st["pool"]) // (H * (-(-(d * d * b // 8 + 4 * d) // 256) * 256))
        z, r, c = _unpack(st["pool"], total, H, d, b)
        S = (r.double()[..., None] * c.double()[..., None, :] * z.double())[st["slots"].long()]
    elif st["S"] is not None:
        S = st["S"].double()
    else:
        S = torch.zeros(n, H, d, d, dtype=torch.float64, device=st["q"].device)
    if case["op"] == "backward":
        return _exact_backward(st, x, S, most, tok)
    begin = S
    outs = []
    for t in range(most):
        S, o = _one(S, *tok(t), first)
        outs.append(o)
    out = _tokens(torch.stack(outs, 2), lens)
    if case["op"] == "forward":
        return {"out": out, "state": S}
    if case["op"] == "step":
        whole = st["S"].double()
        whole[st["slots"].long()] = S
        return {"out": out, "states": whole}
    # the pool's states, requantised by the definition; a slot without tokens keeps what it held
    qmax, om = 2 ** (case["bits"] - 1) - 1, st["omega"].double()
    row = ((S.abs().sum(-1) / d + 1e-8) / (1 + om / (om.sum(-1, keepdim=True) / d))).half().double()
    y = S / row[..., None]
    col = y.abs().max(-2).values / qmax
    z = torch.round(y / col[..., None, :])
    wz = (om * row ** 2)[..., None] * z
    col = ((wz * y).sum(-2) / (wz * z).sum(-2)).half().double()
    z = torch.clamp(torch.round(y / col[..., None, :]), -qmax, qmax)
    new = row[..., None] * col[..., None, :] * z
    some = torch.tensor([ln > 0 for ln in lens], device=new.device)
    return {"out": out, "states": torch.where(some[:, None, None, None], new, begin)}


def _exact_backward(st, x, S, most, tok):
    case, lens = st["case"], st["lens"]
    n, H, d, grp = case["seqs"], case["heads"], case["d"], case["heads"] // case["qk_heads"]
    piece = max(1, min(most, int(2e10 / (n * H * d * d * 8))))
    begins = []
    for t in range(most):
        if t % piece == 0:
            begins.append(S)
        S, _ = _one(S, *tok(t), False)
    G = st["d_state"].double() if st["d_state"] is not None else torch.zeros_like(S)
    got = {m: torch.zeros_like(x[m]) for m in ("q", "k", "v", "alpha", "beta")}
    dot = lambda m, w: torch.matmul(m, w[..., None])[..., 0]  # noqa: E731
    for p in range(len(begins) - 1, -1, -1):
        held, S = [], begins[p]
        for t in range(p * piece, min(most, (p + 1) * piece)):
            held.append(S)
            S, _ = _one(S, *tok(t), False)
        for t in range(min(most, (p + 1) * piece) - 1, p * piece - 1, -1):
            was = held.pop()
            q, k, v, a, b = tok(t)
            do = x["d_out"][:, :, t]
            u = torch.matmul(k[..., None, :], was)[..., 0, :]
            e = v - a * u
            now = a[..., None] * was + (b[..., None] * k)[..., None] * e[..., None, :]
            got["q"][:, :, t] = dot(now, do)
            G = G + q[..., None] * do[..., None, :]
            Ge = dot(G, e)
            de = b[..., None] * torch.matmul(k[..., None, :], G)[..., 0, :]
            got["beta"][:, :, t] = (k * Ge).sum(-1)
            got["v"][:, :, t] = de
            got["k"][:, :, t] = b[..., None] * Ge - a * dot(was, de)
            got["alpha"][:, :, t, 0] = (G * was).sum((-1, -2)) - (de * u).sum(-1)
            G = a[..., None] * (G - k[..., None] * de[..., None, :])
    r = {"d" + m: _tokens(y, lens) for m, y in got.items()}
    for m in ("dq", "dk"):
        r[m] = r[m].reshape(-1, H // grp, grp, d).sum(2)
    r["dalpha"] = r["dalpha"][..., 0]
    if st["S"] is not None:
        r["dstate"] = G
    return r
