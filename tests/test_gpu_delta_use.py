"""The sequence calls as programs use them: strided rows, equal lengths, slots, offsets that break the
rule, NaN beside and between sequences, streams, two calls at once, captured graphs, lengths of zero, rows
past 4 GiB, and the whole of it in a row.  Values are checked against the token-by-token recurrence in
binary64 where they are new; where only the way of calling differs the results must be equal bit for bit
(the kernels add in a fixed order)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402
from test_gpu_delta import BF16, F16, F32, OUT, STATE  # noqa: E402
from test_gpu_prefill import _filled, _plan  # noqa: E402

GRADS = ("dq", "dk", "dv", "dalpha", "dbeta", "dS")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from quantized_delta_rule_amd import delta, stepq
    return stepq, delta


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(lens, K, H, d, dtype, seed=3, kda=False, first=0, last=0):
    cu = R.offsets(lens, first)
    x = R.inputs(seed, cu[-1] + last, K, H, d, len(lens), dtype, kda=kda)
    return {m: t.cuda() for m, t in x.items()}, cu


def _forward(delta, g, cu=None, **kw):
    out = torch.full(g["v"].shape, 55.0, dtype=g["v"].dtype, device="cuda")
    S = torch.full_like(g["S"], 55.0)
    if cu is not None:
        kw["cu_seqlens"] = cu if isinstance(cu, torch.Tensor) else _ints(cu)
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=g["S"], state_out=S, **kw)
    return out, S


def _backward(delta, g, cu=None, into=None, **kw):
    o = into or dict(dq=torch.full_like(g["q"], 55.0), dk=torch.full_like(g["k"], 55.0),
                     dv=torch.empty(g["v"].shape, dtype=g["v"].dtype, device="cuda").fill_(55.0),
                     dalpha=torch.full_like(g["alpha"], 55.0), dbeta=torch.full_like(g["beta"], 55.0),
                     dS=torch.full_like(g["S"], 55.0))
    if cu is not None:
        kw["cu_seqlens"] = cu if isinstance(cu, torch.Tensor) else _ints(cu)
    delta.backward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["do"], o["dq"], o["dk"], o["dv"],
                   o["dalpha"], o["dbeta"], state_in=g["S"], d_state_out=g["dS"], d_state_in=o["dS"], **kw)
    return o


def _same(a, b):
    if isinstance(a, dict):
        return all(torch.equal(a[m], b[m]) for m in a)
    return all(torch.equal(x, y) for x, y in zip(a, b))


# chunks, segments (few long sequences), tokens one by one, both (a long one among short ones)
PATHS = {"chunks": [70, 130, 33], "segments": [5200], "tokens": [2, 0, 5],
         "both": [150, 1, 16, 0, 15] + 11 * [1]}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strided_rows(lib, path, dtype):
    """q, k and v as parts of one projection's rows, out as a part of wider rows: equal to packed rows, and
    nothing outside out's part is written."""
    _, delta = lib
    K, H, d = 2, 4, 64
    g, cu = _case(PATHS[path], K, H, d, dtype)
    T = cu[-1]
    rows = torch.full((T, (2 * K + H) * d + 16), float("nan"), dtype=dtype, device="cuda")
    s = dict(g)
    at = 8
    for m, n in (("q", K), ("k", K), ("v", H)):
        s[m] = rows[:, at:at + n * d].view(T, n, d)
        s[m].copy_(g[m])
        at += n * d
    wide = torch.full((T, H * d + 32), 9.0, dtype=dtype, device="cuda")
    out = wide[:, 16:16 + H * d].view(T, H, d)
    S = torch.empty_like(g["S"])
    delta.forward(s["q"], s["k"], s["v"], s["alpha"], s["beta"], out, state_in=g["S"], state_out=S,
                  cu_seqlens=_ints(cu))
    assert _same(_forward(delta, g, cu), (out, S))
    assert (wide[:, :16] == 9.0).all() and (wide[:, 16 + H * d:] == 9.0).all()
    s["do"] = rows.new_full((T, H * d + 8), float("nan"))[:, 8:].view(T, H, d)
    s["do"].copy_(g["do"])
    ref = _backward(delta, g, cu)
    assert _same(ref, _backward(delta, s, cu, into={m: torch.empty_like(ref[m]) for m in ref}))


@pytest.mark.parametrize("kind", ["state", "no state"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [PATHS["both"], [3] * 30 + [257] + [7] * 20, [1] * 200 + [16, 129, 15]], ids=len)
def test_decoding_and_prompts_in_one_call(lib, lens, dtype, d, kind):
    """Short sequences go token by token and long ones in chunks, each against binary64."""
    _, delta = lib
    cu = R.offsets(lens)
    assert cu[-1] < 16 * len(lens) and cu[-1] - len(lens) >= 128  # both paths
    x = R.inputs(21 + d, cu[-1], 1, 2, d, len(lens), dtype)
    if kind != "state":
        x["S"].zero_()
    g = {m: t.cuda() for m, t in x.items()}
    out, S = torch.empty_like(g["v"]), torch.empty_like(g["S"])
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=g["S"] if kind == "state" else None,
                  state_out=S, cu_seqlens=_ints(cu))
    want, wantS = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S"], cu)
    # Every sequence by itself: a long one must not hide a short one.  Relative to the outputs alone there is
    # no bound: one token from the zero state has o = beta (k.q) v, and a binary32 sum errs by up to d 2^-24
    # sum |k_i q_i| <= d 2^-24 (unit k, q) however small k.q is -- 7.6e-6 beta |v| at d = 128, with |S| = beta |v|.
    # So the states' share counts from the states: STATE |S| for each of the len tokens (|q| = 1).
    for n in range(len(lens)):
        if lens[n]:
            o, w = out[cu[n]:cu[n + 1]].double().cpu(), want[cu[n]:cu[n + 1]]
            bound = 2 * OUT[dtype] * float(w.norm()) + STATE * lens[n] ** 0.5 * float(wantS[n].norm())
            assert float((o - w).norm()) <= bound, n
    assert R.rel(out, want) <= OUT[dtype] and R.rel(S, wantS) <= STATE


@pytest.mark.parametrize("N,L", [(3, 70), (5, 1), (1, 1024), (4, 0)])
def test_equal_lengths_without_offsets(lib, N, L):
    _, delta = lib
    g, cu = _case([L] * N, 1, 2, 64, BF16)
    want = _forward(delta, g, cu)
    assert _same(want, _forward(delta, g, n_seqs=N))
    if N == 1:
        assert _same(want, _forward(delta, g))
    if L == 0:
        assert torch.equal(want[1], g["S"])
    assert _same(_backward(delta, g, cu), _backward(delta, g, n_seqs=N))


@pytest.mark.parametrize("lens", [[0, 0], []], ids=str)
def test_no_tokens(lib, lens):
    _, delta = lib
    g, cu = _case(lens, 1, 2, 128, F16)
    out, S = _forward(delta, g, cu)
    assert torch.equal(S, g["S"])
    o = _backward(delta, g, cu)
    assert torch.equal(o["dS"], g["dS"])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("kda", [False, True])
def test_slots(lib, path, kda):
    """States by slot, in place: -1 and out-of-range slots leave rows and states as they were, the latter
    raise the flag; the rest equals a call on gathered states."""
    stepq, delta = lib
    if kda and path == "segments":
        pytest.skip("KDA has one path")
    lens = {"segments": [7800], "both": [1, 150, 3, 16] + 12 * [1]}.get(path, PATHS[path]) + [40, 20]
    kind = delta.KDA if kda else delta.GDN
    g, cu = _case(lens, 2, 2, 64, BF16, kda=kda)
    n, N = 20, len(lens)
    pool = torch.randn(n, 2, 64, 64, device="cuda")
    pick = list(range(n - 1, n - 1 - N, -1))
    pick[-2], pick[-1] = -1, n  # skip, out of range
    g["S"] = torch.stack([pool[s] if 0 <= s < n else torch.zeros_like(pool[0]) for s in pick])
    out, S = _forward(delta, g, cu, kind=kind)
    was, status = pool.clone(), _ints([0])
    o2 = torch.full_like(out, 55.0)
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], o2, state_in=pool, state_out=pool,
                  cu_seqlens=_ints(cu), slots=_ints(pick), kind=kind, status=status)
    end = cu[N - 2]
    assert torch.equal(o2[:end], out[:end]) and (o2[end:] == 55.0).all()
    for s in range(n):
        want = S[pick.index(s)] if s in pick[:-2] else was[s]
        assert torch.equal(pool[s], want), s
    assert int(status) == stepq.FLAG_BAD_SLOT


@pytest.mark.parametrize("path", PATHS)
def test_broken_offsets_skip_their_sequence(lib, path):
    stepq, delta = lib
    g, cu = _case(PATHS[path] + [{"tokens": 20, "both": 30}.get(path, 64)], 1, 2, 64, BF16)
    N, T = len(cu) - 1, cu[-1]
    want = _forward(delta, g, cu)
    grads = _backward(delta, g, cu)
    for bad in (T + 1, -1, cu[N - 1] - 1, 2 ** 31 - 1, -2 ** 31):
        status, off = _ints([0]), list(cu)
        off[N] = bad  # the last sequence's end
        out, S = _forward(delta, g, off, status=status)
        end = cu[N - 1]
        assert int(status) == stepq.FLAG_BAD_SEQ
        assert torch.equal(out[:end], want[0][:end]) and torch.equal(S[:N - 1], want[1][:N - 1])
        assert (out[end:] == 55.0).all() and (S[N - 1] == 55.0).all()
        status.zero_()
        o = _backward(delta, g, off, status=status)
        assert int(status) == stepq.FLAG_BAD_SEQ
        for m in GRADS[:5]:
            assert torch.equal(o[m][:end], grads[m][:end]) and (o[m][end:] == 55.0).all(), m
        assert torch.equal(o["dS"][:N - 1], grads["dS"][:N - 1]) and (o["dS"][N - 1] == 55.0).all()


@pytest.mark.parametrize("path", PATHS)
def test_offsets_out_of_order_raise_the_flag(lib, path):
    """An offset in the middle that breaks the order: the flag is raised, rows of no sequence and other
    states stay, the call ends (what the other sequences hold is not specified)."""
    stepq, delta = lib
    n = 20 if path in ("tokens", "both") else 64
    g, cu = _case([n] + PATHS[path] + [n], 1, 2, 64, BF16, first=2, last=3)
    for bad in (cu[-1] + 9, -1, 2 ** 31 - 1, -2 ** 31, 0):
        status, off = _ints([0]), list(cu)
        off[1] = bad
        states = torch.full((len(cu) + 1, 2, 64, 64), 55.0, device="cuda")
        out = torch.full_like(g["v"], 55.0)
        delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_out=states,
                      cu_seqlens=_ints(off), slots=_ints(range(1, len(cu))), status=status)
        o = _backward(delta, g, off, status=status)
        assert int(status) == stepq.FLAG_BAD_SEQ
        assert (states[0] == 55.0).all() and (states[len(cu)] == 55.0).all()
        for t in [out] + [o[m] for m in GRADS[:5]]:
            assert (t[cu[-1]:] == 55.0).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_no_sequence_are_not_read(lib, path, dtype):
    """NaN and infinities in rows before, behind and between sequences, and in another sequence, stay
    there; rows of no sequence keep out and the gradients."""
    _, delta = lib
    lens = PATHS[path]
    g, cu = _case(lens + [30], 2, 4, 64, dtype, first=3, last=5)
    want, grads = _forward(delta, g, cu), _backward(delta, g, cu)
    lo, hi = cu[0], cu[len(lens)]
    h = {m: t.clone() for m, t in g.items()}
    for m in ("q", "k", "v", "alpha", "beta", "do"):
        h[m][:lo], h[m][hi:] = float("nan"), float("inf")
    h["S"][-1] = float("nan")
    out, S = _forward(delta, h, cu)
    assert torch.equal(out[lo:hi], want[0][lo:hi]) and torch.equal(S[:-1], want[1][:-1])
    assert (out[:lo] == 55.0).all() and (out[cu[-1]:] == 55.0).all()
    o = _backward(delta, h, cu)
    for m in GRADS[:5]:
        assert torch.equal(o[m][lo:hi], grads[m][lo:hi]), m
        assert (o[m][:lo] == 55.0).all() and (o[m][cu[-1]:] == 55.0).all(), m
    assert torch.equal(o["dS"][:-1], grads["dS"][:-1])


@pytest.mark.parametrize("where", ["q", "k", "v", "alpha", "beta", "S"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("path", PATHS)
def test_a_non_finite_input_shows(lib, where, what, path):
    """It reaches what the recurrence carries it to, and no other head and no earlier chunk."""
    _, delta = lib
    g, cu = _case(PATHS[path], 2, 2, 64, F32)
    want = _forward(delta, g, cu)
    t = cu[1] - 1 if path != "segments" else 700  # in the first sequence
    if where == "S":
        g["S"][0, 1, 5, 7], t = what, 0
    elif where in ("alpha", "beta"):
        g[where][t, 1] = what
    else:
        g[where][t, 1, 7] = what
    out, S = _forward(delta, g, cu)
    assert torch.equal(out[:, 0], want[0][:, 0]) and torch.equal(S[:, 0], want[1][:, 0])
    assert torch.equal(out[cu[1]:], want[0][cu[1]:]) and torch.equal(S[1:], want[1][1:])
    first = 0 if path == "tokens" else t // 64 * 64
    if path == "tokens":
        first = t
    if where != "S":
        assert torch.equal(out[:first, 1], want[0][:first, 1])
    bad = ~torch.isfinite(out[t, 1])
    assert bad.any()
    if where == "q":
        assert torch.isfinite(S[0, 1]).all() or path != "tokens"
    else:
        assert not torch.isfinite(S[0, 1]).all()


def test_state_gradient_in_place(lib):
    _, delta = lib
    g, cu = _case(PATHS["chunks"], 2, 4, 64, BF16)
    want = _backward(delta, g, cu)
    o = {m: torch.empty_like(t) for m, t in want.items()}
    o["dS"] = g["dS"]
    assert _same(want, _backward(delta, g, cu, into=o))


@pytest.mark.parametrize("path", PATHS)
def test_results_do_not_depend_on_the_run(lib, path):
    _, delta = lib
    g, cu = _case(PATHS[path], 1, 4, 128, BF16)
    f, b = _forward(delta, g, cu), _backward(delta, g, cu)
    for _ in range(3):
        assert _same(f, _forward(delta, g, cu)) and _same(b, _backward(delta, g, cu))


def test_streams_and_two_calls_at_once(lib):
    """Calls on two other streams at once, each with the workspace of its own that the binding takes."""
    _, delta = lib
    sets = [_case(PATHS["chunks"], 2, 4, 128, BF16, seed=s) for s in (1, 2)]
    want = [(_forward(delta, g, cu), _backward(delta, g, cu)) for g, cu in sets]
    offs = [_ints(cu) for _, cu in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (g, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):  # the current stream
                got[i].append((_forward(delta, g, offs[i]), _backward(delta, g, offs[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for f, b in got[i]:
            assert _same(f, want[i][0]) and _same(b, want[i][1])
    # a stream as an argument
    g, _ = sets[0]
    out, S = torch.empty_like(g["v"]), torch.empty_like(g["S"])
    torch.cuda.synchronize()
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=g["S"], state_out=S,
                  cu_seqlens=offs[0], stream=streams[1])
    streams[1].synchronize()
    assert _same((out, S), want[0][0])


@pytest.mark.parametrize("path", PATHS)
def test_captured_graphs(lib, path):
    """Forward and backward captured once and replayed with new inputs in place, eager calls between the
    replays; two graphs with a workspace each."""
    _, delta = lib
    g, cu = _case(PATHS[path], 2, 4, 64, BF16)
    c = _ints(cu)
    need = delta.forward_workspace(g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["v"], cu_seqlens=c)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    _forward(delta, g, c)
    torch.cuda.synchronize()
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out, S = torch.empty_like(g["v"]), torch.empty_like(g["S"])
    with torch.cuda.graph(gf):
        delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_in=g["S"], state_out=S,
                      cu_seqlens=c, workspace=ws)
    o = {m: torch.empty_like(t) for m, t in dict(dq=g["q"], dk=g["k"], dv=g["v"], dalpha=g["alpha"],
                                                 dbeta=g["beta"], dS=g["S"]).items()}
    need = delta.backward_workspace(g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["do"], cu_seqlens=c)
    wb = torch.empty(need, dtype=torch.uint8, device="cuda") if path == "chunks" else None
    with torch.cuda.graph(gb):
        _backward(delta, g, c, into=o, workspace=wb)  # None: from the graph's own pool
    for i in range(4):
        for m in ("q", "k", "v", "do", "S"):
            g[m].copy_(torch.roll(g[m], 1, 0))
        gf.replay()
        gb.replay()
        torch.cuda.synchronize()
        assert _same((out, S), _forward(delta, g, c)), i
        assert _same(o, _backward(delta, g, c)), i


def test_prefill_and_read_captured(lib):
    stepq, delta = lib
    plan = _plan(stepq, "gdn", 64, 4)
    g, cu = _case([70, 3], 4, 4, 64, BF16)
    pool = _filled(plan, 4)
    ref, c, pick = pool.clone(), _ints(cu), _ints([3, 1])
    out, S = torch.empty_like(g["v"]), torch.empty(2, 4, 64, 64, dtype=BF16, device="cuda")
    o2, S2 = torch.empty_like(out), torch.empty_like(S)

    need = plan.prefill_workspace(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, cu_seqlens=c)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(pool, out, S):
        plan.prefill_slots(pool, 4, pick, g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, cu_seqlens=c,
                           workspace=ws)
        plan.read_slots(pool, 4, pick, 2, S)
    run(pool.clone(), out, S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(pool, out, S)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        run(ref, o2, S2)
        torch.cuda.synchronize()
        assert torch.equal(pool, ref) and torch.equal(out, o2) and torch.equal(S, S2), i
    split = _plan(stepq, "gdn", 64, 4, mode=stepq.SPLIT)
    for call in ("prefill_slots", "read_slots"):
        graph, err = torch.cuda.CUDAGraph(), None
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):  # the refused call enqueues nothing: the capture ends empty
            try:
                if call == "read_slots":
                    split.read_slots(pool, 4, pick, 2, S)
                else:
                    split.prefill_slots(pool, 4, pick, g["q"], g["k"], g["v"], g["alpha"], g["beta"], out,
                                        cu_seqlens=c, workspace=ws)
            except stepq.StepqError as e:
                err = e
        assert err is not None and call in str(err) and "capturing stream" in str(err), err


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("kind,order", [("gdn", 0), ("kda", 0), ("kda", 1)])
def test_prompt_decode_read_and_go_on(lib, kind, order, mode):
    """The operators in a row: prompts into a packed pool, steps on it, its values read back, and the
    recurrence continued on FP32 states, each against the recurrence in binary64 from what the pool
    held before."""
    stepq, delta = lib
    H, d, n = 4, 64, 6
    plan = _plan(stepq, kind, d, H, mode=mode, order=order)
    kda, first = kind == "kda", bool(order) or kind == "gdn"
    lens, pick = [70, 130], _ints([4, 1])
    g, cu = _case(lens, H, H, d, BF16, kda=kda)
    x = {m: t.cpu() for m, t in g.items()}
    pool = plan.alloc_pool(n)
    pool.zero_()
    out = torch.empty_like(g["v"])
    plan.prefill_slots(pool, n, pick, g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, cu_seqlens=_ints(cu))
    want, S = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], torch.zeros(2, H, d, d), cu, first)
    assert R.rel(out, want) <= OUT[BF16]
    t = R.inputs(9, 2, H, H, d, 2, F32, kda=kda)
    s = {m: v.cuda() for m, v in t.items()}
    held = torch.empty(2, H, d, d, device="cuda")
    for _ in range(3):
        plan.read_slots(pool, n, pick, 2, held)
        one = torch.empty(2, H, d, device="cuda")
        plan.step_slots(pool, n, pick, 2, s["q"], s["k"], s["v"], s["alpha"], s["beta"], one)
        want, _ = R.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], held.cpu(), [0, 1, 2], first)
        assert R.rel(one, want) <= 2 * STATE
    plan.read_slots(pool, n, pick, 2, held)
    S0 = held.cpu()
    o2 = torch.empty(2, H, d, device="cuda")
    delta.forward(s["q"], s["k"], s["v"], s["alpha"], s["beta"], o2, state_in=held, state_out=held,
                  n_seqs=2, kind=plan.kind, order=order)
    want, S1 = R.run(t["q"], t["k"], t["v"], t["alpha"], t["beta"], S0, [0, 1, 2], first)
    assert R.rel(o2, want) <= STATE and R.rel(held, S1) <= STATE
    assert plan.status() == 0


def test_rows_past_four_gib(lib):
    """q, k, v, out and the workspace longer than 2^32 bytes: the last 1,000 tokens, whose first gate is
    zero, equal those tokens alone up to the roundings of either."""
    _, delta = lib
    T, K, H, d, tail = 300_032, 8, 64, 128, 1000
    torch.cuda.empty_cache()
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, dtype=BF16, device="cuda", generator=gen)  # noqa: E731
    g = dict(q=r(T, K, d).mul_(d ** -0.5), k=r(T, K, d).mul_(d ** -0.5), v=r(T, H, d),
             alpha=0.9 + 0.1 * torch.rand(T, H, device="cuda", generator=gen),
             beta=torch.rand(T, H, device="cuda", generator=gen))
    assert g["v"].numel() * 2 > 2 ** 32
    g["alpha"][T - tail] = 0.0
    out, S = torch.empty_like(g["v"]), torch.empty(1, H, d, d, device="cuda")
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], out, state_out=S)
    e = {m: t[T - tail:].clone() for m, t in g.items()}
    o2, S2 = torch.empty_like(e["v"]), torch.empty_like(S)
    delta.forward(e["q"], e["k"], e["v"], e["alpha"], e["beta"], o2, state_out=S2)
    assert R.rel(out[T - tail:], o2) <= 2 * OUT[BF16]
    assert R.rel(S, S2) <= 2 * STATE


def test_python_refusals(lib):
    """Wrong types, shapes, devices and strides are refused before anything is enqueued."""
    stepq, delta = lib
    g, cu = _case([70, 33], 2, 4, 64, BF16)
    out = torch.full_like(g["v"], 55.0)
    S = torch.full_like(g["S"], 55.0)

    def call(error, match, **kw):
        x = dict(g, out=out, state_in=g["S"], state_out=S, cu_seqlens=_ints(cu))
        x.update(kw)
        args = [x.pop(m) for m in ("q", "k", "v", "alpha", "beta", "out")]
        with pytest.raises(error, match=match):
            delta.forward(*args, **{m: x[m] for m in x if m not in ("S", "do", "dS")})

    call(TypeError, "k must be a torch tensor", k=None)
    call(TypeError, "k must be torch.bfloat16", k=g["k"].float())
    call(ValueError, "k must live on cuda:0", k=g["k"].cpu())
    call(ValueError, "k must be", k=g["k"][:-1])
    call(ValueError, "alpha must be", alpha=g["beta"][:, :-1])
    call(ValueError, "alpha must be contiguous", alpha=g["alpha"].t().contiguous().t())
    call(ValueError, "alpha must be", kind=delta.KDA)
    call(ValueError, "heads of a token must be packed", q=g["q"].transpose(0, 1).contiguous().transpose(0, 1))
    call(ValueError, "tokens must not overlap", q=g["q"][:1].expand_as(g["q"]))
    call(stepq.StepqError, "q_stride", q=torch.zeros(103, 2 * 64 + 4, dtype=BF16, device="cuda")[:, :128].view(103, 2, 64))
    call(stepq.StepqError, "16-byte aligned", q=torch.zeros(103 * 128 + 1, dtype=BF16, device="cuda")[1:].view(103, 2, 64))
    call(stepq.StepqError, "multiple of n_qk_heads", q=torch.zeros(103, 3, 64, dtype=BF16, device="cuda"),
         k=torch.zeros(103, 3, 64, dtype=BF16, device="cuda"))
    call(ValueError, "n_seqs is 3", n_seqs=3)
    call(TypeError, "cu_seqlens must be torch.int32", cu_seqlens=_ints(cu).long())
    call(stepq.StepqError, "multiple of n_seqs", cu_seqlens=None, n_seqs=2)
    call(ValueError, "state_out must be", state_out=S[:1])
    call(ValueError, "state_in must be", state_in=g["S"][:1])
    call(ValueError, "slots must be", slots=_ints([0]))
    call(ValueError, "slots need", slots=_ints([0, 1]), state_in=None, state_out=None)
    call(stepq.StepqError, "workspace of 256 bytes", workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    call(stepq.StepqError, "256-byte aligned", workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[16:])
    with pytest.raises(ValueError, match="dbeta must be"):
        delta.backward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["do"], g["q"].clone(), g["k"].clone(),
                       g["v"].clone(), g["alpha"].clone(), g["beta"][:-1].clone())
    plan = _plan(stepq, "gdn", 64, 5)
    pool = _filled(plan, 3)
    was = pool.clone()
    with pytest.raises(ValueError, match="plan's heads"):
        plan.prefill_slots(pool, 3, _ints([0, 1]), g["q"], g["k"], g["v"], g["alpha"], g["beta"], out,
                           cu_seqlens=_ints(cu))
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        plan.read_slots(pool, 3, _ints([0]), 1, torch.empty(1, 5, 64, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="S has"):
        plan.read_slots(pool, 3, _ints([0]), 1, torch.empty(1, 4, 64, 64, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 55.0).all() and (S == 55.0).all() and torch.equal(pool, was)
