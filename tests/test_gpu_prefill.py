"""Prompts through packed pools and packed states read back by slot.

Reading is checked against the pool's debug decode (r, c, z as stored): r c z is one exact product, so the
binary32 values are equal and the 16-bit ones are their roundings.  A prompt pass is checked in three
steps that share no arithmetic with it: the recurrence in binary64 from the states the pool held, the
outputs against that, and the packed result against encoding the sequence call's own last states (the same
refit kernel on the same binary32 states: equal bytes)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import deltalib as R  # noqa: E402
from test_gpu_delta import BF16, F16, F32, OUT  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from quantized_delta_rule_amd import delta, stepq
    return stepq, delta


def _plan(stepq, kind, d, H, seed=0, mode=0, order=0, max_batch=16):
    g = np.random.default_rng(seed + d)
    om = (0.2 + g.random((H, d))).astype(np.float32)
    piv = np.zeros((H, d), np.uint8)
    if kind == "gdn":
        bits = np.repeat(np.array([2, 4, 6, 8] * H, np.int8)[:H, None], d, 1)
        piv[H - 1] = 1  # an FP16 pivot head
    else:
        bits = g.choice([2, 4, 6, 8], size=(H, d)).astype(np.int8)
        piv[0, [0, 5, d - 1]] = 1
    k = stepq.GDN if kind == "gdn" else stepq.KDA
    return stepq.Plan(k, bits, piv, om, mode=mode, max_batch=max_batch, order=order)


def _filled(plan, n_slots, seed=1):
    g = torch.Generator().manual_seed(seed)
    S = 0.3 * torch.randn(n_slots, plan.H, plan.d, plan.d, generator=g)
    pool = plan.alloc_pool(n_slots)
    plan.encode(S.cuda(), pool, n_slots)
    return pool


def _slots(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("kind", ["gdn", "kda"])
@pytest.mark.parametrize("d", [64, 128])
def test_read_slots(lib, kind, d, mode):
    stepq, _ = lib
    plan = _plan(stepq, kind, d, 5, mode=mode)
    pool = _filled(plan, 7)
    whole = plan.unpack(pool, 7)[0].reshape(7, 5, d, d)
    pick = [6, -1, 0, 3, 9]
    for dt in (F32, BF16, F16):
        S = torch.full((5, 5, d, d), 77.0, dtype=dt, device="cuda")
        plan.read_slots(pool, 7, _slots(pick), 5, S)
        for b, s in enumerate(pick):
            want = whole[s].to(dt) if 0 <= s < 7 else torch.full_like(S[b], 77.0)
            assert torch.equal(S[b], want), (dt, b, s)
    assert plan.status(reset=True) == stepq.FLAG_BAD_SLOT


@pytest.mark.parametrize("kind,order", [("gdn", 0), ("kda", 0), ("kda", 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_prefill_slots(lib, kind, order, d, dtype):
    stepq, delta = lib
    H, n_slots, lens, pick = 5, 8, [70, 0, 1, 33, 20], [7, 2, 5, 0, -1]
    plan = _plan(stepq, kind, d, H, order=order)
    pool = _filled(plan, n_slots)
    pool.view(n_slots, -1)[5].zero_()  # a cleared slot is the zero state
    before, was = pool.clone(), plan.unpack(pool, n_slots)[0].reshape(n_slots, H, d, d)
    cu = R.offsets(lens)
    x = R.inputs(17 + d, cu[-1], H, H, d, 5, dtype, kda=kind == "kda")
    g = {m: t.cuda() for m, t in x.items()}
    c = _slots(cu)
    out = torch.full(g["v"].shape, 55.0, dtype=dtype, device="cuda")
    plan.prefill_slots(pool, n_slots, _slots(pick), g["q"], g["k"], g["v"], g["alpha"], g["beta"], out,
                       cu_seqlens=c)
    # the skipped sequence keeps its rows, unused and empty slots keep their bytes
    assert (out[cu[4]:] == 55.0).all()
    changed = [not torch.equal(a, b) for a, b in zip(pool.view(n_slots, -1), before.view(n_slots, -1))]
    assert changed == [s in (7, 5, 0) for s in range(n_slots)]
    assert float(was[5].abs().max()) == 0.0
    S0 = torch.stack([was[s] if s >= 0 else torch.zeros_like(was[0]) for s in pick])
    want, _ = R.run(x["q"], x["k"], x["v"], x["alpha"], x["beta"], S0.cpu(), cu, bool(order) or kind == "gdn")
    assert R.rel(out[:cu[4]], want[:cu[4]]) <= OUT[dtype]
    S1, o2 = torch.empty_like(S0), torch.empty_like(out)
    delta.forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], o2, state_in=S0.contiguous(), state_out=S1,
                  cu_seqlens=c, kind=plan.kind, order=order)
    assert torch.equal(o2[:cu[4]], out[:cu[4]])
    ref = before.clone()
    plan.encode_slots(S1, ref, n_slots, _slots([7, -1, 5, 0, -1]), 5)
    assert torch.equal(ref, pool)
    assert plan.status() == 0


@pytest.mark.parametrize("mode", [0, 1])
def test_prompts_without_tokens_report_their_slots_and_offsets(lib, mode):
    """No token at all: every slot keeps its bytes, and a bad slot or bad offsets raise their flags as they do
    beside sequences with tokens."""
    stepq, _ = lib
    plan = _plan(stepq, "gdn", 64, 4, mode=mode)
    pool = _filled(plan, 3)
    was = pool.clone()
    x = {m: t.cuda() for m, t in R.inputs(1, 0, 4, 4, 64, 2, BF16).items()}
    out = torch.empty_like(x["v"])
    for cu, pick, flag in (([0, 0, 0], [1, -1], 0), ([0, 0, 0], [1, 3], stepq.FLAG_BAD_SLOT),
                           ([0, 5, 0], [1, 2], stepq.FLAG_BAD_SEQ)):
        plan.prefill_slots(pool, 3, _slots(pick), x["q"], x["k"], x["v"], x["alpha"], x["beta"], out,
                           cu_seqlens=_slots(cu))
        assert plan.status(reset=True) == flag, (cu, pick)
        assert torch.equal(pool, was)
