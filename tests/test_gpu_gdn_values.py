"""GPU tests of the scalar-gate delta rule at values and sizes that a program meets seldom: a NaN among the
gates, betas near the smallest number, rows that no sequence owns, resets."""
import math

import pytest
import torch

import gdn_reference as ref
import gated_delta_rule_45_amd as kda

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
KEYS = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")


def say(*a):
    print(*a, flush=True)


def states(n, Hv, dk, dv, dtype=F32, std=0.3, seed=7):
    return (std * torch.randn(n, Hv, dk, dv, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def like(x, seed=11):
    return torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype).to(DEV)


# ---------------------------------------------------------------------------------- a NaN gate --
@pytest.mark.parametrize("io,gates", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,at", [(1, 0), (70, 3), (200, 100), (200, 199)])
def test_a_nan_gate_reaches_its_results(io, gates, T, at):
    """Wherever the definition gives a NaN, so do the kernels; other heads and sequences keep their bits."""
    say(f"[{io} gates {gates}] T={T} at {at}")
    x = ref.inputs(2, T, 2, 4, 64, 64, io, gates, seed=T, device=DEV)
    s0, dsf, do = states(2, 4, 64, 64), states(2, 4, 64, 64, seed=8), like(x[2])
    bad = [t.clone() for t in x]
    bad[3][1, at, 2] = float("nan")  # value head 2, with head 3 on key head 1
    (o, f), (ob, fb) = kda.gdn_chunk_fwd(*x, s0), kda.gdn_chunk_fwd(*bad, s0)
    assert ob[1, at:, 2].isnan().all() and fb[1, 2].isnan().all()
    assert torch.equal(ob[0], o[0]) and torch.equal(fb[0], f[0])
    for h in (0, 1, 3):
        assert torch.equal(ob[1, :, h], o[1, :, h]) and torch.equal(fb[1, h], f[1, h])
    d, db = kda.gdn_chunk_bwd(*x, do, s0, dsf), kda.gdn_chunk_bwd(*bad, do, s0, dsf)
    want = ref.delta_rule_grads(*bad, do, s0, dsf)
    assert want["dq"].isnan().any() and want["dg"].isnan().any()  # (dv not, where the gate is the first token's)
    for key in KEYS:
        lost = want[key].isnan() & ~db[key].isnan()
        assert not lost.any(), (key, int(lost.sum()))
        assert torch.equal(db[key][0], d[key][0]), key
    for key in ("dv", "dg", "dbeta"):
        for h in (0, 1, 3):
            assert torch.equal(db[key][1, :, h], d[key][1, :, h]), (key, h)
    for key in ("dq", "dk"):
        assert torch.equal(db[key][1, :, 0], d[key][1, :, 0]), key
    # and the recurrent form agrees
    pool, pool_b = s0.clone(), s0.clone()
    y, yb = kda.gdn_decode(*x, pool), kda.gdn_decode(*bad, pool_b)
    assert yb[1, at:, 2].isnan().all() and pool_b[1, 2].isnan().all()
    assert torch.equal(yb[1, :, 3], y[1, :, 3]) and torch.equal(pool_b[0], pool[0])


@pytest.mark.parametrize("io", [BF, F32])
def test_a_nan_gate_in_a_split_walk(io):
    T, at = 8192, 5000
    start = at - at % (64 if io == BF else 32)
    x = ref.inputs(1, T, 1, 2, 64, 64, io, F32, seed=3, device=DEV)
    x[3].mul_(0.05)
    do = like(x[2])
    o, f = kda.gdn_chunk_fwd(*x)
    d = kda.gdn_chunk_bwd(*x, do)
    x[3][0, at, 1] = float("nan")
    ob, fb = kda.gdn_chunk_fwd(*x)
    assert ob[0, at:, 1].isnan().all() and fb[0, 1].isnan().all()
    assert torch.equal(ob[0, :start, 1], o[0, :start, 1])
    assert torch.equal(ob[0, :, 0], o[0, :, 0]) and torch.equal(fb[0, 0], f[0, 0])
    db = kda.gdn_chunk_bwd(*x, do)
    assert db["dg"][0, :at + 1, 1].isnan().all() and db["dv"][0, :at + 1, 1].isnan().all()
    assert db["dq"][0, at:].isnan().all() and db["d_initial_state"][0, 1].isnan().all()
    for key in ("dv", "dg", "dbeta"):
        assert torch.equal(db[key][0, :, 0], d[key][0, :, 0]), key


# ------------------------------------------------------------------------------- tiny betas --
def close(name, got, want, rel2):
    g, w = got.double(), want.double()
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    r2 = float((g - w).norm() / w.norm())
    say(f"  {name}: rel2={r2:.2e}")
    assert r2 <= rel2, f"{name}: rel2 {r2:.3e} > {rel2}"


@pytest.mark.parametrize("io,gates", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T", [60, 300])
@pytest.mark.parametrize("tiny", [2.0 ** -63, 2.0 ** -65, 1e-30, 1e-37, 1e-38, 1e-40])
def test_a_tiny_beta_has_its_gradient(io, gates, T, tiny):
    """dbeta does not depend on how small its own beta is: what a token with beta near the smallest normal number
    (or below it) would have written is weighed as for beta = 0.  Bounds as for the other gradients (nine
    roundings to bf16, 256 fp32 terms)."""
    say(f"[{io} gates {gates}] T={T} beta={tiny:.2g}")
    x = ref.inputs(1, T, 2, 4, 64, 64, io, gates, seed=5, device=DEV)
    x[4][:, ::3] = tiny
    s0, dsf, do = states(1, 4, 64, 64), states(1, 4, 64, 64, seed=8), like(x[2])
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf), ref.delta_rule_grads(*x, do, s0, dsf)
    bound = 8e-3 if io == BF or gates == BF else 1.5e-5
    for key in KEYS:
        close(key, got[key], want[key], bound)
    close("dbeta of the tiny ones", got["dbeta"][:, ::3], want["dbeta"][:, ::3], 2e-2 if io == BF else bound)
    x[4].fill_(tiny)
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf), ref.delta_rule_grads(*x, do, s0, dsf)
    close("dbeta, all tiny", got["dbeta"], want["dbeta"], bound)


# ------------------------------------------------------------------ rows that no sequence owns --
@pytest.mark.parametrize("gates", [BF, F32])
def test_rows_of_a_small_packed_batch_that_no_sequence_owns_are_left_alone(gates):
    """As for larger batches (few gates: bf16 gradients on fp32 operands)."""
    lens, extra = [20, 0, 3, 40], 17
    n = sum(lens)
    x = ref.inputs(1, n + extra, 2, 4, 64, 64, BF, gates, seed=14, device=DEV)
    do = like(x[2])
    for t in (*x, do):
        t[:, n:] = float("nan")
    cu = ref.packed(lens, DEV)
    out = {k: torch.full_like(t, 7.0) for k, t in zip(KEYS, x)} | {"d_initial_state": None}
    room = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)  # NaN whatever the type
    got = kda.gdn_chunk_bwd(*x, do, None, None, cu, need_d_initial_state=False, out=out, workspace=room)
    alone = kda.gdn_chunk_bwd(*[t[:, :n].contiguous() for t in x], do[:, :n].contiguous(), None, None, cu)
    for key in KEYS[:5]:
        assert torch.equal(got[key][:, :n], alone[key]), key
        assert (got[key][:, n:] == 7).all(), key


# -------------------------------------------------------------------------------- resets --
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T", [60, 150])
def test_gradients_at_resets(io, T):
    """g = -inf forgets what came before: dg is 0 there, not what is left of sums that cancel."""
    say(f"[{io}] T={T}")
    x = ref.inputs(1, T, 2, 4, 128, 128, io, F32, seed=9, device=DEV)
    at = [t for t in (0, 5, 31, 63, 64, 100) if t < T]
    x[3][:, at] = -math.inf
    s0, dsf, do = states(1, 4, 128, 128), states(1, 4, 128, 128, seed=8), like(x[2])
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf), ref.delta_rule_grads(*x, do, s0, dsf)
    assert (want["dg"][:, at] == 0).all() and (want["d_initial_state"] == 0).all()
    for key in KEYS[:5]:
        close(key, got[key], want[key], 8e-3 if io == BF else 1.5e-5)
    say("  dg at the resets:", float(got["dg"][:, at].abs().max()), "of", float(want["dg"].abs().max()))
    assert (got["dg"][:, at] == 0).all() and (got["d_initial_state"] == 0).all()


# ------------------------------------------------------------------------ the shortest split walk --
@pytest.mark.parametrize("T,split", [(224, False), (225, True), (255, True)])
def test_the_binding_gives_room_to_every_split(T, split):
    x = ref.inputs(1, T, 1, 2, 64, 64, F32, seed=T, device=DEV)
    s0 = states(1, 2, 64, 64)
    room = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    a, b = kda.gdn_chunk_fwd(*x, s0), kda.gdn_chunk_fwd(*x, s0, workspace=room)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, f = ref.delta_rule(*x, s0)
    close("out", a[0], o, 1.5e-5)
    close("final", a[1], f, 1.5e-5)
    one = kda.gdn_chunk_fwd(*x, s0, workspace=room[:0])
    assert torch.equal(one[0], a[0]) != split  # two ways of summing
