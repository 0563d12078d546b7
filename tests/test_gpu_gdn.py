"""GPU parity of the scalar-gate delta rule (gdn_chunk_fwd, gdn_chunk_bwd, gdn_decode) and of norm_gate_bwd
against the fp64 reference (gdn_reference.py).

Tolerances, derived before the first run.  rel2 = ||gpu - ref||_2 / ||ref||_2, relmax = max|gpu - ref| / max|ref|.
A rounding to bf16 is uniform in half a step, at most 2^-8 of the value: u = 2^-8 / sqrt(3) = 2.3e-3 in the
2-norm.  Independent roundings on a path add up in squares.
  bf16 forward: state, X, inverse, Y, P and the output: six, sqrt(6) u = 5.6e-3  -> rel2 <= 6e-3
  bf16 final states: state, X, inverse, Y (twice), the output: the same bound
  bf16 gradients: S, Z's path (three), dS's path (three), E or F, the output: nine, 3 u = 6.8e-3 -> rel2 <= 8e-3
     for tensors of at least 1,024 values; the roundings of few values do not average: rel2 <= 2e-2 for them
  relmax: 2e-2, the bar of the library's other bf16 operators
  fp32: 2^-24 per operation, at most 128 + 64 + 64 terms in a row -> 256 * 2^-24 = 1.5e-5: rel2 <= 1.5e-5,
     relmax <= 1e-4 (the bar of the library's other fp32 operators)
  A tensor stored in bf16 whatever the operands (gates' gradients beside fp32 io): its own rounding, u.
  One key repeated with beta = 1 (bf16): Y_t = v_t - v_{t-1}, of size sqrt(2) |v|, and the sums over a chunk's 64
     tokens (O, the state, dQ, dK and what follows from them) telescope to one v, so that 64 independent roundings of
     Y or Z stand against |v|: sqrt(2 * 64) u = 2.6e-2 in rel2; relmax 4 times that, the largest of some 1e4
     such sums.  Backwards dX_t = dY_t - dY_{t+1}, where dY_t sums the on average 32 tokens behind t in its chunk
     and dX_t is one of them: in squares 32 from rounding dZ, 32 from the inverse's entries (near -1), 2 * 32 from
     P's entries in both terms, 32 from M B between the 32-token blocks: sqrt(160) u = 2.9e-2; the gradients of
     beta, g and k are products of dX and Z, which carry 160 and 2 * 64 of them: sqrt(288) u = 3.8e-2
  token by token (decode): fp32 arithmetic, one rounding of a bf16 output or state: rel2 <= u = 2.3e-3 (bf16), 1.5e-5
"""
import math

import pytest
import torch

import gdn_reference as ref
import gated_delta_rule_45_amd as kda

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)


def close(name, got, want, rel2, relmax=None):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    g, w = got.double(), want.double()
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    if g.numel() == 0:
        return
    d = g - w
    n, m = float(w.norm()), float(w.abs().max())
    r2 = float(d.norm()) / n if n else float(d.norm())
    rm = float(d.abs().max()) / m if m else float(d.abs().max())
    say(f"  {name}: rel2={r2:.2e} relmax={rm:.2e}")
    assert r2 <= rel2, f"{name}: rel2 {r2:.3e} > {rel2}"
    assert relmax is None or rm <= relmax, f"{name}: relmax {rm:.3e} > {relmax}"


def tol(dtype, grad=False, n=1 << 20):
    if dtype == F32:
        return 1.5e-5, 1e-4
    return (6e-3 if not grad else 8e-3 if n >= 1024 else 2e-2), 2e-2


def state(n, Hv, dk, dv, dtype, std=0.3, seed=7):
    return (std * torch.randn(n, Hv, dk, dv, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


U = 2 ** -8 / math.sqrt(3)
TELESCOPING, TELESCOPING_BACK = ((math.sqrt(n) * U, 4 * math.sqrt(n) * U) for n in (2 * 64, 160 + 2 * 64))


def check_fwd(x, s0=None, cu=None, scale=1.0, label="", bound=None, **kw):
    say(f"[{label}] q={tuple(x[0].shape)} v={tuple(x[2].shape)} {x[0].dtype} gates={x[3].dtype}")
    out, fin = kda.gdn_chunk_fwd(*x, s0, cu, scale=scale, **kw)
    torch.cuda.synchronize()
    o, f = ref.delta_rule(*x, s0, cu, scale)
    close("out", out, o, *(bound or tol(out.dtype)))
    if fin is not None:
        # an fp32 state of a bf16 call has bf16 products behind it
        close("final", fin, f, *(bound or tol(x[0].dtype)))
    return out, fin


def check_bwd(x, s0=None, dsf=None, cu=None, scale=1.0, label="", seed=11, bound=None, **kw):
    say(f"[{label}] q={tuple(x[0].shape)} v={tuple(x[2].shape)} {x[0].dtype} gates={x[3].dtype}")
    v = x[2]
    do = torch.randn(v.shape, generator=torch.Generator().manual_seed(seed)).to(v.dtype).to(DEV)
    got = kda.gdn_chunk_bwd(*x, do, s0, dsf, cu, scale=scale, **kw)
    torch.cuda.synchronize()
    want = ref.delta_rule_grads(*x, do, s0, dsf, cu, scale)
    for key, w in want.items():
        if got[key] is not None:
            t = tol(v.dtype, True, w.numel())
            if v.dtype == F32 and got[key].dtype == BF:
                t = 2.3e-3, 2e-2
            close(key, got[key], w, *(bound or t))
    return got, do


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 31, 33, 64, 65, 130])
def test_forward_lengths_and_head_sizes(io, dk, dv, T):
    x = ref.inputs(2, T, 2, 4, dk, dv, io, seed=T + dk + 2 * dv, device=DEV)
    check_fwd(x, state(2, 4, dk, dv, F32), scale=dk ** -0.5, label=f"T{T} {dk}x{dv}")


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 7), (3, 3), (2, 8)])
@pytest.mark.parametrize("io,gates,sdt", [(BF, F32, F32), (BF, BF, BF), (F32, BF, BF), (F32, F32, F32)])
def test_forward_heads_and_types(Hk, Hv, io, gates, sdt):
    x = ref.inputs(1, 100, Hk, Hv, 64, 128, io, gates, seed=Hv, device=DEV)
    s0 = state(1, Hv, 64, 128, sdt)
    out, fin = kda.gdn_chunk_fwd(*x, s0)
    o, f = ref.delta_rule(*x, s0)
    close("out", out, o, *tol(io))
    assert fin.dtype == sdt
    close("final", fin, f, *tol(BF if sdt == BF else io))
    inplace = s0.clone()
    out2, fin2 = kda.gdn_chunk_fwd(*x, inplace, final_state=inplace)
    assert fin2 is inplace and torch.equal(out2, out) and torch.equal(inplace, fin)


LENS = [0, 1, 64, 0, 63, 130, 2, 200, 0]


@pytest.mark.parametrize("io", [BF, F32])
def test_forward_packed(io):
    x = ref.inputs(1, sum(LENS), 2, 4, 128, 128, io, seed=5, device=DEV)
    cu, s0 = ref.packed(LENS, DEV), state(len(LENS), 4, 128, 128, F32)
    out, fin = check_fwd(x, s0, cu, label="packed", cu_seqlens_host=cu.cpu())
    for i in (0, 3, 8):
        assert torch.equal(fin[i], s0[i])  # an empty sequence passes its state through
    # each sequence alone gives the same bits
    a, b = int(cu[5]), int(cu[6])
    o1, f1 = kda.gdn_chunk_fwd(*[t[:, a:b].contiguous() for t in x], s0[5:6].contiguous())
    assert torch.equal(o1, out[:, a:b]) and torch.equal(f1[0], fin[5])


def views(x, pad=0):
    """q, k, v as slices of one projection's output."""
    q, k, v = x[:3]
    parts = [t.flatten(2) for t in (q, k, v)]
    if pad:
        parts.append(torch.full((*q.shape[:2], pad), float("nan"), dtype=q.dtype, device=q.device))
    p = torch.cat(parts, -1)
    n, m = parts[0].shape[-1], parts[2].shape[-1]
    return [p[..., :n].unflatten(-1, q.shape[2:]), p[..., n:2 * n].unflatten(-1, k.shape[2:]),
            p[..., 2 * n:2 * n + m].unflatten(-1, v.shape[2:])] + list(x[3:])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,T", [(1, 77), (3, 70), (4, 1)])
def test_strided_inputs_give_the_same_bits(io, B, T):
    x = ref.inputs(B, T, 2, 4, 64, 64, io, seed=B, device=DEV)
    y = views(x, pad=16)
    assert not y[0].is_contiguous()
    for a, b in zip(kda.gdn_chunk_fwd(*x), kda.gdn_chunk_fwd(*y)):
        assert torch.equal(a, b)
    do = torch.randn_like(x[2])
    a, b = kda.gdn_chunk_bwd(*x, do), kda.gdn_chunk_bwd(*y, do)
    for key in a:
        assert torch.equal(a[key], b[key]), key
    sa, sb = state(B, 4, 64, 64, F32), state(B, 4, 64, 64, F32)
    assert torch.equal(kda.gdn_decode(*x, sa), kda.gdn_decode(*y, sb)) and torch.equal(sa, sb)


def special(case, io, T=150):
    x = ref.inputs(1, T, 2, 4, 128, 128, io, F32, seed=9, device=DEV)
    q, k, v, g, b = x
    if case == "beta0":
        b.zero_()
    if case == "some_beta0":
        b[:, ::3] = 0
    if case == "no_decay":
        g.zero_()
    if case == "strong":
        g.mul_(300)
    if case == "resets":  # e^g = 0: what came before is forgotten
        for t in (0, 5, 63, 64, 100):
            g[:, t] = -math.inf
    if case == "same_key":  # every entry below the diagonal of K K^T is 1
        k.copy_(k[:, :1].expand_as(k).clone())
        b.fill_(1.0)
        g.fill_(-1e-3)
    if case == "long_memory":
        g.fill_(-1e-4)
    return x


CASES = ["beta0", "some_beta0", "no_decay", "strong", "resets", "same_key", "long_memory"]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_forward_gates_and_keys(case, io):
    x = special(case, io)
    check_fwd(x, state(1, 4, 128, 128, F32), label=case, bound=TELESCOPING if io == BF and case == "same_key" else None)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_backward_gates_and_keys(case, io):
    x = special(case, io)
    s0, dsf = state(1, 4, 128, 128, F32), state(1, 4, 128, 128, F32, 0.1, 8)
    if case == "resets":  # the reference cannot differentiate e^-inf: a gate that is as good as one
        x[3].clamp_(min=-2000.0)
    check_bwd(x, s0, dsf, label=case, bound=TELESCOPING_BACK if io == BF and case == "same_key" else None)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 33, 64, 130])
def test_backward_lengths_and_head_sizes(io, dk, dv, T):
    # six value heads on two key heads; above 512 gates bf16 operands, below fp32 ones
    B = 4 if T == 130 else 2
    x = ref.inputs(B, T, 2, 6, dk, dv, io, seed=T + dk + 2 * dv, device=DEV)
    check_bwd(x, state(B, 6, dk, dv, io), state(B, 6, dk, dv, io, 0.1, 8), scale=dk ** -0.5, label=f"T{T} {dk}x{dv}")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("gates", [BF, F32])
def test_backward_packed(io, gates):
    lens = LENS + [257]
    x = ref.inputs(1, sum(lens), 2, 4, 128, 64, io, gates, seed=6, device=DEV)
    n = len(lens)
    dsf = state(n, 4, 128, 64, F32, 0.1, 8)
    got, _ = check_bwd(x, state(n, 4, 128, 64, F32), dsf, ref.packed(lens, DEV), label="packed")
    for i in (0, 3, 8):
        assert torch.equal(got["d_initial_state"][i], dsf[i])


def test_backward_without_states():
    x = ref.inputs(2, 90, 2, 4, 128, 128, BF, seed=12, device=DEV)
    got, do = check_bwd(x, label="no states", need_d_initial_state=False)
    assert got["d_initial_state"] is None
    again = kda.gdn_chunk_bwd(*x, do, need_d_initial_state=False)
    for key in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[key], again[key]), f"{key} does not repeat"
    # into the tensors of an earlier call
    for t in got.values():
        if t is not None:
            t.fill_(float("nan"))
    kda.gdn_chunk_bwd(*x, do, need_d_initial_state=False, out=got)
    assert torch.equal(got["dk"], again["dk"])


@pytest.mark.parametrize("io", [BF, F32])
def test_gradient_against_differences(io):
    """<gradient, direction> = d loss / d step for the library's own forward in fp32 (rounding of the
    difference: the loss is a sum of about 1e4 fp32 values, so 1e-2 of the step's effect is asked)."""
    x = [t.float() for t in ref.inputs(1, 150, 2, 4, 64, 64, io, seed=13, device=DEV)]
    s0, dsf, do = state(1, 4, 64, 64, F32), state(1, 4, 64, 64, F32, 0.1, 8), torch.randn_like(x[2])
    y = x if io == F32 else [t.to(BF) for t in x]
    d = kda.gdn_chunk_bwd(*y, do.to(io), s0, dsf)

    def loss(x):
        o, f = kda.gdn_chunk_fwd(*x, s0)
        return float((do.to(io).double() * o.double()).sum() + (dsf.double() * f.double()).sum())

    for i, key in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        step = d[key].float()
        h = 1e-2 / float(step.norm())
        up, down = [list(x), list(x)]
        up[i], down[i] = x[i] + h * step, x[i] - h * step
        num = (loss(up) - loss(down)) / (2 * h)
        want = float(step.double().square().sum())
        say(f"  {key}: {num:.6e} against {want:.6e}")
        assert abs(num - want) <= 1e-2 * abs(want), key


def test_rows_behind_the_last_sequence_are_left_alone():
    """Tokens that no sequence owns (a padded packed batch) are neither read into a result nor written."""
    lens, extra = [70, 3, 129], 60
    x = ref.inputs(1, sum(lens) + extra, 2, 4, 128, 128, BF, seed=14, device=DEV)
    for t in x:
        t[:, sum(lens):] = float("nan")
    cu = ref.packed(lens, DEV)
    y = [t[:, :sum(lens)].contiguous() for t in x]
    out = torch.full_like(x[2], 7.0)
    o, f = kda.gdn_chunk_fwd(*x, None, cu, out=out)
    o1, f1 = kda.gdn_chunk_fwd(*y, None, cu)
    assert torch.equal(o[:, :sum(lens)], o1) and torch.equal(f, f1) and (o[:, sum(lens):] == 7).all()
    do = torch.randn_like(x[2])
    do[:, sum(lens):] = float("nan")
    like = {"dq": x[0], "dk": x[1], "dv": x[2], "dg": x[3], "dbeta": x[4]}
    g = kda.gdn_chunk_bwd(*x, do, None, None, cu, out={**{n: torch.full_like(t, 7.0) for n, t in like.items()},
                                                       "d_initial_state": torch.empty_like(f)})
    g1 = kda.gdn_chunk_bwd(*y, do[:, :sum(lens)].contiguous(), None, None, cu)
    for key in like:
        assert torch.equal(g[key][:, :sum(lens)], g1[key]) and (g[key][:, sum(lens):] == 7).all(), key
    pool = state(3, 4, 128, 128, F32)
    out.fill_(7.0)
    kda.gdn_decode(*x, pool, None, cu, out=out)
    assert torch.isfinite(pool).all() and (out[:, sum(lens):] == 7).all()


def test_a_sequence_with_nan_does_not_reach_its_neighbours():
    lens = [65, 40, 70]
    x = ref.inputs(1, sum(lens), 2, 4, 64, 64, BF, seed=15, device=DEV)
    y = [t.clone() for t in x]
    for t in y:
        t[:, 65:105] = float("nan")
    cu = ref.packed(lens, DEV)
    do = torch.randn_like(x[2])
    for a, b in ((kda.gdn_chunk_fwd(*x, None, cu), kda.gdn_chunk_fwd(*y, None, cu)),):
        for i in (slice(0, 65), slice(105, None)):
            assert torch.equal(a[0][:, i], b[0][:, i])
        assert torch.equal(a[1][0], b[1][0]) and torch.equal(a[1][2], b[1][2])
    a, b = kda.gdn_chunk_bwd(*x, do, None, None, cu), kda.gdn_chunk_bwd(*y, do, None, None, cu)
    for key in ("dq", "dk", "dv", "dg", "dbeta"):
        for i in (slice(0, 65), slice(105, None)):
            assert torch.equal(a[key][:, i], b[key][:, i]), key


def test_split_walks_agree():
    """A prompt in two calls, the state carried in fp32, against one call (other chunk boundaries)."""
    x = ref.inputs(2, 200, 2, 4, 128, 128, F32, seed=16, device=DEV)
    o, f = kda.gdn_chunk_fwd(*x)
    a, s = kda.gdn_chunk_fwd(*[t[:, :77].contiguous() for t in x])
    b, s = kda.gdn_chunk_fwd(*[t[:, 77:].contiguous() for t in x], s, final_state=s)
    close("out", torch.cat([a, b], 1), o, *tol(F32))
    close("final", s, f, *tol(F32))


# -------------------------------------------------------------------------------------- decode --
@pytest.mark.parametrize("io,sdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("T", [1, 3])
def test_decode(io, sdt, dk, dv, T):
    n, pool_n = 5, 9
    x = ref.inputs(n, T, 2, 6, dk, dv, io, seed=T + dk, device=DEV)
    pool = state(pool_n, 6, dk, dv, sdt)
    slots = torch.tensor([7, 0, 3, 8, 2], dtype=torch.int32, device=DEV)
    before = pool.clone()
    out = kda.gdn_decode(*x, pool, slots, scale=0.5, state_slots_host=slots.cpu())
    o, f = ref.delta_rule(*x, before[slots.long()], None, 0.5)
    close("out", out, o, 2.3e-3 if io == BF else 1.5e-5)
    close("state", pool[slots.long()], f, 2.3e-3 if sdt == BF else 1.5e-5)
    rest = [i for i in range(pool_n) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_decode_padded_rows_and_ragged_drafts():
    lens = [2, 0, 1, 4, 1]
    x = ref.inputs(1, sum(lens), 1, 2, 128, 128, BF, seed=3, device=DEV)
    cu = ref.packed(lens, DEV)
    pool = state(6, 2, 128, 128, F32)
    before = pool.clone()
    # sequence 2 is padded (-1), sequence 3 names a slot that is not there
    slots = torch.tensor([4, 1, -1, 6, 0], dtype=torch.int32, device=DEV)
    out = torch.full_like(x[2], 7.0)
    kda.gdn_decode(*x, pool, slots, cu, out=out)
    o, f = ref.delta_rule(*x, before[torch.tensor([4, 1, 0, 0, 0], device=DEV)], cu)
    for i, s in ((0, 4), (1, 1), (4, 0)):
        a, b = int(cu[i]), int(cu[i + 1])
        if b > a:
            close(f"out {i}", out[:, a:b], o[:, a:b], 2.3e-3)
        close(f"state {i}", pool[s], f[i], 1.5e-5)
    assert (out[:, int(cu[2]):int(cu[4])] == 7).all()
    for s in (1, 2, 3, 5):
        assert torch.equal(pool[s], before[s])


def test_decode_continues_a_prefill():
    x = ref.inputs(3, 40, 2, 4, 128, 128, F32, seed=4, device=DEV)
    o, f = kda.gdn_chunk_fwd(*x)
    _, pool = kda.gdn_chunk_fwd(*[t[:, :33].contiguous() for t in x])
    outs = [kda.gdn_decode(*[t[:, i:i + 1].contiguous() for t in x], pool) for i in range(33, 36)]
    outs.append(kda.gdn_decode(*[t[:, 36:].contiguous() for t in x], pool))  # four drafted tokens at once
    close("out", torch.cat(outs, 1), o[:, 33:], *tol(F32))
    close("state", pool, f, *tol(F32))


def test_offsets_behind_32_bits():
    """A slot of a pool behind 2^31 elements, and tokens of a projection behind 2^31 elements."""
    per = 32 * 128 * 128
    n = 2 ** 31 // per + 2
    pool = torch.empty(n, 32, 128, 128, dtype=BF, device=DEV)
    x = ref.inputs(1, 1, 32, 32, 128, 128, BF, seed=1, device=DEV)
    pool[n - 1] = state(1, 32, 128, 128, BF)[0]
    small = pool[n - 1:].clone()
    a = kda.gdn_decode(*x, pool, torch.tensor([n - 1], dtype=torch.int32, device=DEV))
    b = kda.gdn_decode(*x, small)
    assert torch.equal(a, b) and torch.equal(pool[n - 1], small[0])
    del pool
    T, ld = 2 ** 15 + 100, 2 ** 16
    wide = torch.zeros(1, T, ld, dtype=BF, device=DEV)
    y = ref.inputs(1, T, 1, 1, 128, 128, BF, mu=-4.0, seed=2, device=DEV)
    for i in range(3):
        wide[..., 128 * i:128 * i + 128] = y[i][:, :, 0]
    z = [wide[..., 128 * i:128 * i + 128].unflatten(-1, (1, 128)) for i in range(3)] + y[3:]
    for p, q in zip(kda.gdn_chunk_fwd(*z), kda.gdn_chunk_fwd(*y)):
        assert torch.equal(p, q)
    do = torch.randn_like(y[2])
    p, q = kda.gdn_chunk_bwd(*z, do), kda.gdn_chunk_bwd(*y, do)
    for key in p:
        assert torch.equal(p[key], q[key]), key


# ------------------------------------------------------------------------------- norm gradients --
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 16, 4099, 70001])
def test_norm_gate_bwd(io, d, rows):
    gen = torch.Generator().manual_seed(rows + d)
    o, z, dy = (torch.randn(rows, d, generator=gen).to(io).to(DEV) for _ in range(3))
    w = torch.randn(d, generator=gen).to(DEV)
    if rows > 4:
        o[1] = 0  # a row of zeros: r = eps^-1/2
        z[2, :4] = torch.tensor([100.0, -100.0, 30.0, -30.0])  # saturated gates
        o[3] *= 1e4
    got = kda.norm_gate_bwd(o, z, w, dy)
    x = [t.double().requires_grad_() for t in (o, z, w)]
    want = torch.autograd.grad((ref.norm_gate(*x) * dy.double()).sum(), x)
    # one rounding of the outputs; fp32 sums of 128 terms (1e-5), d_weight a sum over rows in fp32 and fp64
    for name, a, b in zip(("d_o", "d_gate", "d_weight"), got, want):
        close(name, a, b, 1.5e-5 if a.dtype == F32 else 2.3e-3)
    again = kda.norm_gate_bwd(o, z, w, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_norm_gate_bwd_without_rows():
    o = torch.empty(0, 64, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    d_o, d_z, d_w = kda.norm_gate_bwd(o, o, w, o)
    assert d_o.shape == o.shape and (d_w == 0).all()


# ------------------------------------------------------------------------------------ together --
def test_a_training_step_of_the_block():
    """Forward, epilogue and back through both, against the reference's autograd."""
    x = ref.inputs(2, 160, 2, 4, 128, 128, F32, seed=21, device=DEV)
    z, dy = torch.randn_like(x[2]), torch.randn_like(x[2])
    w = 1 + 0.1 * torch.randn(128, device=DEV)
    sc = 128 ** -0.5
    o, _ = kda.gdn_chunk_fwd(*x, scale=sc)
    y = kda.norm_gate(o, z, w)
    d_o, d_z, d_w = kda.norm_gate_bwd(o, z, w, dy)
    d = kda.gdn_chunk_bwd(*x, d_o, scale=sc)
    r = [t.double().requires_grad_() for t in (*x, z, w)]
    out, _ = ref.delta_rule(*r[:5], scale=sc)
    yr = ref.norm_gate(out, r[5], r[6])
    want = torch.autograd.grad((yr * dy.double()).sum(), r)
    close("y", y, yr.detach(), *tol(F32))
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dz", "dw"),
                          (d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d_z, d_w), want):
        close(name, a, b, 4e-5, 1e-4)  # two operators' errors, the norm's on rows of small outputs


def test_a_serving_run():
    """Packed prompts into slots of a pool, then decoding steps with a padded row, each with the epilogue."""
    lens, Hv = [70, 5, 129], 4
    x = ref.inputs(1, sum(lens), 2, Hv, 128, 128, BF, seed=22, device=DEV)
    w = torch.ones(128, device=DEV)
    cu = ref.packed(lens, DEV)
    out, fin = kda.gdn_chunk_fwd(*views(x), None, cu, state_dtype=F32)
    pool = torch.zeros(8, Hv, 128, 128, device=DEV)
    where = [5, 2, 7]
    pool[where] = fin
    o, S = ref.delta_rule(*x, None, cu)
    close("prompt", out, o, *tol(BF))
    slots = torch.tensor(where + [-1], dtype=torch.int32, device=DEV)
    for step in range(3):
        t = ref.inputs(4, 1, 2, Hv, 128, 128, BF, seed=30 + step, device=DEV)
        z = torch.randn_like(t[2])
        got = kda.norm_gate(kda.gdn_decode(*t, pool, slots, out=torch.zeros_like(t[2])), z, w)
        o, S = ref.delta_rule(*[a[:3] for a in t], S)
        # the states began with the prompt's error, the epilogue keeps relative errors and rounds once more
        close(f"step {step}", got[:3], ref.norm_gate(o, z[:3], w), 1.2e-2, 3e-2)
    close("states", pool[where], S, *tol(BF))
    assert (pool[[0, 1, 3, 4, 6]] == 0).all()


def test_captured_and_replayed_beside_eager_work():
    x = ref.inputs(2, 200, 2, 4, 128, 128, BF, seed=23, device=DEV)
    do, z, w = torch.randn_like(x[2]), torch.randn_like(x[2]), torch.ones(128, device=DEV)
    pool = state(2, 4, 128, 128, F32)
    tok = [t[:, :1].contiguous() for t in x]

    def step():
        o, f = kda.gdn_chunk_fwd(*x)
        d = kda.gdn_chunk_bwd(*x, do)
        n = kda.norm_gate_bwd(o, z, w, do)
        return [o, f, d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["d_initial_state"], *n, kda.gdn_decode(*tok, pool)]

    start = pool.clone()
    want = [t.clone() for t in step()]
    end = pool.clone()
    pool.copy_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        pool.copy_(start)
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        assert torch.equal(pool, end), i
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        pool.copy_(start)
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), i  # eager work between the replays


def test_two_streams_at_once():
    xs = [ref.inputs(2, 300, 2, 4, 128, 128, BF, seed=40 + i, device=DEV) for i in range(2)]
    dos = [torch.randn_like(x[2]) for x in xs]
    want = [(kda.gdn_chunk_fwd(*x), kda.gdn_chunk_bwd(*x, d)) for x, d in zip(xs, dos)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, d, s in zip(xs, dos, streams):
            got.append((kda.gdn_chunk_fwd(*x, stream=s), kda.gdn_chunk_bwd(*x, d, stream=s)))
        torch.cuda.synchronize()
        for (a, b), (c, d) in zip(got, want):
            assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
            assert all(torch.equal(b[k], d[k]) for k in b)


@pytest.mark.parametrize("io,sdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [8192, 4096 + 1])
def test_forward_split_over_its_length(io, sdt, dk, dv, T):
    # long sequences on few heads: with room the walk is split; mild decays, so the first segment's state is seen
    # in the last one
    x = ref.inputs(2, T, 1, 2, dk, dv, io, seed=T + dk, device=DEV)
    x[3].mul_(0.05)
    s0 = state(2, 2, dk, dv, sdt)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    a = kda.gdn_chunk_fwd(*x, s0, scale=dk ** -0.5, workspace=none)
    o, f = ref.delta_rule(*x, s0, scale=dk ** -0.5)
    for name, got in (("one walk", a), ("split", kda.gdn_chunk_fwd(*x, s0, scale=dk ** -0.5))):
        close(name + " out", got[0], o, *tol(io))
        close(name + " final", got[1], f, *tol(BF if sdt == BF else io))
    assert not torch.equal(a[0], got[0])  # two ways of summing
    inplace = s0.clone()
    again = kda.gdn_chunk_fwd(*x, inplace, scale=dk ** -0.5, final_state=inplace)
    assert torch.equal(again[0], got[0]) and torch.equal(inplace, got[1])
    assert torch.equal(kda.gdn_chunk_fwd(*x, s0, scale=dk ** -0.5, output_final_state=False)[0], got[0])


def test_split_forward_keeps_a_bad_value_behind_it():
    x = ref.inputs(1, 8192, 1, 2, 128, 128, BF, seed=3, device=DEV)
    want = kda.gdn_chunk_fwd(*x)  # within a chunk of 64 tokens (here from 4992) a NaN meets the zeros of the causal mask
    x[2][0, 5000, 0, 7] = float("nan")
    x[2][0, 8191, 1, 9] = float("inf")
    out, fin = kda.gdn_chunk_fwd(*x)
    assert torch.equal(out[:, :4992], want[0][:, :4992])
    assert torch.equal(out[:, :8128, 1], want[0][:, :8128, 1])
    other = [i for i in range(128) if i != 7]
    assert torch.equal(out[:, :, 0, other], want[0][:, :, 0, other]) and torch.equal(fin[0, 0][:, other], want[1][0, 0][:, other])
    assert out[0, 5000:, 0, 7].isnan().all() and fin[0, 0, :, 7].isnan().all()


def test_split_forward_captured_and_workspaces_of_the_caller():
    x = ref.inputs(1, 8192, 1, 2, 128, 128, BF, seed=3, device=DEV)
    want = [t.clone() for t in kda.gdn_chunk_fwd(*x)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.gdn_chunk_fwd(*x)
    for i in range(4):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(torch.equal(a, b) for a, b in zip(kda.gdn_chunk_fwd(*x), want)), i
    with pytest.raises(ValueError):
        kda.gdn_chunk_fwd(*x, workspace=torch.empty(1 << 24, dtype=torch.uint8))  # on the host
    with pytest.raises(kda.KdaError):
        kda.gdn_chunk_fwd(*x, workspace=want[0].view(torch.uint8).flatten(), out=want[0])  # is the output
    with pytest.raises(kda.KdaError):
        kda.gdn_chunk_fwd(*x, workspace=torch.empty(1 << 24, dtype=torch.uint8, device=DEV)[4:])  # alignment
    small = torch.empty(256, dtype=torch.uint8, device=DEV)  # too little room: as without
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    a, b = kda.gdn_chunk_fwd(*x, workspace=small), kda.gdn_chunk_fwd(*x, workspace=none)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("io,sdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [2048, 1300 + 1])
def test_backward_split_over_its_length(io, sdt, dk, dv, T):
    x = ref.inputs(1, T, 1, 2, dk, dv, io, seed=T + dk, device=DEV)
    x[3].mul_(0.05)
    s0, dsf = state(1, 2, dk, dv, sdt), state(1, 2, dk, dv, sdt, seed=8)
    got, do = check_bwd(x, s0, dsf, scale=dk ** -0.5, label=f"split T{T}")
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)  # the same as a packed batch: one walk
    one = kda.gdn_chunk_bwd(*x, do, s0, dsf, cu, scale=dk ** -0.5)
    assert not torch.equal(one["dk"], got["dk"])  # two ways of summing
    again = kda.gdn_chunk_bwd(*x, do, s0, dsf, scale=dk ** -0.5)
    assert all(torch.equal(again[k], got[k]) for k in got)
    bare, _ = check_bwd(x, scale=dk ** -0.5, label="without states", need_d_initial_state=False)
    assert bare["d_initial_state"] is None


def test_backward_split_with_many_sequences_and_captured():
    x = ref.inputs(3, 2100, 2, 4, 128, 64, BF, seed=4, device=DEV)
    x[3].mul_(0.05)
    got, do = check_bwd(x, state(3, 4, 128, 64, F32), state(3, 4, 128, 64, F32, seed=9), label="three sequences")
    want = kda.gdn_chunk_bwd(*x, do)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = kda.gdn_chunk_bwd(*x, do)
    for i in range(4):
        for t in caught.values():
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(caught[k], want[k]) for k in want), i
        eager = kda.gdn_chunk_bwd(*x, do)
        assert all(torch.equal(eager[k], want[k]) for k in want), i


def test_arguments_are_named_in_errors():
    x = ref.inputs(1, 40, 2, 4, 64, 64, BF, seed=3, device=DEV)
    q, k, v, g, b = x
    for args, name in (((q, k.float(), v, g, b), "k"), ((q, k, v.cpu(), g, b), "v"), ((q, k, v, g[:, :39], b), "g"),
                       ((q, k, v, g, b.to(torch.float64)), "beta"), ((q, k, v[..., :32], g, b), "v"),
                       ((q, k[:, ::2], v, g, b), "k"), ((q, k, v.transpose(1, 2), g, b), "v")):
        with pytest.raises((TypeError, ValueError), match=f"^{name}\\b"):
            kda.gdn_chunk_fwd(*args)
    with pytest.raises(ValueError, match="^initial_state"):
        kda.gdn_chunk_fwd(*x, torch.zeros(2, 4, 64, 64, device=DEV))
    with pytest.raises(TypeError, match="^state_slots"):
        kda.gdn_decode(*[t[:, :1].contiguous() for t in x], torch.zeros(3, 4, 64, 64, device=DEV),
                       torch.zeros(1, dtype=torch.int64, device=DEV))
