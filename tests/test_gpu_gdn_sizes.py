"""GPU tests of the scalar-gate delta rule on both sides of the rules that its launches go by: many packed sequences
(ranked by their chunks up to 256 of them), split walks of the smallest heads, bf16 gradients of few gates.

Bounds: fp32 256 * 2^-24 = 1.5e-5; bf16 forward sqrt(6) and gradients sqrt(9) independent roundings of 2.3e-3
(2^-8 / sqrt(3)); tensors of under 1,024 values 2e-2, as their roundings do not average."""
import pytest
import torch

import gdn_reference as ref
import gated_delta_rule_45_amd as kda

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
KEYS = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")


def states(n, Hv, dk, dv, dtype=F32, std=0.3, seed=7):
    return (std * torch.randn(n, Hv, dk, dv, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def like(x, seed=11):
    return torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype).to(DEV)


def error(got, want):
    g, w = got.double(), want.double()
    assert torch.isfinite(g).all()
    return float((g - w).norm() / w.norm())


def close(name, got, want, bound):
    e = error(got, want)
    print(f"  {name}: rel2={e:.2e}", flush=True)
    assert e <= bound, f"{name}: {e:.3e} > {bound}"


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("n", [255, 256, 257, 600])
def test_many_packed_sequences(io, n):
    """Of 256 sequences the longest start first, more keep their order; neither changes a bit of a sequence."""
    print(f"[{io}] {n} sequences", flush=True)
    lens = torch.randint(0, 9, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    lens[0], lens[n // 2], lens[n - 1] = 70, 130, 65
    x = ref.inputs(1, sum(lens), 1, 2, 64, 64, io, seed=n, device=DEV)
    cu, s0, dsf, do = ref.packed(lens, DEV), states(n, 2, 64, 64), states(n, 2, 64, 64, seed=8), like(x[2])
    out, fin = kda.gdn_chunk_fwd(*x, s0, cu)
    o, f = ref.delta_rule(*x, s0, cu)
    close("out", out, o, 6e-3 if io == BF else 1.5e-5)
    close("final", fin, f, 6e-3 if io == BF else 1.5e-5)
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf, cu), ref.delta_rule_grads(*x, do, s0, dsf, cu)
    for key in KEYS:
        close(key, got[key], want[key], 8e-3 if io == BF else 1.5e-5)
    for i in (0, n // 2, n - 1):
        a, b = int(cu[i]), int(cu[i + 1])
        o1, f1 = kda.gdn_chunk_fwd(*[t[:, a:b].contiguous() for t in x], s0[i:i + 1].contiguous())
        assert torch.equal(o1, out[:, a:b]) and torch.equal(f1[0], fin[i]), i


@pytest.mark.parametrize("io", [BF, F32])
def test_split_walks_of_the_smallest_heads(io):
    x = ref.inputs(1, 4000, 1, 2, 64, 64, io, seed=1, device=DEV)
    x[3].mul_(0.05)
    s0, dsf, do = states(1, 2, 64, 64), states(1, 2, 64, 64, seed=8), like(x[2])
    out, fin = kda.gdn_chunk_fwd(*x, s0)
    one = kda.gdn_chunk_fwd(*x, s0, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert not torch.equal(one[0], out)  # two ways of summing: the walk is split
    o, f = ref.delta_rule(*x, s0)
    close("out", out, o, 6e-3 if io == BF else 1.5e-5)
    close("final", fin, f, 6e-3 if io == BF else 1.5e-5)
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf), ref.delta_rule_grads(*x, do, s0, dsf)
    for key in KEYS:
        close(key, got[key], want[key], 8e-3 if io == BF else 1.5e-5)
    one = kda.gdn_chunk_bwd(*x, do, s0, dsf, torch.tensor([0, 4000], dtype=torch.int32, device=DEV))
    assert not torch.equal(one["dk"], got["dk"])


@pytest.mark.parametrize("T,Hv,wide", [(1, 2, True), (128, 4, True), (256, 2, True), (256, 1, True), (129, 4, False),
                                       (257, 1, False), (512, 1, False)])
def test_bf16_gradients_of_few_gates(T, Hv, wide):
    """At most 256 tokens and 512 gates: fp32 operands, so that only what is stored in bf16 is rounded, once, by at
    most 2^-8 of each value; the gates' gradients (fp32 here) and the state's have fp32's error."""
    print(f"T={T} Hv={Hv}", flush=True)
    x = ref.inputs(1, T, 1, Hv, 64, 64, BF, F32, seed=T, device=DEV)
    s0, dsf, do = states(1, Hv, 64, 64), states(1, Hv, 64, 64, seed=8), like(x[2])
    got, want = kda.gdn_chunk_bwd(*x, do, s0, dsf), ref.delta_rule_grads(*x, do, s0, dsf)
    for key in KEYS:
        if wide:
            bound = 2 ** -8 + 1.5e-5 if got[key].dtype == BF else 1.5e-5
        else:
            bound = 8e-3 if want[key].numel() >= 1024 else 2e-2
        close(key, got[key], want[key], bound)
    assert (error(got["dg"], want["dg"]) <= 1.5e-5) == wide
