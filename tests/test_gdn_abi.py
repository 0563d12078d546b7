"""Refusals of kda_gdn_* and kda_norm_gate_bwd, on the host: a bad call returns its status and a message and
launches nothing (so this runs without a GPU, on addresses that are never read)."""
import ctypes

import pytest
import torch

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd.gdn import GdnProblem

INVALID, UNSUPPORTED, WORKSPACE = kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
at = lambda i: ctypes.c_void_p(0x10000000 * (i + 1))  # noqa: E731  aligned, far apart
arr = lambda *x: (ctypes.c_int32 * len(x))(*x)  # noqa: E731


def prob(**kw):
    base = dict(batch=1, seq_len=15, num_seqs=0, num_heads_k=2, num_heads_v=4, head_dim_k=64, head_dim_v=64,
                io_dtype=kda.KDA_BF16, gate_dtype=kda.KDA_F32, state_dtype=kda.KDA_F32, scale=1.0, stride_q=0,
                stride_k=0, stride_v=0)
    base.update(kw)
    return GdnProblem(**base)


def fwd(p, q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=None, cu_host=None, out=at(5), sf=None, ws=None,
        n=0):
    return kda.library().kda_gdn_chunk_fwd(None if p is None else ctypes.byref(p), q, k, v, g, beta, s0, cu, cu_host,
                                           out, sf, ws, n, None)


def bwd(p, q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=None, d_out=at(5), dsf=None, dq=at(6), dk=at(7),
        dv=at(8), dg=at(9), db=at(10), ds0=None, ws=at(11), n=1 << 40):
    return kda.library().kda_gdn_chunk_bwd(ctypes.byref(p), q, k, v, g, beta, s0, cu, None, d_out, dsf, dq, dk, dv, dg,
                                           db, ds0, ws, n, None)


def decode(p, state=at(6), slots=8, idx=at(7), idx_host=None, cu=None, cu_host=None, out=at(5), q=at(0)):
    return kda.library().kda_gdn_decode(ctypes.byref(p), q, at(1), at(2), at(3), at(4), state, slots, idx, idx_host, cu,
                                        cu_host, out, None)


def message():
    return kda.library().kda_last_error().decode()


BAD = [
    (dict(num_heads_k=0), INVALID), (dict(num_heads_v=0), INVALID), (dict(num_heads_v=5), INVALID),
    (dict(num_heads_k=4, num_heads_v=2), INVALID), (dict(batch=-1), INVALID), (dict(seq_len=-1), INVALID),
    (dict(head_dim_k=96), UNSUPPORTED), (dict(head_dim_v=256), UNSUPPORTED), (dict(io_dtype=2), INVALID),
    (dict(gate_dtype=-1), INVALID), (dict(state_dtype=9), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(stride_q=120), INVALID), (dict(stride_k=132), INVALID),
    (dict(stride_v=-256), INVALID), (dict(stride_v=1 << 59), UNSUPPORTED),
    (dict(batch=2 ** 31 - 1, num_heads_v=2 ** 31 - 2, num_heads_k=2), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_every_call_refuses_bad_problems(kw, status):
    p = prob(**kw)
    for call in (fwd, bwd, decode):
        assert call(p) == status
        assert message()
    n = ctypes.c_size_t(7)
    assert kda.library().kda_gdn_chunk_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == status and n.value == 0


def test_pointers_are_checked():
    assert fwd(None) == INVALID
    for name in ("q", "k", "v", "g", "beta", "out"):
        assert fwd(prob(), **{name: None}) == INVALID and f"{name} is NULL" in message()
    for name in ("q", "k", "v", "out", "s0", "sf"):
        assert fwd(prob(), **{name: ctypes.c_void_p(0x70000008)}) == INVALID and "aligned" in message()
    assert fwd(prob(), g=ctypes.c_void_p(0x70000002)) == INVALID
    for name in ("d_out", "dq", "dk", "dv", "dg", "db"):
        assert bwd(prob(), **{name: None}) == INVALID and "NULL" in message()
    assert decode(prob(), state=None) == INVALID
    assert decode(prob(), state=ctypes.c_void_p(0x70000004)) == INVALID


def test_overlaps_are_refused():
    off = lambda p, n: ctypes.c_void_p(p.value + n)  # noqa: E731
    assert fwd(prob(), out=off(at(2), 256)) == INVALID and "aliases v" in message()
    assert fwd(prob(), out=off(at(0), -4096)) == INVALID  # its end reaches into q
    assert fwd(prob(), s0=at(7), sf=off(at(7), 16)) == INVALID  # states may be one buffer, not shifted ones
    assert fwd(prob(), s0=at(7), out=at(7)) == INVALID
    assert bwd(prob(), dq=at(0)) == INVALID and "aliases q" in message()
    assert bwd(prob(), dq=at(7)) == INVALID
    assert bwd(prob(), s0=at(12), ds0=at(12)) == INVALID
    assert bwd(prob(), ws=at(6)) == INVALID
    assert decode(prob(), out=off(at(6), 16)) == INVALID


def test_offsets_and_slots_are_checked():
    p = prob(num_seqs=4)
    good = arr(0, 3, 8, 8, 15)
    assert fwd(prob(num_seqs=4, batch=2), cu=at(9)) == INVALID
    for bad in (arr(1, 3, 8, 8, 15), arr(0, 3, 2, 8, 15), arr(0, 3, 8, 8, 14)):
        assert fwd(p, cu=at(9), cu_host=bad) == INVALID
    assert fwd(p, cu_host=good) == INVALID
    assert fwd(p, cu=ctypes.c_void_p(0x70000002)) == INVALID
    q = prob(batch=3, seq_len=1)
    assert decode(q, slots=2, idx=None) == INVALID
    assert decode(q, idx_host=arr(0, 8, 1)) == INVALID and "there are 8" in message()
    assert decode(q, idx_host=arr(4, 2, 4)) == INVALID and "both 4" in message()
    assert decode(q, idx=None, idx_host=arr(0, 1, 2)) == INVALID
    assert decode(q, slots=-1) == INVALID
    assert decode(q, slots=2 ** 31) == INVALID


def test_backward_needs_its_workspace():
    lib, p = kda.library(), prob(seq_len=1000)
    n = ctypes.c_size_t(0)
    assert lib.kda_gdn_chunk_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == kda.KDA_OK
    # S and dS of 16 chunks, Z of 1,000 tokens
    assert n.value >= 2 * 16 * 4 * 64 * 64 * 2 + 1000 * 4 * 64 * 2
    assert bwd(p, n=n.value - 1) == WORKSPACE
    assert bwd(p, ws=None) == WORKSPACE
    assert bwd(p, ws=ctypes.c_void_p(0xb0000010)) == INVALID  # 256-byte aligned
    assert lib.kda_gdn_chunk_bwd_workspace(ctypes.byref(p), None) == INVALID


def test_empty_calls_launch_nothing():
    for kw in (dict(batch=0), dict(seq_len=0)):
        assert fwd(prob(**kw), q=None, k=None, v=None, g=None, beta=None, out=None) == kda.KDA_OK
        assert bwd(prob(**kw), q=None, k=None, v=None, g=None, beta=None, d_out=None, dq=None, dk=None, dv=None, dg=None,
                   db=None, ws=None, n=0) == kda.KDA_OK
        assert decode(prob(**kw), q=None, out=None) == kda.KDA_OK
    assert decode(prob(batch=0), slots=0, state=None) == kda.KDA_OK


def norm(rows=4, d=64, io=kda.KDA_BF16, eps=1e-6, o=at(0), gate=at(1), w=at(2), dy=at(3), do=at(4), dz=at(5), dw=at(6),
         ws=None, n=0):
    return kda.library().kda_norm_gate_bwd(rows, d, io, eps, o, gate, w, dy, do, dz, dw, ws, n, None)


def test_norm_gate_bwd_refusals():
    lib = kda.library()
    assert norm(rows=-1) == INVALID
    assert norm(d=96) == UNSUPPORTED
    assert norm(io=3) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(eps=eps) == INVALID
    for name in ("o", "gate", "w", "dy", "do", "dz", "dw"):
        assert norm(**{name: None}) == INVALID
        assert norm(**{name: ctypes.c_void_p(0x70000004)}) == INVALID
    assert norm(do=at(0)) == INVALID and norm(dz=at(4)) == INVALID and norm(dw=at(2)) == INVALID
    assert norm(rows=2 ** 50) == UNSUPPORTED
    need = lib.kda_norm_gate_bwd_workspace(10 ** 6, 128, kda.KDA_BF16)
    assert need > 0 and norm(rows=10 ** 6, d=128, ws=at(30), n=need - 1) == WORKSPACE
    assert lib.kda_norm_gate_bwd_workspace(-1, 128, 1) == 0 and lib.kda_norm_gate_bwd_workspace(9, 100, 1) == 0


def test_binding_checks_its_tensors():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    q, v, g = t(2, 3, 1, 64), t(2, 3, 2, 64), t(2, 3, 2)
    with pytest.raises(ValueError, match="GPU"):
        kda.gdn_chunk_fwd(q, q, v, g, g)
    with pytest.raises(TypeError):
        kda.gdn_chunk_fwd(q, q.float(), v, g, g)
    with pytest.raises(TypeError):
        kda.gdn_chunk_fwd(q, q, v, g, g.float())
    with pytest.raises(TypeError):
        kda.gdn_chunk_fwd(q.half(), q.half(), v.half(), g, g)
    with pytest.raises(ValueError, match="shape"):
        kda.gdn_chunk_fwd(q, q, v[:, :2], g, g)
    with pytest.raises(ValueError, match="heads of a token"):
        kda.gdn_chunk_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), q, v, g, g)
    with pytest.raises(ValueError, match="heads of a token"):
        kda.gdn_chunk_fwd(q[:, :1].expand(2, 3, 1, 64), q, v, g, g)
    with pytest.raises(ValueError, match="B == 1"):
        kda.gdn_chunk_fwd(q, q, v, g, g, cu_seqlens=torch.tensor([0, 3], dtype=torch.int32))
    with pytest.raises(TypeError):
        kda.gdn_decode(q, q, v, g, g, torch.zeros(2, 2, 64, 64), state_slots=torch.zeros(2, dtype=torch.int64))
