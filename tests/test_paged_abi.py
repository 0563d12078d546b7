"""Refusals of kda_rope*, kda_paged_* on the host: a bad call returns its status and a message and launches nothing (so
this runs without a GPU, on addresses that are never read); what the binding refuses; frequencies."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd.paged import PagedProblem, Rope, RopeProblem

OK, INVALID, UNSUPPORTED, WORKSPACE = kda.KDA_OK, kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
at = lambda i: ctypes.c_void_p(0x100000000 * (i + 1))  # noqa: E731  aligned, far apart
off = lambda p, n: ctypes.c_void_p(p.value + n)  # noqa: E731
odd = ctypes.c_void_p(0x7700000008)
arr = lambda *x: (ctypes.c_int32 * len(x))(*x)  # noqa: E731


def message():
    return kda.library().kda_last_error().decode()


# ------------------------------------------------------------------------------------ rotary --
def rprob(**kw):
    base = dict(batch=2, seq_len=15, num_heads_q=4, num_heads_k=2, head_dim=64, io_dtype=kda.KDA_BF16, rot_dim=64, interleaved=0,
                inverse=0, amplitude=1.0, stride_q=0, stride_k=0, stride_q_out=0, stride_k_out=0)
    base.update(kw)
    return RopeProblem(**base)


def rope(p, q=at(0), k=at(1), pos=at(2), freq=at(3), qo=at(4), ko=at(5)):
    return kda.library().kda_rope(None if p is None else ctypes.byref(p), q, k, pos, freq, qo, ko, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(seq_len=-1), INVALID), (dict(num_heads_q=0), INVALID), (dict(num_heads_k=-1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(io_dtype=5), INVALID), (dict(rot_dim=24), INVALID), (dict(rot_dim=80), INVALID),
    (dict(rot_dim=-16), INVALID), (dict(interleaved=2), INVALID), (dict(inverse=-1), INVALID),
    (dict(amplitude=math.inf), INVALID), (dict(stride_q=248), INVALID), (dict(stride_k=132), INVALID),
    (dict(stride_q_out=-256), INVALID), (dict(stride_k_out=1 << 59), UNSUPPORTED), (dict(batch=1 << 20, seq_len=1 << 20), UNSUPPORTED),
    (dict(num_heads_q=1 << 30), UNSUPPORTED), (dict(batch=1 << 15, seq_len=1 << 15, num_heads_q=64), UNSUPPORTED),
])
def test_rope_refuses_bad_problems(kw, status):
    assert rope(rprob(**kw)) == status and message()


def test_rope_checks_its_pointers():
    assert rope(None) == INVALID
    for name in ("q", "k", "freq", "qo", "ko"):
        assert rope(rprob(), **{name: None}) == INVALID and "NULL" in message()
    for name in ("q", "k", "qo", "ko"):
        assert rope(rprob(), **{name: odd}) == INVALID and "aligned" in message()
    assert rope(rprob(), pos=ctypes.c_void_p(0x7700000002)) == INVALID
    assert rope(rprob(), qo=off(at(0), 16)) == INVALID and "aliases q" in message()
    assert rope(rprob(), qo=at(1)) == INVALID and "aliases k" in message()
    assert rope(rprob(), ko=at(4)) == INVALID
    assert rope(rprob(stride_q=512), qo=at(0)) == INVALID  # the same buffer in another stride
    # slices of one tensor: rows beside each other do not meet, rows over each other do
    wide = dict(stride_q=512, stride_q_out=512)
    assert rope(rprob(**wide), q=at(0), qo=off(at(0), 400)) == INVALID
    assert rope(rprob(seq_len=0), q=None, k=None, freq=None, qo=None, ko=None) == OK
    assert rope(rprob(seq_len=0, num_heads_k=0), q=None, k=None, freq=None, qo=None, ko=None) == OK


@pytest.mark.parametrize("args", [(24, 1e4, 0, 1., 0, 1., 32.), (-16, 1e4, 0, 1., 0, 1., 32.), (64, 1., 0, 1., 0, 1., 32.),
                                  (64, math.nan, 0, 1., 0, 1., 32.), (64, 1e4, 4, 1., 0, 1., 32.), (64, 1e4, 1, .5, 0, 1., 32.),
                                  (64, 1e4, 3, 2., 0, 1., 32.), (64, 1e4, 3, 2., 99, 3., 3.), (64, 1e4, 3, 2., 99, -1., 3.)])
def test_frequencies_refuse(args):
    lib, f, a = kda.library(), (ctypes.c_float * 64)(), ctypes.c_float()
    assert lib.kda_rope_frequencies(*args, ctypes.addressof(f), ctypes.addressof(a)) == INVALID
    assert lib.kda_rope_frequencies(64, 1e4, 0, 1., 0, 1., 32., None, ctypes.addressof(a)) == INVALID
    assert lib.kda_rope_frequencies(64, 1e4, 0, 1., 0, 1., 32., ctypes.addressof(f), None) == INVALID


def test_frequencies():
    i = torch.arange(0, 48, 2, dtype=torch.float64)
    plain = 10000.0 ** (-i / 48)
    f, a = kda.rope_frequencies(48)
    assert a == 1.0 and torch.equal(f, plain.float())
    f, a = kda.rope_frequencies(48, scaling="linear", factor=4.0)
    assert a == 1.0 and torch.equal(f, (plain / 4).float())
    f, a = kda.rope_frequencies(48, scaling="base", factor=4.0)  # the fastest pair kept, the slowest squeezed by 4
    assert a == 1.0 and f[0] == 1.0 and math.isclose(float(f[-1]), float(plain[-1]) / 4, rel_tol=1e-6)
    f, a = kda.rope_frequencies(48, scaling="parts", factor=8.0, original_len=4096, slow=1.0, fast=32.0)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(f[turns >= 32], plain[turns >= 32].float()) and torch.allclose(f[turns <= 1].double(), plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (f[mid].double() < plain[mid]).all() and (f[mid].double() > plain[mid] / 8).all()
    assert math.isclose(a, 0.1 * math.log(8.0) + 1, rel_tol=1e-6)
    assert kda.rope_frequencies(0)[0].numel() == 0
    with pytest.raises(ValueError, match="scaling"):
        kda.rope_frequencies(48, scaling="other")


# ------------------------------------------------------------------------------------- paged --
def prob(**kw):
    base = dict(batch=3, seq_len=5, num_seqs=0, num_heads_q=4, num_heads_kv=2, head_dim_k=64, head_dim_v=128,
                io_dtype=kda.KDA_BF16, page_size=16, max_pages=7, num_pages=40, stride_table=0, stride_q=0, stride_k=0, stride_v=0,
                k_page_stride=0, k_head_stride=0, k_cell_stride=0, v_page_stride=0, v_head_stride=0, v_cell_stride=0)
    base.update(kw)
    return PagedProblem(**base)


TURN = Rope(64, 0, 1.0, at(20), None)


def append(p, k=at(0), v=at(1), q=None, rope=None, table=at(3), lens=at(4), cu=None, host=None, kp=at(5), vp=at(6), qo=None):
    return kda.library().kda_paged_append(None if p is None else ctypes.byref(p), k, v, q, None if rope is None else ctypes.byref(rope),
                                          table, lens, cu, host, kp, vp, qo, None)


def attn(p, q=at(0), kp=at(5), vp=at(6), table=at(3), lens=at(4), cu=None, host=None, scale=1.0, window=0, out=at(7), lse=None,
         ws=at(9), n=1 << 40):
    return kda.library().kda_paged_attn(None if p is None else ctypes.byref(p), q, kp, vp, table, lens, cu, host, scale, window, out,
                                        lse, ws, n, None)


def room(p):
    n = ctypes.c_size_t(7)
    return kda.library().kda_paged_attn_workspace(ctypes.byref(p), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(seq_len=-1), INVALID), (dict(num_heads_q=0), INVALID), (dict(num_heads_kv=0), INVALID),
    (dict(num_heads_q=3), INVALID), (dict(io_dtype=7), INVALID), (dict(head_dim_k=256), UNSUPPORTED), (dict(head_dim_v=80), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(max_pages=-1), INVALID),
    (dict(max_pages=(1 << 26) + 1), UNSUPPORTED), (dict(k_page_stride=1 << 40, k_head_stride=1 << 36, k_cell_stride=1 << 27), UNSUPPORTED), (dict(num_pages=-1), INVALID), (dict(num_pages=1 << 31), INVALID), (dict(stride_table=6), INVALID),
    (dict(stride_table=-9), INVALID), (dict(stride_q=100), INVALID), (dict(stride_q=260), INVALID), (dict(stride_k=64), INVALID),
    (dict(stride_v=252), INVALID), (dict(stride_v=1 << 59), UNSUPPORTED), (dict(batch=1 << 20, seq_len=1 << 12), UNSUPPORTED),
    (dict(k_page_stride=2048, k_head_stride=1024, k_cell_stride=32), INVALID),   # cells over each other
    (dict(k_page_stride=1024, k_head_stride=1024, k_cell_stride=64), INVALID),   # heads over pages
    (dict(k_page_stride=2048, k_head_stride=1024), INVALID),                     # cell stride 0
    (dict(v_page_stride=4104, v_head_stride=2048, v_cell_stride=132), INVALID),  # not 16 bytes
    (dict(v_page_stride=-4096, v_head_stride=2048, v_cell_stride=128), INVALID),
    (dict(v_page_stride=1 << 60, v_head_stride=2048, v_cell_stride=128), UNSUPPORTED),
    (dict(num_heads_q=1 << 22, num_heads_kv=1, seq_len=0), UNSUPPORTED),
])
def test_paged_calls_refuse_bad_problems(kw, status):
    p = prob(**kw)
    for call in (append, attn):
        assert call(p) == status and message()
    assert room(p) == (status, 0)


def test_paged_calls_check_their_pointers():
    assert append(None) == INVALID and attn(None) == INVALID
    for name in ("k", "v", "table", "lens", "kp", "vp"):
        assert append(prob(), **{name: None}) == INVALID and "NULL" in message()
    for name in ("q", "kp", "vp", "table", "lens", "out"):
        assert attn(prob(), **{name: None}) == INVALID and "NULL" in message()
    for name in ("k", "v", "kp", "vp"):
        assert append(prob(), **{name: odd}) == INVALID and "aligned" in message()
    for name in ("q", "kp", "vp", "out", "ws"):
        assert attn(prob(), **{name: odd}) == INVALID and "aligned" in message()
    for name in ("table", "lens"):
        assert append(prob(), **{name: ctypes.c_void_p(0x7700000002)}) == INVALID
    assert attn(prob(), lse=ctypes.c_void_p(0x7700000002)) == INVALID
    assert attn(prob(), cu=ctypes.c_void_p(0x7700000002)) == INVALID
    # rotation
    assert append(prob(), q=at(2), qo=at(8)) == INVALID and "without rope" in message()
    assert append(prob(), rope=TURN, qo=at(8)) == INVALID
    assert append(prob(), rope=TURN, q=at(2)) == INVALID and "q_out is NULL" in message()
    for bad in (Rope(72, 0, 1.0, at(20), None), Rope(128, 0, 1.0, at(20), None), Rope(64, 3, 1.0, at(20), None),
                Rope(64, 0, math.nan, at(20), None), Rope(64, 0, 1.0, None, None)):
        assert append(prob(), rope=bad) == INVALID and message()


def test_paged_calls_refuse_overlaps():
    assert append(prob(), kp=at(0)) == INVALID and "aliases" in message()
    assert append(prob(), vp=off(at(5), 64)) == INVALID
    assert append(prob(), vp=at(3)) == INVALID
    assert append(prob(), kp=off(at(4), -16)) == INVALID
    assert append(prob(), rope=TURN, q=at(2), qo=at(0)) == INVALID
    assert append(prob(), rope=TURN, q=at(2), qo=off(at(2), 16)) == INVALID
    assert attn(prob(), out=at(0)) == INVALID and attn(prob(), out=at(6)) == INVALID and attn(prob(), lse=at(7)) == INVALID
    assert attn(prob(), out=off(at(3), -512)) == INVALID
    # keys beside values in one tensor [pages, 2, heads, cells, d]: no overlap, so the next check is what refuses
    side = dict(head_dim_v=64, k_page_stride=4096, k_head_stride=1024, k_cell_stride=64, v_page_stride=4096, v_head_stride=1024,
                v_cell_stride=64, num_seqs=4, batch=1, seq_len=15)
    bad = dict(cu=at(10), host=arr(0, 3, 2, 8, 15))
    assert append(prob(**side), vp=off(at(5), 4096), **bad) == INVALID and "decreases" in message()
    assert append(prob(**side), vp=off(at(5), 4094 - 14), **bad) == INVALID and "aliases" in message()
    # queries in place beside keys and values of one projection
    fused = dict(stride_q=512, stride_k=512, stride_v=512, head_dim_v=64, num_seqs=4, batch=1, seq_len=15)
    slices = dict(q=at(0), qo=at(0), k=off(at(0), 512), v=off(at(0), 768), rope=TURN)
    assert append(prob(**fused), **slices, **bad) == INVALID and "decreases" in message()


def test_offsets_are_checked():
    p = prob(batch=1, seq_len=15, num_seqs=4)
    for bad in (arr(1, 3, 8, 8, 15), arr(0, 3, 2, 8, 15), arr(0, 3, 8, 8, 14)):
        assert append(p, cu=at(10), host=bad) == INVALID and attn(p, cu=at(10), host=bad) == INVALID
    assert append(p, host=arr(0, 3, 8, 8, 15)) == INVALID and attn(p, host=arr(0, 3, 8, 8, 15)) == INVALID
    assert append(prob(num_seqs=4), cu=at(10)) == INVALID  # batch of 3
    assert attn(prob(batch=1, num_seqs=-1), cu=at(10)) == INVALID


def test_attention_scalars_and_workspace():
    for kw in (dict(scale=math.nan), dict(scale=math.inf), dict(window=-1)):
        assert attn(prob(), **kw) == INVALID and message()
    long = prob(max_pages=4096)
    st, need = room(long)
    assert st == OK and need > 0
    assert attn(long, n=need - 1) == WORKSPACE and attn(long, ws=None) == WORKSPACE
    assert attn(long, ws=at(7)) == INVALID and "aliases" in message()
    assert kda.library().kda_paged_attn_workspace(ctypes.byref(long), None) == INVALID
    # a packed batch may need more than the plain one of the same rows, and the query covers both
    assert room(prob(batch=1, seq_len=64, num_seqs=64, max_pages=4096))[1] >= room(prob(batch=1, seq_len=64, max_pages=4096))[1]
    # what a window or host offsets spare is never more than the query's answer
    assert room(prob(num_pages=0, max_pages=4096))[0] == OK


def test_empty_calls_launch_nothing():
    for kw in (dict(batch=0), dict(seq_len=0)):
        assert append(prob(**kw), k=None, v=None, table=None if "batch" in kw else at(3), lens=at(4)) == OK
        assert attn(prob(**kw), q=None, out=None, ws=None, n=0, table=at(3)) == OK


def test_binding_checks_its_tensors():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    q, k, kp, table, lens = t(2, 3, 4, 64), t(2, 3, 2, 64), t(9, 2, 16, 64), t(2, 5, dt=torch.int32), t(2, dt=torch.int32)
    freq = torch.ones(16)
    with pytest.raises(ValueError, match="GPU"):
        kda.paged_attention(q, kp, kp, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        kda.paged_append(k, k, kp, kp, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        kda.rope(q, k, freq)
    for bad in (dict(kp=kp.float()), dict(q=q.half(), kp=kp.half()), dict(table=table.long()), dict(lens=lens.long())):
        with pytest.raises(TypeError):
            kda.paged_attention(bad.get("q", q), bad.get("kp", kp), bad.get("kp", kp), bad.get("table", table), bad.get("lens", lens))
    for bad in (dict(kp=kp[:, :, :, ::2]), dict(kp=kp[0]), dict(kp=t(9, 2, 16, 128)), dict(table=table[:1]), dict(table=table[0]),
                dict(table=table.t().contiguous().t()), dict(lens=lens[:1]), dict(q=q[0]), dict(kp=kp[:1].expand(9, 2, 16, 64))):
        with pytest.raises(ValueError):
            kda.paged_attention(bad.get("q", q), bad.get("kp", kp), bad.get("kp", kp), bad.get("table", table), bad.get("lens", lens))
    with pytest.raises(ValueError, match="v_pages"):
        kda.paged_attention(q, kp, kp[:8], table, lens)
    with pytest.raises(ValueError, match="B == 1"):
        kda.paged_attention(q, kp, kp, table, lens, torch.tensor([0, 6], dtype=torch.int32))
    with pytest.raises(ValueError, match="inv_freq"):
        kda.paged_append(k, k, kp, kp, table, lens, q=q)
    with pytest.raises(ValueError, match="without q"):
        kda.paged_append(k, k, kp, kp, table, lens, inv_freq=freq, q_out=q)
    with pytest.raises(ValueError, match="do not fit"):
        kda.paged_append(q, q, kp, kp, table, lens)
    with pytest.raises(TypeError):
        kda.rope(q, k.float(), freq)
    with pytest.raises(TypeError):
        kda.rope(q, k, freq.double())
    with pytest.raises(ValueError, match="one axis"):
        kda.rope(q, k, freq[None])
    with pytest.raises(TypeError):
        kda.rope(q, k, freq, torch.zeros(2, 3, dtype=torch.int64))
    with pytest.raises(ValueError, match="heads of a token"):
        kda.rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, freq)
