"""Host side of the scalar-gate delta rule without a GPU: sizes of workspaces, ranges of launches."""
import ctypes

import pytest

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd import gdn
from gated_delta_rule_45_amd.gdn import GdnProblem


def prob(**kw):
    base = dict(batch=1, seq_len=15, num_seqs=0, num_heads_k=2, num_heads_v=4, head_dim_k=64, head_dim_v=64,
                io_dtype=kda.KDA_BF16, gate_dtype=kda.KDA_F32, state_dtype=kda.KDA_F32, scale=1.0, stride_q=0,
                stride_k=0, stride_v=0)
    base.update(kw)
    return GdnProblem(**base)


def size(query, p):
    n = ctypes.c_size_t(7)
    st = getattr(kda.library(), query)(ctypes.byref(p), ctypes.byref(n))
    return st, n.value


QUERIES = ["kda_gdn_chunk_fwd_workspace", "kda_gdn_chunk_bwd_workspace"]
SHAPES = [dict(batch=3, seq_len=1000), dict(batch=2, seq_len=8192, num_heads_k=1, num_heads_v=2), dict(seq_len=8192),
          dict(seq_len=8191, io_dtype=kda.KDA_F32), dict(seq_len=60), dict(batch=0), dict(seq_len=0)]


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("num_seqs", [-1, 1, 2, 3, 17])
def test_a_plain_batch_may_carry_any_num_seqs(query, kw, num_seqs):
    """num_seqs is ignored without cu_seqlens, by the workspace queries too: what they say is enough for the plain batch."""
    st, need = size(query, prob(**kw))
    assert st == kda.KDA_OK
    st, said = size(query, prob(**kw, num_seqs=num_seqs))
    assert st == kda.KDA_OK and said >= need
    if num_seqs < 1 or kw.get("batch", 1) != 1:  # cannot be a packed batch
        assert said == need


def test_a_packed_batch_has_room_for_its_chunks():
    # 40 sequences of up to 8,192 tokens in all: a chunk slot more for each
    st, need = size("kda_gdn_chunk_bwd_workspace", prob(seq_len=8192, num_seqs=40))
    assert st == kda.KDA_OK and need >= 2 * (8192 // 64 + 40) * 4 * 64 * 64 * 2 + 8192 * 4 * 64 * 2


NULL = [None] * 12


def test_launches_stay_in_range():
    """A launch has at most 2^32 - 1 work-items: more (sequence, head, columns) than that are refused by name."""
    lib = kda.library()
    fwd = lambda p: lib.kda_gdn_chunk_fwd(ctypes.byref(p), *NULL[:11], 0, None)  # noqa: E731
    bwd = lambda p: lib.kda_gdn_chunk_bwd(ctypes.byref(p), *NULL, *NULL[:5], 0, None)  # noqa: E731
    decode = lambda p: lib.kda_gdn_decode(ctypes.byref(p), *NULL[:6], 1 << 30, *NULL[:6])  # noqa: E731
    # a workgroup of 512 for 32 columns of a head
    kw = dict(seq_len=1, num_heads_k=8, num_heads_v=32, head_dim_v=128)
    for call in (fwd, bwd):
        assert call(prob(batch=65535, **kw)) == kda.KDA_ERR_INVALID_ARGUMENT  # these pointers are missing
        assert b"is NULL" in lib.kda_last_error()
        assert call(prob(batch=65536, **kw)) == kda.KDA_ERR_UNSUPPORTED
    for query in QUERIES:
        assert size(query, prob(batch=65536, **kw)) == (kda.KDA_ERR_UNSUPPORTED, 0)
    # a wave of 64
    assert decode(prob(batch=65536, **kw)) == kda.KDA_ERR_INVALID_ARGUMENT and b"is NULL" in lib.kda_last_error()
    assert decode(prob(batch=8 * 65536, **kw)) == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("io", [kda.KDA_BF16, kda.KDA_F32])
def test_the_binding_asks_for_a_workspace_wherever_the_library_uses_one(io):
    """Below the binding's least length the library splits nothing, whatever the heads."""
    least = []
    for batch, heads, dk, dv in ((1, 1, 64, 64), (1, 2, 128, 64), (2, 2, 64, 128), (1, 8, 128, 128), (1, 32, 64, 64)):
        for T in range(1, 300):
            st, need = size("kda_gdn_chunk_fwd_workspace",
                            prob(batch=batch, seq_len=T, num_heads_k=1, num_heads_v=heads, head_dim_k=dk, head_dim_v=dv, io_dtype=io))
            assert st == kda.KDA_OK
            if need:
                least.append(T)
                break
    assert all(T >= gdn._SPLIT_TOKENS for T in least)
    if io == kda.KDA_F32:
        assert min(least) == gdn._SPLIT_TOKENS
