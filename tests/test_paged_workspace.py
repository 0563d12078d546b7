"""The room that kda_paged_attn_workspace names is enough for every call on the problem.  The calls get addresses that are never
read: without a GPU they end at the launch at the latest, and where there is one these tests do not run."""
import ctypes
import os
import random

import pytest

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd.paged import PagedProblem

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="launches on made-up addresses: only without a GPU")

at = lambda i: ctypes.c_void_p(0x100000000000 * (i + 1))  # noqa: E731  aligned, far apart


def problem(batch, T, Hq, Hk, dk, dv, io, page, pages, num_seqs=0):
    return PagedProblem(batch, T, num_seqs, Hq, Hk, dk, dv, io, page, pages, 1 << 14)


def room(p):
    n = ctypes.c_size_t(7)
    assert kda.library().kda_paged_attn_workspace(ctypes.byref(p), ctypes.byref(n)) == kda.KDA_OK
    return n.value


def call(p, size, window=0, cu=False, host=None):
    """Status and message of a call with so many bytes of workspace."""
    lib = kda.library()
    if host is not None:
        host = (ctypes.c_int32 * len(host))(*host)
    st = lib.kda_paged_attn(ctypes.byref(p), at(0), at(1), at(2), at(3), at(4), at(5) if cu else None, host, 1.0, window, at(6), None,
                            at(7) if size else None, size, None)
    return st, lib.kda_last_error().decode()


def enough(p, **kw):
    st, message = call(p, room(p), **kw)
    assert st == kda.KDA_ERR_HIP, (message, [(n, getattr(p, n)) for n, _ in p._fields_], kw)


@pytest.mark.parametrize("T,N,Hq,Hk,d,io,page,pages,window", [
    (4096, 4, 32, 8, 128, kda.KDA_BF16, 64, 66, 1024), (8192, 1, 32, 8, 128, kda.KDA_BF16, 64, 130, 1024),
    (16384, 1, 32, 8, 128, kda.KDA_BF16, 64, 258, 4096), (1024, 6, 32, 8, 128, kda.KDA_BF16, 64, 18, 1000),
    (1024, 6, 32, 8, 128, kda.KDA_BF16, 64, 18, 1100), (4096, 4, 16, 4, 64, kda.KDA_F32, 64, 66, 2047),
])
def test_prompts_under_a_window(T, N, Hq, Hk, d, io, page, pages, window):
    p = problem(N, T, Hq, Hk, d, d, io, page, pages)
    for w in (0, 1, window - 1, window, 2 * window, 2 ** 31 - 1):
        enough(p, window=w)


def log(rng, a, b):
    return int(round(a * (b / a) ** rng.random()))


def draw(rng, packed):
    hk = rng.choice([1, 2, 3, 4, 8, 16, 64, 300, 600])
    tokens, n = log(rng, 1, 20000), log(rng, 1, 600)
    shape = (1, tokens) if packed else (n, max(1, tokens // n))
    return problem(*shape, hk * rng.choice([1, 2, 4, 5, 8]), hk, rng.choice([64, 128]), rng.choice([64, 128]),
                   rng.choice([kda.KDA_BF16, kda.KDA_F32]), rng.choice([16, 64, 256]), log(rng, 1, 4000), n if packed else 0)


@pytest.mark.parametrize("packed", [False, True])
def test_any_window(packed):
    rng, reached = random.Random(11 + packed), 0
    for _ in range(6000):
        p = draw(rng, packed)
        cells = p.max_pages * p.page_size
        enough(p, window=rng.choice([0, log(rng, 1, 2 * cells), log(rng, 1, 5000)]), cu=packed)
        reached += room(p) > 0
    assert reached > 1000


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("pages", [4, 16, 64, 128, 512, 2048])
@pytest.mark.parametrize("lens", [[24] + [1] * 30 + [0] * 30, [1] * 10 + [90] + [0] * 117, [0] * 500 + [500], [64] * 8 + [0] * 504])
def test_long_sequences_among_empty_ones_by_host_offsets(lens, pages):
    """No more tokens than sequences: without host offsets one launch, with them two."""
    for hq, hk in ((32, 8), (4, 1), (96, 96)):
        p = problem(1, sum(lens), hq, hk, 128, 128, kda.KDA_BF16, 64, pages, len(lens))
        for window in (0, 700):
            enough(p, cu=True, host=offsets(lens), window=window)
            enough(p, cu=True, window=window)


def test_any_host_offsets():
    rng, few = random.Random(13), 0
    for _ in range(6000):
        p = draw(rng, True)
        cut = sorted(rng.randint(0, p.seq_len) for _ in range(p.num_seqs - 1))
        if rng.random() < 0.5:  # some sequences hold all tokens
            cut = sorted(rng.choice(cut[:3] or [0]) for _ in cut)
        enough(p, cu=True, host=[0, *cut, p.seq_len], window=rng.choice([0, 0, log(rng, 1, 5000)]))
        few += p.seq_len <= p.num_seqs and p.io_dtype == kda.KDA_BF16
    assert few > 500


@pytest.mark.parametrize("io,T,Hk,most", [(kda.KDA_BF16, 33, 8, (2 ** 32 - 1) // 512 // 8),  # tiles of 256 rows, 512 threads
                                          (kda.KDA_F32, 16, 8, (2 ** 32 - 1) // 256 // 8)])  # of 16 rows, 256 threads
def test_more_workgroups_than_a_launch_has(io, T, Hk, most):
    """A tile a sequence and head; the work-items of a launch are at most 2^32 - 1."""
    enough(problem(most, T, Hk, Hk, 64, 64, io, 64, 64))
    for n in (most + 1, most + most // 2):
        p, size = problem(n, T, Hk, Hk, 64, 64, io, 64, 64), ctypes.c_size_t(7)
        if n * T * Hk >= 2 ** 31:
            continue
        assert kda.library().kda_paged_attn_workspace(ctypes.byref(p), ctypes.byref(size)) == kda.KDA_ERR_UNSUPPORTED
        assert size.value == 0
        st, message = call(p, 1 << 40)
        assert st == kda.KDA_ERR_UNSUPPORTED and "workgroups" in message
