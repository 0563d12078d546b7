"""What the binding hands to the paged calls for block tables of every stride: read back through the pointer and the
stride that C gets, as the kernels read them (on the CPU, in place of the library)."""
import ctypes

import pytest
import torch

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd import paged

I32 = torch.int32


class Calls:
    """Stands in for the library: takes the entries of the table that a call names."""

    def __init__(self, monkeypatch):
        self.table = None
        monkeypatch.setattr(paged, "library", lambda: self)
        monkeypatch.setattr(paged, "_Launch", lambda device, stream: self)

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        pass

    def read(self, p, table):
        p, n = p._obj, 0
        n = p.num_seqs or p.batch
        step = p.stride_table or p.max_pages
        assert step >= p.max_pages
        x = ctypes.cast(table, ctypes.POINTER(ctypes.c_int32))
        self.table = [[x[i * step + j] for j in range(p.max_pages)] for i in range(n)]
        return kda.KDA_OK

    def kda_paged_attn_workspace(self, p, need):
        return kda.KDA_OK

    def kda_paged_attn(self, p, q, kp, vp, table, *rest):
        return self.read(p, table)

    def kda_paged_append(self, p, k, v, q, rope, table, *rest):
        return self.read(p, table)


def zeros(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt)


def tables(n, m):
    """Name, table [n, m] of entries 0, 1, ...; whether its rows are one."""
    dense = torch.arange(n * m, dtype=I32).view(n, m)
    wide = torch.full((n, m + 3), -9, dtype=I32)
    wide[:, :m] = dense
    return [("dense", dense, False), ("slice", wide[:, :m], False), ("expanded", dense[:1].expand(n, m), n > 1),
            ("expanded slice", wide[:1, :m].expand(n, m), n > 1), ("last row", wide[-1:, :m].expand(n, m), n > 1)]


@pytest.mark.parametrize("n,m", [(1, 1), (3, 5), (4, 1), (2, 9)])
@pytest.mark.parametrize("packed", [False, True])
def test_the_table_that_c_reads(monkeypatch, n, m, packed):
    calls = Calls(monkeypatch)
    B, T = (1, n) if packed else (n, 1)
    cu = torch.arange(n + 1, dtype=I32) if packed else None
    q, k, pages, lens = zeros(B, T, 4, 64), zeros(B, T, 2, 64), zeros(9, 2, 16, 64), zeros(n, dt=I32)
    for name, table, shared in tables(n, m):
        calls.table = None
        kda.paged_attention(q, pages, pages, table, lens, cu)
        assert calls.table == table.tolist(), name
        calls.table = None
        if shared:
            with pytest.raises(ValueError, match="share"):
                kda.paged_append(k, k, pages, pages.clone(), table, lens, cu)
            assert calls.table is None
        else:
            kda.paged_append(k, k, pages, pages.clone(), table, lens, cu)
            assert calls.table == table.tolist(), name


def test_tables_without_entries(monkeypatch):
    calls = Calls(monkeypatch)
    q, pages = zeros(3, 1, 4, 64), zeros(9, 2, 16, 64)
    kda.paged_attention(q, pages, pages, zeros(1, 0, dt=I32).expand(3, 0), zeros(3, dt=I32))
    assert calls.table == [[], [], []]


def test_rows_that_overlap_are_refused_by_name():
    """Rows 2 entries apart that hold 5: the call gets their stride and refuses it."""
    q, pages, lens = zeros(3, 1, 4, 64), zeros(9, 2, 16, 64), zeros(3, dt=I32)
    p, _ = paged._paged(q, 3, 1, 4, pages, pages, torch.arange(9, dtype=I32).as_strided((3, 5), (2, 1)), lens, None, 0, 0, 0)
    assert (p.stride_table, p.max_pages) == (2, 5)
    need = ctypes.c_size_t(0)
    assert kda.library().kda_paged_attn_workspace(ctypes.byref(p), ctypes.byref(need)) == kda.KDA_ERR_INVALID_ARGUMENT
    assert "stride_table" in kda.library().kda_last_error().decode()
