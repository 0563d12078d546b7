"""Queries turned in place on their way: what q_out the binding takes for q (on the CPU, in place of the library)."""
import pytest
import torch

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd import paged

BF = torch.bfloat16


class Calls:
    def __init__(self, monkeypatch):
        self.q = self.out = self.stride = None
        monkeypatch.setattr(paged, "library", lambda: self)
        monkeypatch.setattr(paged, "_Launch", lambda device, stream: self)

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        pass

    def kda_paged_append(self, p, k, v, q, rope, table, lens, cu, host, kp, vp, out, stream):
        self.q, self.out, self.stride = q, out, p._obj.stride_q
        return kda.KDA_OK


def call(q, out):
    B, T = q.shape[:2]
    k, pages = torch.zeros(B, T, 2, 64, dtype=BF), torch.zeros(9, 2, 16, 64, dtype=BF)
    return kda.paged_append(k, k, pages, pages.clone(), torch.zeros(B, 5, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), q=q,
                            inv_freq=torch.ones(32), q_out=out)


def test_q_out(monkeypatch):
    calls = Calls(monkeypatch)
    wide = torch.zeros(2, 5, 512, dtype=BF)
    slices = [wide[..., :256].unflatten(-1, (4, 64)) for _ in range(2)]  # two views of the same tokens
    dense = torch.zeros(2, 5, 4, 64, dtype=BF)
    for q, out, in_place in [(slices[0], slices[0], True), (slices[0], slices[1], True), (dense, dense, True),
                             (dense, dense.view(2, 5, 4, 64), True), (slices[0], dense, False), (slices[0], None, False)]:
        y = call(q, out)
        assert out is None or y is out
        assert (calls.q, calls.out, calls.stride) == (q.data_ptr(), y.data_ptr(), 0 if q is dense else 512)
        assert (calls.q == calls.out) == in_place
    # dense tokens over the first part of a projection: neither q in place nor memory of its own
    over = wide.view(-1)[:2 * 5 * 256].view(2, 5, 4, 64)
    assert over.data_ptr() == slices[0].data_ptr() and over.is_contiguous()
    calls.out = None
    with pytest.raises(ValueError, match="q_out"):
        call(slices[0], over)
    with pytest.raises(ValueError, match="contiguous"):
        call(dense, slices[0])
    with pytest.raises(TypeError):
        call(dense, dense.float())
    assert calls.out is None
