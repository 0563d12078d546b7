"""Calls of the paged cache that its users make beside the plain ones: tables that share a row.  Against the same calls
on copies and the fp64 reference (paged_reference.py), with the tolerances of test_gpu_paged.py."""
import pytest
import torch

import gated_delta_rule_45_amd as kda
from test_gpu_paged import BF, F32, Case, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_sequences_that_share_a_context(io, new):
    """One row of the table for all sequences, as a view of it and as a copy."""
    say(f"[shared table, {new} tokens, {io}]")
    c = Case([new] * 4, [300, 170, 1, 299], 4, 2, 64, 128, io, 16, seed=41)
    row = c.table[:1, :19]
    c.table = row.expand(4, 19)
    want, wl = kda.paged_attention(c.q, c.kp, c.vp, c.table.contiguous(), c.lens, return_lse=True)
    out, lse = c.check("expanded")
    assert torch.equal(out, want) and torch.equal(lse, wl)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = kda.paged_attention(*c.args(), stream=s)  # the copy is made on the call's stream
    torch.cuda.synchronize()
    assert torch.equal(out, want)
