"""Calls of the paged cache that its users make beside the plain ones: tables that share a row, windows over prompts, offsets
known on the host, keys beside values in a page, queries in place, positions of the caller. Against the same calls on copies
and the fp64 reference (paged_reference.py), with the tolerances of test_gpu_paged.py."""
import pytest
import torch

import gated_delta_rule_45_amd as kda
import paged_reference as ref
from test_gpu_paged import BF, DEV, F32, Case, batch, check_turned, gen, i32, rnd, say

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


@pytest.mark.parametrize("io,new,cells,Hq,Hk,window,wide", [
    (BF, 2048, [2048, 2048], 32, 8, 1024, False),  # every tile a workgroup: no room is needed
    (BF, 2048, [2048, 2040], 32, 8, 1024, True),
    (F32, 2200, [2200], 4, 4, 2100, False),
    (BF, 600, [4000], 8, 2, 1500, True),           # parts and their join
    (F32, 100, [3000, 2900], 2, 1, 1500, True),
])
def test_plain_prompts_under_a_window(io, new, cells, Hq, Hk, window, wide):
    """Without a workspace of the caller's: the binding asks for the room of the problem, which has no window."""
    say(f"[window {window} over {new} of {cells}, {io}]")
    c = Case([new] * len(cells), cells, Hq, Hk, 64, 128, io, 64, seed=42, packed=False, wide=wide)
    out, lse = c.check("prompts", window=window)
    again, l2 = kda.paged_attention(*c.args(), window=window, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("new,cells,Hq,Hk", [
    ([1] * 10 + [90] + [0] * 117, [(i * 331) % 4000 for i in range(10)] + [4000] + [0] * 117, 32, 8),
    ([24] + [1] * 30 + [0] * 30, [2000] + [(i * 577) % 1900 for i in range(30)] + [0] * 30, 32, 8),
    ([0] * 300 + [300], [0] * 300 + [5000], 4, 1),
    ([64] * 2 + [0] * 126, [3000, 2000] + [0] * 126, 48, 48),  # not as many parts as without a limit to their room
])
@pytest.mark.parametrize("window", [0, 700])
def test_long_sequences_among_single_tokens_by_host_offsets(new, cells, Hq, Hk, window):
    """No more tokens than sequences: one launch, and two that share their room where the host's offsets show long sequences."""
    say(f"[{sum(new)} tokens in {len(new)} sequences, {Hq}/{Hk} heads, window {window}]")
    c = Case(new, cells, Hq, Hk, 64, 128, BF, 64, seed=43, packed=True)
    host = c.cu.cpu()
    c.check("without", window=window)
    out, lse = c.check("with", window=window, cu_seqlens_host=host)
    again, l2 = kda.paged_attention(*c.args(), window=window, return_lse=True, cu_seqlens_host=host)
    assert torch.equal(out, again) and torch.equal(lse, l2)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    a, b = torch.empty_like(out), torch.empty_like(lse)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        kda.paged_attention(*c.args(), window=window, out=a, lse=b, cu_seqlens_host=host)
    for i in range(3):
        a.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, lse), i


def beside(layout, pages, heads, size, dk, dv, io):
    """Keys and values [pages, heads, size, d] as slices of one tensor."""
    if layout == "cell":      # a head's key, then its value
        x = torch.zeros(pages, heads, size, dk + dv, dtype=io, device=DEV)
        return x[..., :dk], x[..., dk:]
    if layout == "cells first":
        x = torch.zeros(pages, size, heads, dk + dv, dtype=io, device=DEV).transpose(1, 2)
        return x[..., :dk], x[..., dk:]
    if layout == "heads":     # all keys of a cell, then all values
        x = torch.zeros(pages, size, heads * (dk + dv), dtype=io, device=DEV)
        return (t.unflatten(-1, (heads, -1)).transpose(1, 2) for t in (x[..., :heads * dk], x[..., heads * dk:]))
    x = torch.zeros(pages, heads, size * (dk + dv), dtype=io, device=DEV)  # all keys of a head in a page, then its values
    return (t.unflatten(-1, (size, -1)) for t in (x[..., :size * dk], x[..., size * dk:]))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("layout", ["cell", "cells first", "heads", "head"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("wide", [False, True])
def test_keys_beside_values_in_a_page(io, layout, dk, dv, wide):
    """Appended to and read where keys and values are slices of one tensor, as in pools of their own."""
    say(f"[{layout}, {dk}x{dv}, {io}]")
    c = Case([70, 1, 3], [300, 41, 90], 4, 2, dk, dv, io, 32, seed=44, wide=wide)
    g = gen(45)
    k, v = rnd(g, 1, 74, 2, dk, dtype=io), rnd(g, 1, 74, 2, dv, dtype=io)
    kp, vp = beside(layout, c.kp.shape[0], 2, 32, dk, dv, io)
    kp.copy_(c.kp), vp.copy_(c.vp)
    for pools in ((kp, vp), (c.kp, c.vp)):
        kda.paged_append(k, v, *pools, c.table, c.lens, c.cu)
    assert torch.equal(kp, c.kp) and torch.equal(vp, c.vp)
    want = kda.paged_attention(*c.args())
    c.kp, c.vp = kp, vp
    out, _ = c.check(layout)
    assert torch.equal(out, want)


def test_queries_in_place_by_a_second_view():
    """q_out as another view of q's tokens, which lie apart."""
    g = gen(46)
    wide = rnd(g, 3, 2, 6 * 64)
    q, k, v = (x.unflatten(-1, (-1, 64)) for x in wide.split([256, 64, 64], -1))
    rest = wide[..., 256:].clone()
    kp, vp = rnd(g, 9, 1, 16, 64), rnd(g, 9, 1, 16, 64)
    table, lens, freq = i32(3, 1, 8, 2, 5, 4).view(3, 2), i32(21, 5, 2), kda.rope_frequencies(64, device=DEV)[0]
    want = kda.paged_append(k, v, kp, vp, table, lens, q=q, inv_freq=freq)
    view = wide[..., :256].unflatten(-1, (4, 64))
    assert kda.paged_append(k, v, kp, vp, table, lens, q=q, inv_freq=freq, q_out=view) is view
    assert torch.equal(q, want) and torch.equal(wide[..., 256:], rest)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,cells", [([3, 3, 3], [3, 40, 1]), ([17, 0, 1, 60], [17, 5, 130, 64]), ([900, 2100], [900, 3000])])
def test_append_at_positions_that_are_not_the_cells(io, interleaved, new, cells):
    """Positions of the caller's (a scrolled cache, a picture's rows): what rope does at them, in the tokens' cells."""
    g = gen(47 + len(new))
    packed = len(set(new)) > 1
    B, T, cu = batch(g, new, packed)
    k, v, q = (rnd(g, B, T, h, d, dtype=io) for h, d in ((2, 64), (2, 128), (6, 64)))
    table, pages = ref.table_of(cells, 16, 2, g, DEV)
    kp, vp = ref.pools(pages, 2, 16, 64, 128, io, g, DEV)
    lens, freq = i32(*cells), kda.rope_frequencies(48, device=DEV)[0]
    pos = torch.randint(-(2 ** 20), 2 ** 20, (B, T), generator=g, dtype=torch.int32).to(DEV)
    say(f"[positions {new} {cells} {io}]")
    mark, k0, v0 = torch.full_like(q, 7.0), kp.cpu(), vp.cpu()
    y = kda.paged_append(k, v, kp, vp, table, lens, cu, q=q, inv_freq=freq, positions=pos, interleaved=interleaved, amplitude=1.25,
                         q_out=mark)
    tq, tk = kda.rope(q, k, freq, pos, interleaved=interleaved, amplitude=1.25)
    check_turned("q", tq, q, pos, freq, interleaved, 1.25)
    wk, wv = ref.append(tk.cpu(), v.cpu(), k0, v0, table.cpu(), lens.cpu(), None if cu is None else cu.cpu())
    assert torch.equal(kp.cpu(), wk) and torch.equal(vp.cpu(), wv)
    there = torch.zeros(B * T, dtype=torch.bool)
    for t0, t, c in ref.sequences(B, T, lens, cu, B * T):
        there[t0 + max(0, t - c):t0 + t] = True  # (padding has no cell and is left as it is)
    there = there.view(B, T).to(DEV)
    assert torch.equal(y[there], tq[there]) and (y[~there] == 7).all()
