"""GPU parity of rotary positions, the paged cache and attention over it (rope, rope_bwd, paged_append,
paged_attention) against the fp64 reference (paged_reference.py).

Tolerances, derived before the first run; a rounding is off by at most eps / 2 of the value: e = 2^-24 (fp32), 2^-8 (bf16).
  rotation: per value amplitude (|x1| + |x2|) (the angle's rest, its sine and cosine, their product with the amplitude,
     the product with x, the sum: five roundings of e and the series' 2e-9) -> 5.1 e (|x1| + |x2|) amplitude, and for
     bf16 the result's own 2^-8 |y|
  attention, fp32: sums of at most 128 terms for a score and as many as cells for an output, whose roundings add up in
     squares but for the matrix unit's chains of 4: rel2 <= 1.5e-5, relmax <= 1e-4, the library's bars for fp32
  attention, bf16: weights and outputs are rounded to bf16, u = 2^-8 / sqrt(3) = 2.3e-3 in the 2-norm each, weights'
     errors average like the values they weigh: sqrt(2) u = 3.2e-3, with fp32 sums 3.3e-3 in rel2 for at least 1,024
     values; few values do not average: 2 * 2^-8 = 8e-3; relmax 2e-2, the library's bar
  lse: a score's error, 128 e |q| |k| scale / 4 in chains of four, with |q| |k| scale of about sqrt(d_k) at the default
     scale, below 25 whatever the draw: 6e-5 absolute; at other scales in proportion (|q| |k| below 25 sqrt(d_k))
"""
import math

import pytest
import torch

import paged_reference as ref
import gated_delta_rule_45_amd as kda

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
I32 = torch.int32


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def i32(*x):
    return torch.tensor(x, dtype=I32, device=DEV)


def close(name, got, want, rel2, relmax=None):
    g, w = got.double(), want.double()
    assert g.shape == w.shape, (name, g.shape, w.shape)
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    if g.numel() == 0:
        return
    d, n, m = g - w, float(w.norm()), float(w.abs().max())
    r2 = float(d.norm()) / n if n else float(d.norm())
    rm = float(d.abs().max()) / m if m else float(d.abs().max())
    say(f"  {name}: rel2={r2:.2e} relmax={rm:.2e}")
    assert r2 <= rel2, f"{name}: rel2 {r2:.3e} > {rel2}"
    assert relmax is None or rm <= relmax, f"{name}: relmax {rm:.3e} > {relmax}"


def tol(dtype, n):
    return (1.5e-5, 1e-4) if dtype == F32 else (3.3e-3 if n >= 1024 else 8e-3, 2e-2)


# ---------------------------------------------------------------------------------- rotation --
def check_turned(name, y, x, pos, freq, interleaved, amplitude=1.0, inverse=False):
    want = ref.rotate(x, pos, freq, interleaved, amplitude, inverse)
    rot = 2 * len(freq)
    i = torch.arange(rot // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    size = torch.zeros_like(want)
    both = amplitude * (x[..., one].double().abs() + x[..., two].double().abs())
    size[..., one], size[..., two] = both, both
    bound = 5.1 * 2 ** -24 * size + (2 ** -8 * want.abs() if y.dtype == BF else 0)
    err = (y.double() - want).abs()
    say(f"  {name}: worst error / bound {float((err / bound.clamp_min(1e-30)).max()) if err.numel() else 0:.2f}")
    assert (err <= bound).all(), name
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (2, 37, 5, 2), (3, 700, 16, 3)])
def test_rope(io, d, rot, interleaved, B, T, Hq, Hk):
    g = gen(T + d + rot)
    q, k = rnd(g, B, T, Hq, d, dtype=io), rnd(g, B, T, Hk, d, dtype=io)
    freq, _ = kda.rope_frequencies(rot, device=DEV)
    say(f"[rope {B}x{T}x{Hq}+{Hk} d{d} rot{rot}]")
    pos = torch.arange(T, dtype=I32, device=DEV).expand(B, T)
    yq, yk = kda.rope(q, k, freq, interleaved=interleaved)
    check_turned("q", yq, q, pos, freq, interleaved)
    check_turned("k", yk, k, pos, freq, interleaved)
    far = torch.randint(-(2 ** 20), 2 ** 20, (B, T), generator=g, dtype=I32).to(DEV)
    yq, none = kda.rope(q, None, freq, far, interleaved=interleaved, amplitude=1.375)
    assert none is None
    check_turned("far", yq, q, far, freq, interleaved, 1.375)
    dq, dk = kda.rope_bwd(q, k, freq, far, interleaved=interleaved, amplitude=1.375)
    check_turned("dq", dq, q, far, freq, interleaved, 1.375, inverse=True)
    check_turned("dk", dk, k, far, freq, interleaved, 1.375, inverse=True)


def test_rope_at_the_largest_positions():
    g = gen(3)
    q = rnd(g, 1, 4, 2, 64, dtype=F32)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    pos = i32(2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0).view(1, 4)
    y, _ = kda.rope(q, None, freq, pos)
    # 2^31 * 2 / pi quarter turns in 64 bits are off by up to 2^31 * 2^-53 * 2 / pi * 2 of a quarter: under 1e-6 of a turn's e
    want = ref.rotate(q, pos, freq, False)
    assert float((y.double() - want).abs().max()) <= 2e-6


def test_rope_in_place_and_of_slices():
    g = gen(5)
    wide = rnd(g, 2, 33, 8 * 64)
    q, k, rest = wide[..., :256].unflatten(-1, (4, 64)), wide[..., 256:384].unflatten(-1, (2, 64)), wide[..., 384:]
    freq, amp = kda.rope_frequencies(32, scaling="parts", factor=8.0, original_len=64, device=DEV)
    want_q, want_k = kda.rope(q.contiguous(), k.contiguous(), freq, amplitude=amp)
    yq, yk = kda.rope(q, k, freq, amplitude=amp)
    assert torch.equal(yq, want_q) and torch.equal(yk, want_k)
    before = rest.clone()
    kda.rope(q, k, freq, amplitude=amp, out=(q, k))
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(rest, before)


def test_rope_gradient_by_differences():
    g = gen(6)
    x, delta, dy = (rnd(g, 1, 9, 3, 64, dtype=F32) for _ in range(3))
    freq, _ = kda.rope_frequencies(48, device=DEV)
    a, _ = kda.rope(x + delta, None, freq, amplitude=1.5)
    b, _ = kda.rope(x - delta, None, freq, amplitude=1.5)
    dx, _ = kda.rope_bwd(dy, None, freq, amplitude=1.5)
    lhs = float((dy.double() * (a.double() - b.double())).sum()) / 2
    rhs = float((dx.double() * delta.double()).sum())
    size = float((dy.double().abs() * (a.double().abs() + b.double().abs())).sum())
    assert abs(lhs - rhs) <= 12 * 2 ** -24 * size


# ------------------------------------------------------------------------------------ append --
def batch(g, new, packed):
    """Rows of a batch with `new` tokens a sequence: (B, T, cu)."""
    if packed:
        return 1, sum(new), i32(0, *torch.tensor(new).cumsum(0).tolist())
    return len(new), new[0], None


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("new,cells,size,first", [([1], [1], 16, False), ([3, 3], [3, 40], 32, True),
                                                  ([17, 0, 1, 60], [17, 5, 130, 64], 16, False)])
def test_append(io, dk, dv, new, cells, size, first):
    g = gen(dk + 2 * dv + len(new))
    packed = len(set(new)) > 1
    B, T, cu = batch(g, new, packed)
    k, v, q = (rnd(g, B, T, h, d, dtype=io) for h, d in ((2, dk), (2, dv), (6, dk)))
    table, pages = ref.table_of(cells, size, 2, g, DEV)
    kp, vp = ref.pools(pages, 2, size, dk, dv, io, g, DEV, first)
    lens = i32(*cells)
    say(f"[append {new} {cells} {io}]")
    k0, v0 = kp.clone(), vp.clone()
    assert kda.paged_append(k, v, kp, vp, table, lens, cu) is None
    wk, wv = ref.append(k, v, k0, v0, table, lens, cu)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    # turned on the way: what rope does at the cells' positions
    pos = torch.zeros(B * T, dtype=I32)
    for t0, t, c in ref.sequences(B, T, lens, cu, B * T):
        pos[t0:t0 + t] = torch.arange(c - t, c)
    pos = pos.view(B, T).to(DEV)
    freq, _ = kda.rope_frequencies(48, device=DEV)
    kp, vp = k0.clone(), v0.clone()
    if first:
        kp, vp = k0.transpose(1, 2).contiguous().transpose(1, 2), v0.transpose(1, 2).contiguous().transpose(1, 2)
    yq = kda.paged_append(k, v, kp, vp, table, lens, cu, q=q, inv_freq=freq, interleaved=True, amplitude=1.25)
    tq, tk = kda.rope(q, k, freq, pos, interleaved=True, amplitude=1.25)
    wk, wv = ref.append(tk, v, k0, v0, table, lens, cu)
    assert torch.equal(kp, wk) and torch.equal(vp, wv) and torch.equal(yq, tq)
    check_turned("q", yq, q, pos, freq, True, 1.25)


def test_append_many_rows_and_sequences():
    """Four heads a thread, and more sequences than are searched in LDS."""
    g = gen(8)
    new = torch.randint(0, 9, (1500,), generator=g).tolist()
    cells = [n + int(x) for n, x in zip(new, torch.randint(0, 30, (1500,), generator=g))]
    B, T, cu = batch(g, new, True)
    k, v, q = rnd(g, B, T, 5, 64), rnd(g, B, T, 5, 128), rnd(g, B, T, 10, 64)
    table, pages = ref.table_of(cells, 16, 1, g, DEV)
    kp, vp = ref.pools(pages, 5, 16, 64, 128, BF, g, DEV)
    lens = i32(*cells)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    pos = torch.cat([torch.arange(c - t, c, dtype=I32) for t, c in zip(new, cells)]).view(1, T).to(DEV)
    tq, tk = kda.rope(q, k, freq, pos)
    k0, v0 = kp.cpu(), vp.cpu()
    yq = kda.paged_append(k, v, kp, vp, table, lens, cu, q=q, inv_freq=freq)
    wk, wv = ref.append(tk.cpu(), v.cpu(), k0, v0, table.cpu(), lens.cpu(), cu.cpu())
    assert torch.equal(kp.cpu(), wk) and torch.equal(vp.cpu(), wv) and torch.equal(yq, tq)


def test_append_padding_and_bad_pages():
    g = gen(9)
    new, cells = [4, 4, 4, 4], [2, 20, 64, 200]  # two padding tokens; a bad page; one past the table
    k, v = rnd(g, 4, 4, 1, 64), rnd(g, 4, 4, 1, 64)
    q = rnd(g, 4, 4, 1, 64)
    table = i32(0, 1, 2, 3, 7, -1, 6, 6, 4, 5, 9, 2 ** 30, 8, 10, 11, 12).view(4, 4)
    kp, vp = ref.pools(13, 1, 16, 64, 64, BF, g, DEV)
    lens, freq = i32(*cells), kda.rope_frequencies(64, device=DEV)[0]
    k0, v0, mark = kp.clone(), vp.clone(), torch.full_like(q, 7.0)
    kda.paged_append(k, v, kp, vp, table, lens)
    wk, wv = ref.append(k, v, k0, v0, table, lens)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    y = kda.paged_append(k, v, kp, vp, table, lens, q=q, inv_freq=freq, q_out=mark)
    pos = (lens[:, None] - 4 + torch.arange(4, device=DEV)).to(I32)
    want, _ = kda.rope(q, None, freq, pos)
    assert (y[0, :2] == 7).all()  # padding is left as it is
    assert torch.equal(y[0, 2:], want[0, 2:]) and torch.equal(y[1:], want[1:])


def test_append_of_slices_into_slices():
    """q, k, v of one projection, keys and values of a page in one tensor, queries turned in place."""
    g = gen(10)
    wide = rnd(g, 2, 5, 6 * 64)
    q, k, v = (x.unflatten(-1, (-1, 64)) for x in wide.split([256, 64, 64], -1))
    both = rnd(g, 9, 2, 1, 16, 64)
    kp, vp = both[:, 0], both[:, 1]
    table, lens = i32(3, 1, 8, 2).view(2, 2), i32(21, 5)
    freq = kda.rope_frequencies(64, device=DEV)[0]
    pos = (lens[:, None] - 5 + torch.arange(5, device=DEV)).to(I32)
    tq, tk = kda.rope(q.contiguous(), k.contiguous(), freq, pos)
    wk, wv = ref.append(tk, v.contiguous(), kp, vp, table, lens)
    y = kda.paged_append(k, v, kp, vp, table, lens, q=q, inv_freq=freq, q_out=q)
    assert y is q and torch.equal(q, tq) and torch.equal(kp, wk) and torch.equal(vp, wv)


# --------------------------------------------------------------------------------- attention --
class Case:
    """wide: a table with room for 2^20 cells a sequence, as a server keeps them: calls are then never of little work, and
    sequences of more than 64 rows (bf16) go to the kernel for many."""

    def __init__(self, new, cells, Hq, Hk, dk, dv, io, size, seed=1, first=False, packed=None, q_scale=1.0, wide=False):
        g = gen(seed)
        self.packed = len(set(new)) > 1 if packed is None else packed
        B, T, self.cu = batch(g, new, self.packed)
        self.q = rnd(g, B, T, Hq, dk, dtype=io) * q_scale
        self.table, pages = ref.table_of(cells, size, 2, g, DEV)
        if wide:
            room = torch.full((len(new), 2 ** 20 // size), -1, dtype=I32, device=DEV)
            room[:, :self.table.shape[1]] = self.table
            self.table = room
        self.kp, self.vp = ref.pools(pages, Hk, size, dk, dv, io, g, DEV, first)
        self.lens = i32(*cells)

    def args(self):
        return self.q, self.kp, self.vp, self.table, self.lens, self.cu

    def check(self, label, **kw):
        out, lse = kda.paged_attention(*self.args(), return_lse=True, **kw)
        torch.cuda.synchronize()
        kw = {k: v for k, v in kw.items() if k in ("scale", "window")}
        want, wl, owned = ref.attention(*self.args(), **kw)
        say(f"[{label}] q={tuple(self.q.shape)} {self.q.dtype} pages={tuple(self.kp.shape)}")
        o, w, l, wl = out[owned], want[owned], lse[owned], wl[owned]
        close("out", o, w, *tol(self.q.dtype, o.numel()))
        empty = torch.isinf(wl)
        assert torch.equal(torch.isinf(l) & (l < 0), empty)
        err = float((l.double() - wl)[~empty].abs().max()) if (~empty).any() else 0.0
        say(f"  lse: {err:.2e}")
        assert err <= 6e-5 * max(1.0, abs(kw.get("scale", 0.0)) * self.q.shape[-1] ** 0.5)
        return out, lse


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("new,cells", [([1], [1]), ([1, 1], [17, 16]), ([1], [700]), ([5, 5, 5], [5, 130, 333]),
                                       ([33, 33], [33, 300]), ([150], [150])])
def test_attention_lengths_and_head_sizes(wide, io, dk, dv, new, cells):
    Case(new, cells, 4, 2, dk, dv, io, 16, seed=dk + dv + len(new) + cells[-1], wide=wide).check(f"{new} {cells} {dk}x{dv}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (5, 1), (24, 3), (32, 1), (8, 8)])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_attention_head_groups(wide, io, Hq, Hk, new):
    Case([new] * 2, [new + 90, new], Hq, Hk, 64, 64, io, 32, seed=Hq, wide=wide).check(f"{Hq}/{Hk} x{new}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("size,first", [(16, True), (64, False), (128, True), (1024, False)])
def test_attention_page_sizes(wide, io, size, first):
    Case([1, 70, 0, 2, 9], [1030, 70, 40, 515, 129], 8, 2, 128, 128, io, size, seed=size, first=first, wide=wide).check(f"pages of {size}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 15, 128, 200, 5000, 2 ** 31 - 1])
def test_attention_windows(wide, io, window):
    Case([1, 130, 6], [900, 300, 1300], 6, 2, 64, 128, io, 16, seed=window % 97, wide=wide).check(f"window {window}", window=window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_attention_scales(wide, io, scale):
    """Sharp rows too: scores of some 30."""
    Case([1, 20, 40], [500, 20, 333], 4, 1, 64, 64, io, 16, seed=3, wide=wide).check(f"scale {scale}", scale=scale)


@pytest.mark.parametrize("Hq,wide", [(4, False), (32, True)])
@pytest.mark.parametrize("io", [BF, F32])
def test_attention_rows_without_cells(io, Hq, wide):
    """Sequences with fewer cells than new tokens, without cells, without tokens; rows that no sequence owns."""
    c = Case([4, 6, 0, 20, 1], [2, 0, 9, 11, 1], Hq, 2, 64, 64, io, 16, seed=4, wide=wide)
    c.check("empty rows")
    c.lens = i32(2, -5, 9, 11, 1)
    c.check("negative length")
    c.cu = i32(0, 4, 10, 10, 25, 26)  # five rows fewer are owned
    c.lens = i32(2, 0, 9, 11, 1)
    mark, ml = torch.full((1, 31, Hq, 64), 7.0, dtype=io, device=DEV), torch.full((1, 31, Hq), 7.0, device=DEV)
    out, lse = c.check("padded", out=mark, lse=ml)
    assert (out[:, 26:] == 7).all() and (lse[:, 26:] == 7).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_does_not_see_what_is_masked(wide, io, bad):
    """NaN and infinities in cells behind a sequence's end, in other pages, before the window, and in cells of the chunk that
    only later tokens see; those tokens get them."""
    new, cells = [1, 30, 7, 150], [77, 130, 90, 290]
    c = Case(new, cells, 4, 2, 64, 128, io, 16, seed=6, wide=wide)
    pages = c.kp.shape[0]
    used = torch.zeros(pages, 16, dtype=torch.bool)
    for n, m in enumerate(cells):
        for p in range(m):
            used[c.table[n, p // 16], p % 16] = True
    hole = ~used.to(DEV)
    for x in (c.kp, c.vp):
        x.masked_fill_(hole[:, None, :, None], bad)
    c.check("behind the end")
    for n, p in ((1, 115), (3, 200), (2, 88)):  # a cell in the middle of the chunk
        c.vp[c.table[n, p // 16], :, p % 16, 3:5] = bad
    out, lse = kda.paged_attention(*c.args(), return_lse=True)
    want, wl, _ = ref.attention(*c.args())
    ok = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
    close("finite", out[ok], want[ok], *tol(io, int(ok.sum())))
    assert torch.isfinite(lse).all()
    # with a window the same cell leaves sight again
    out = kda.paged_attention(*c.args(), window=9)
    want, _, _ = ref.attention(*c.args(), window=9)
    ok = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
    close("window", out[ok], want[ok], *tol(io, int(ok.sum())))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
def test_attention_pages_that_do_not_exist(io, wide):
    c = Case([1, 40, 3], [600, 200, 333], 4, 2, 64, 64, io, 32, seed=7, wide=wide)
    c.table[0, 3] = -1
    c.table[0, 9] = 2 ** 30
    c.table[1, 1] = c.kp.shape[0]
    c.table[2, :] = -7  # nothing at all
    c.check("holes")
    c.table = c.table[:, :4].contiguous()  # 128 cells: positions go on behind them
    c.check("short table")
    c.kp, c.vp = c.kp[:0], c.vp[:0]
    out, lse = kda.paged_attention(*c.args(), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("new,cells", [([1], [5000]), ([3], [4099]), ([1] * 5, [3000, 1, 0, 2500, 4096]),
                                       ([70, 1, 1], [2100, 3500, 3]), ([1] * 300, [(i * 37) % 1900 for i in range(300)])])
def test_attention_split_over_the_cells(io, new, cells):
    c = Case(new, cells, 4, 1, 64, 128, io, 64, seed=len(new))
    out, lse = c.check(f"{len(new)} sequences of up to {max(cells)}")
    again, l2 = kda.paged_attention(*c.args(), return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, l2)
    if c.cu is not None:
        host, l3 = kda.paged_attention(*c.args(), return_lse=True, cu_seqlens_host=c.cu.cpu())
        close("with host offsets", host, out, *tol(io, out.numel()))
    c.check("window", window=1100)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_holes_beside_infinities(wide, io, bad):
    """Every other page missing and a cell of each page that is there infinite: all tokens see them."""
    c = Case([5, 40], [700, 900], 2, 1, 64, 64, io, 16, seed=21, wide=wide)
    c.table[:, ::2] = -1
    for n in (0, 1):
        for page in c.table[n].tolist():
            if page >= 0:
                c.vp[page, 0, 3, 7] = bad
    out, lse = kda.paged_attention(*c.args(), return_lse=True)
    want, wl, _ = ref.attention(*c.args())
    ok = torch.isfinite(want)
    assert not ok[..., 7].any() and torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
    close("finite", out[ok], want[ok], *tol(io, int(ok.sum())))
    assert float((lse.double() - wl).abs().max()) <= 6e-5


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
def test_attention_one_chunk_among_empty_sequences(wide, io):
    """No more tokens than sequences, all of them one sequence's; and offsets that decrease on the device."""
    new = [0] * 60
    new[17] = 41
    cells = [5] * 60
    cells[17] = 400
    Case(new, cells, 4, 1, 64, 128, io, 16, seed=22, wide=wide).check("one chunk")
    c = Case([30, 10, 20], [100, 50, 70], 4, 2, 64, 64, io, 16, seed=23, wide=wide)
    c.cu = i32(0, 30, 25, 60)  # the second is empty, the third starts inside the first
    out, lse = kda.paged_attention(*c.args(), return_lse=True)
    torch.cuda.synchronize()
    want, _, _ = ref.attention(*c.args())
    close("first rows", out[:, :25], want[:, :25], *tol(io, 25 * 4 * 64))
    close("last rows", out[:, 30:], want[:, 30:], *tol(io, 30 * 4 * 64))


def test_attention_more_sequences_than_threads():
    g = gen(24)
    n = 1200
    cells = torch.randint(0, 90, (n,), generator=g).tolist()
    new = [int(c > 0) for c in cells]
    cells[700], new[700] = 6000, 1
    cells[30], new[30] = 3000, 33
    c = Case(new, cells, 4, 2, 64, 64, BF, 32, seed=25)
    c.check("1,200 sequences")
    c.check("window", window=50)


def test_attention_of_a_large_pool():
    """Cells behind 2^31 elements of the pool."""
    g = gen(11)
    pages, size = 2 ** 31 // (64 * 1024) + 5, 1024  # [pages, 1, 1024, 64] bf16: 4.3 GB
    kp = torch.zeros(pages, 1, size, 64, dtype=BF, device=DEV)
    vp = torch.zeros(pages, 1, size, 64, dtype=BF, device=DEV)
    table, lens = i32(pages - 1, 0, pages - 3, -1).view(1, 4), i32(2500)
    k, v, q = rnd(g, 1, 2500, 1, 64), rnd(g, 1, 2500, 1, 64), rnd(g, 1, 2500, 2, 64)
    kda.paged_append(k, v, kp, vp, table, lens)
    assert torch.equal(kp[pages - 1, 0], k[0, :1024, 0]) and torch.equal(vp[pages - 3, 0, :452], v[0, 2048:, 0])
    small = [x[[0, pages - 3, pages - 1]].contiguous() for x in (kp, vp)]
    for rows in (q, q[:, -1:].contiguous()):
        a = kda.paged_attention(rows, kp, vp, table, lens)
        b = kda.paged_attention(rows, *small, i32(2, 0, 1, -1).view(1, 4), lens)
        assert torch.equal(a, b)


def test_attention_wide_tables_and_strides():
    """A table whose rows are apart, queries as slices, keys and values of a page in one tensor."""
    g = gen(12)
    c = Case([1, 1, 1], [200, 33, 64], 4, 2, 64, 64, BF, 16, seed=13)
    want = kda.paged_attention(*c.args())
    wide = torch.full((3, 99), -1, dtype=I32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    assert torch.equal(kda.paged_attention(c.q, c.kp, c.vp, wide[:, :c.table.shape[1]], c.lens), want)
    both = torch.stack([c.kp, c.vp], 1)
    fused = torch.cat([c.q.flatten(-2), rnd(g, 3, 1, 128)], -1)[..., :256].unflatten(-1, (4, 64))
    assert torch.equal(kda.paged_attention(fused, both[:, 0], both[:, 1], c.table, c.lens), want)


def test_attention_on_streams_and_in_graphs():
    c = Case([1, 1, 40, 2], [3000, 7, 900, 2000], 8, 2, 128, 128, BF, 64, seed=14)
    want, wl = kda.paged_attention(*c.args(), return_lse=True)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [kda.paged_attention(*c.args(), return_lse=True, stream=s) for s in side]  # a workspace each
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, wl) for o, l in got)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    with torch.cuda.stream(s):
        kda.paged_attention(*c.args(), out=out, lse=lse)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        kda.paged_attention(*c.args(), out=out, lse=lse)
    for i in range(3):
        out.fill_(9)
        c.lens.sub_(1)  # the lengths are the device's
        eager, el = kda.paged_attention(*c.args(), return_lse=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, el), i


def test_rope_and_append_on_streams_and_in_graphs():
    g = gen(31)
    k, v, q = rnd(g, 3, 2, 2, 64), rnd(g, 3, 2, 2, 64), rnd(g, 3, 2, 4, 64)
    table, pages = ref.table_of([40, 18, 5], 16, 1, g, DEV)
    wide = torch.full((3, 50), -1, dtype=I32, device=DEV)
    wide[:, :table.shape[1]] = table
    k0, v0 = ref.pools(pages, 2, 16, 64, 64, BF, g, DEV)
    freq, lens = kda.rope_frequencies(64, device=DEV)[0], i32(40, 18, 5)
    torch.cuda.synchronize()

    def call(kp, vp, s=None, tab=table):
        y = kda.paged_append(k, v, kp, vp, tab, lens, q=q, inv_freq=freq, stream=s)
        return y, kda.rope(y, None, freq, stream=s)[0]

    kp, vp = k0.clone(), v0.clone()
    want = call(kp, vp)
    torch.cuda.synchronize()
    for s, tab in ((torch.cuda.Stream(), table), (torch.cuda.Stream(), wide[:, :table.shape[1]])):
        a, b = k0.clone(), v0.clone()
        torch.cuda.synchronize()
        got = call(a, b, s, tab)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a, kp) and torch.equal(b, vp)
    graph, s, a, b = torch.cuda.CUDAGraph(), torch.cuda.Stream(), k0.clone(), v0.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = call(a, b)
    for i in range(3):
        lens.sub_(1)
        a.copy_(k0), b.copy_(v0), kp.copy_(k0), vp.copy_(v0)
        graph.replay()
        want = call(kp, vp)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a, kp) and torch.equal(b, vp), i


def test_a_serving_run():
    """Prompts in chunks, then token by token, through rope, cache and attention: as attention over the whole."""
    g, H, Hk, d, size = gen(15), 4, 2, 64, 16
    total, chunks = 83, [40, 21, 1, 1, 3, 1, 16]
    assert sum(chunks) == total
    freq, amp = kda.rope_frequencies(32, scaling="base", factor=4.0, device=DEV)
    q, k, v = (rnd(g, 2, total, h, d) for h in (H, Hk, Hk))
    table, pages = ref.table_of([total, total], size, 0, g, DEV)
    kp, vp = ref.pools(pages, Hk, size, d, d, BF, g, DEV, fill=math.nan)
    outs, at = [], 0
    for t in chunks:
        lens, cut = i32(at + t, at + t), slice(at, at + t)
        part = [x[:, cut].contiguous() for x in (q, k, v)]
        yq = kda.paged_append(part[1], part[2], kp, vp, table, lens, q=part[0], inv_freq=freq, amplitude=amp)
        outs.append(kda.paged_attention(yq, kp, vp, table, lens))
        at += t
    tq, tk = kda.rope(q, k, freq, amplitude=amp)
    s = torch.einsum("bthgd,bshd->bhgts", tq.double().unflatten(2, (Hk, H // Hk)), tk.double()) * d ** -0.5
    s = s.masked_fill(~torch.ones(total, total, dtype=torch.bool, device=DEV).tril(), -math.inf).softmax(-1)
    want = torch.einsum("bhgts,bshd->bthgd", s, v.double()).flatten(2, 3)
    got = torch.cat(outs, 1)
    close("run", got, want, *tol(BF, got.numel()))


def test_beside_the_delta_rule():
    """A decode step of a hybrid: three delta-rule layers on state slots and one over the pages, on one stream."""
    g, N, H, Hk, d = gen(16), 3, 4, 2, 64
    state = torch.zeros(5, H, d, d, device=DEV)
    slots = i32(4, 0, 2)
    c = Case([1] * N, [50, 20, 1], H, Hk, d, d, BF, 16, seed=17)
    x = [rnd(g, N, 1, h, d) for h in (Hk, Hk, H)]
    x[0], x[1] = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF) for t in x[:2])
    gate = -torch.rand(N, 1, H, generator=g).to(DEV)
    y = c.q
    for _ in range(3):
        o = kda.gdn_decode(x[0], x[1], x[2], gate, gate.exp(), state, slots, scale=d ** -0.5)
        y = y + kda.norm_gate(o.contiguous(), y.contiguous(), torch.ones(d, device=DEV))
    kda.paged_append(x[1], x[2][:, :, :Hk].contiguous(), c.kp, c.vp, c.table, c.lens)
    c.q = y.contiguous()
    c.check("hybrid")
