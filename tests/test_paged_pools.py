"""Which pools of keys and values paged_append takes for one memory: strides of every nesting, and layouts that hold keys beside
values.  Every call has offsets that decrease, which is checked behind the pools: nothing is ever launched."""
import ctypes
import itertools
import random

import pytest

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd.paged import PagedProblem

BASE = 0x500000000000


def meet(size, ks, vs, apart, dk, dv, io=kda.KDA_BF16):
    """Whether pools of size (pages, heads, cells), strides in elements, `apart` bytes between them, are refused."""
    pages, heads, cells = size
    p = PagedProblem(1, 15, 4, heads, heads, dk, dv, io, cells, 7, pages, 0, 0, 0, 0, *ks, *vs)
    at = lambda i: ctypes.c_void_p(0x100000000000 * (i + 1))  # noqa: E731
    lib, offsets = kda.library(), (ctypes.c_int32 * 5)(0, 3, 2, 8, 15)
    st = lib.kda_paged_append(ctypes.byref(p), at(0), at(1), None, None, at(2), at(3), at(5), offsets, ctypes.c_void_p(BASE),
                              ctypes.c_void_p(BASE + apart), None, None)
    message = lib.kda_last_error().decode()
    assert st == kda.KDA_ERR_INVALID_ARGUMENT and ("aliases" in message or "decreases" in message), message
    if "aliases" in message:
        assert "k_pages" in message and "v_pages" in message
    return "aliases" in message


def strides(size, order, d, pad=(0, 0, 0)):
    """Strides of axes laid out from the outermost of `order` in; pad: elements behind an axis's entries."""
    out, step = [0, 0, 0], d
    for i in reversed(order):
        out[i] = step + pad[i]
        step = out[i] * size[i]
    return out


@pytest.mark.parametrize("io", [kda.KDA_BF16, kda.KDA_F32])
def test_keys_beside_values(io):
    size, e = (5, 3, 32), 2 if io == kda.KDA_BF16 else 4
    pages, heads, cells = size
    for d in (64, 128):
        whole = heads * cells * d
        for name, s, apart in [
            ("pages, 2, heads, cells, d", (2 * whole, cells * d, d), whole), ("pages, heads, 2, cells, d", (2 * whole, 2 * cells * d, d), cells * d),
            ("pages, heads, cells, 2 d", (2 * whole, 2 * cells * d, 2 * d), d), ("pages, cells, 2, heads, d", (2 * whole, d, 2 * heads * d), heads * d),
            ("pages, cells, heads, 2 d", (2 * whole, 2 * d, 2 * heads * d), d), ("2, pages, heads, cells, d", (whole, cells * d, d), pages * whole),
        ]:
            for a in (apart, -apart):
                assert not meet(size, s, s, a * e, d, d, io), name
                for shift in (-16, 16):  # (whole pools that move apart do not meet)
                    assert meet(size, s, s, a * e + shift, d, d, io) == (name[0] == "p" or a * shift < 0), name
            assert meet(size, s, s, 0, d, d, io)
    # keys of 64 beside values of 128: in a cell, and the heads of a cell
    s = (heads * cells * 192, cells * 192, 192)
    assert not meet(size, s, s, 64 * e, 64, 128, io) and meet(size, s, s, 48 * e, 64, 128, io)
    k, v = (heads * cells * 192, 64, heads * 192), (heads * cells * 192, 128, heads * 192)
    assert not meet(size, k, v, heads * 64 * e, 64, 128, io) and meet(size, k, v, heads * 64 * e - 16, 64, 128, io)
    assert meet(size, k, v, heads * 64 * e + 16, 64, 128, io)  # the last values reach the next cell's keys
    # whole pools one behind the other, in other orders
    k, v = strides(size, (0, 1, 2), 64), strides(size, (0, 2, 1), 128)
    assert not meet(size, k, v, pages * heads * cells * 64 * e, 64, 128, io)
    assert not meet(size, k, v, -pages * heads * cells * 128 * e, 64, 128, io)
    assert meet(size, k, v, (pages * heads * cells * 64 - 64) * e, 64, 128, io)


def granules(size, s, d, start):
    """16-byte pieces of a bf16 pool, strides in elements, start in pieces."""
    cells = (i * s[0] + j * s[1] + c * s[2] for i, j, c in itertools.product(*map(range, size)))
    return {start + x // 8 + k for x in cells for k in range(d // 8)}


def test_against_every_byte():
    rng, seen = random.Random(5), [0, 0]
    for _ in range(400):
        size = (rng.randint(1, 3), rng.randint(1, 3), rng.choice([16, 32]))
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        order = rng.sample(range(3), 3)
        pad = [rng.choice([0, 0, 8, 64, 128, 192, 1024, 4096]) for _ in range(3)]
        k = strides(size, order, max(dk, dv), pad)
        v = k if rng.random() < 0.8 else strides(size, rng.sample(range(3), 3), dv, pad)
        mine = granules(size, k, dk, 0)
        last = max(mine)
        apart = rng.choice([0, 8, dk // 8, last + 1, last, *(x // 8 for x in k), *(x // 8 + dk // 8 for x in k), rng.randint(0, last)])
        apart *= rng.choice([1, -1])
        want = not mine.isdisjoint(granules(size, v, dv, apart))
        got = meet(size, k, v, 16 * apart, dk, dv)
        assert got == want if v is k else got or not want, (size, k, v, dk, dv, apart)
        seen[want] += 1
    assert min(seen) > 80, seen
