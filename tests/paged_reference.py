"""Rotary positions, the paged cache and attention over it in 64 bits, from their definitions; seeded inputs."""
import math

import torch

F64 = torch.float64


def rotate(x, pos, freq, interleaved, amplitude=1.0, inverse=False):
    """x [..., heads, d], pos [...] -> fp64."""
    x, rot = x.to(F64).clone(), 2 * len(freq)
    a = pos.to(F64)[..., None, None] * freq.to(F64).to(x.device) * (-1 if inverse else 1)
    c, s = amplitude * a.cos(), amplitude * a.sin()
    i = torch.arange(rot // 2, device=x.device)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    x1, x2 = x[..., one], x[..., two]
    x[..., one], x[..., two] = x1 * c - x2 * s, x1 * s + x2 * c
    return x


def sequences(B, T, lens, cu, tokens):
    """(first row, new tokens, cells) of each sequence."""
    if cu is None:
        return [(n * T, T, int(m)) for n, m in enumerate(lens.tolist())]
    c = [min(max(x, 0), tokens) for x in cu.tolist()]
    return [(c[n], max(c[n + 1] - c[n], 0), int(m)) for n, m in enumerate(lens.tolist())]


def append(k, v, kp, vp, table, lens, cu=None):
    """Pools (clones) after the rows of k and v, [B, T, H, d], are stored."""
    kp, vp = kp.clone(), vp.clone()
    B, T = k.shape[:2]
    kf, vf, size, tab = k.flatten(0, 1), v.flatten(0, 1), kp.shape[2], table.tolist()
    for n, (t0, new, cells) in enumerate(sequences(B, T, lens, cu, B * T)):
        for i in range(new):
            p = cells - new + i
            if p < 0 or p // size >= table.shape[1] or not 0 <= tab[n][p // size] < kp.shape[0]:
                continue
            kp[tab[n][p // size], :, p % size] = kf[t0 + i].to(kp.dtype)
            vp[tab[n][p // size], :, p % size] = vf[t0 + i].to(vp.dtype)
    return kp, vp


def attention(q, kp, vp, table, lens, cu=None, scale=None, window=0):
    """out, lse (fp64) and which rows of [B T] a sequence owns; what a token does not see is not touched."""
    B, T, Hq, dk = q.shape
    pages, Hk, size, dv = vp.shape
    G, scale = Hq // Hk, dk ** -0.5 if scale is None else scale
    qf = q.flatten(0, 1).to(F64).unflatten(1, (Hk, G))
    out = torch.zeros(B * T, Hk, G, dv, dtype=F64, device=q.device)
    lse = torch.full((B * T, Hk, G), -math.inf, dtype=F64, device=q.device)
    owned = torch.zeros(B * T, dtype=torch.bool)
    for n, (t0, new, cells) in enumerate(sequences(B, T, lens, cu, B * T)):
        owned[t0:t0 + new] = True
        cell = torch.arange(min(max(cells, 0), table.shape[1] * size), device=q.device)
        page = table[n].to(q.device).long()[cell // size]
        cell = cell[(page >= 0) & (page < pages)]
        page = table[n].to(q.device).long()[cell // size]
        k, v = (x[page, :, cell % size].transpose(0, 1) for x in (kp, vp))  # [Hk, cells, d]
        k, v = k.to(F64), v.to(F64)
        for i in range(new):
            pos = cells - new + i
            a = int((cell <= pos - window).sum()) if window else 0
            b = int((cell <= pos).sum())
            if a >= b:
                continue
            s = scale * (qf[t0 + i] @ k[:, a:b].mT)
            z = s.logsumexp(-1)
            lse[t0 + i] = z
            out[t0 + i] = (s - z[..., None]).exp() @ v[:, a:b]
    return out.reshape(B, T, Hq, dv), lse.reshape(B, T, Hq), owned.reshape(B, T)


def pools(pages, heads, size, dk, dv, dtype, gen, device, cells_first=False, fill=None):
    def one(d):
        shape = (pages, size, heads, d) if cells_first else (pages, heads, size, d)
        x = torch.randn(*shape, generator=gen).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype)
        x = x.to(device)
        return x.transpose(1, 2) if cells_first else x
    return one(dk), one(dv)


def table_of(cells, size, spare, gen, device, extra_pages=2):
    """A shuffled page table for sequences of so many cells; unused entries are -1.  Returns (table, pages)."""
    need = [-(-max(c, 0) // size) for c in cells]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen).to(torch.int32)
    table, at = torch.full((len(cells), max(need + [0]) + extra_pages), -1, dtype=torch.int32), 0
    for n, m in enumerate(need):
        table[n, :m] = perm[at:at + m]
        at += m
    return table.to(device), total
