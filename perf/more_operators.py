"""Timed cases of a hybrid model's full-attention layers: rotary positions, the paged key-value cache and its reader.

Three operators, each as the library offers it (``own`` true) and in plain torch (``own`` false):

* ``rope``    queries and keys rotated by their positions, or (``back``) the gradients of that
* ``append``  new tokens' keys and values into a paged cache, keys (and queries) rotated on the way
* ``attn``    attention of each sequence's new tokens, one or many, over its pages

A head's pairs (x1, x2) become a (x1 cos t - x2 sin t, x1 sin t + x2 cos t) with t = position * frequency.  Query head
h of Hq reads key-value head h // (Hq // Hkv).  The i-th of a sequence's `new` tokens sits at kv_len - new + i and
sees the cells up to its own (the last `window` of them).  Cell p of a sequence is cell p % page of page table[p // page].
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases --
def listed():
    # past: cells of a sequence before its new tokens; ragged: lengths spread below T and past; single: so many
    # sequences have one new token whatever T; order: the page's axes, heads or cells first; fused: views of a projection
    r = dict(op="rope", N=4, T=4096, Hq=16, Hk=16, d=128, io="bf16", rot=128, pairs="half", scaled="none", at=0,
             back=False, fused=False)
    a = dict(op="append", ragged=0, single=0, past=0, Hq=32, Hk=8, dk=128, dv=128, io="bf16", page=64, order="heads", rot=128,
             pairs="half", scaled="none", fused=False)
    s = dict(op="attn", ragged=0, single=0, past=0, Hq=32, Hk=8, dk=128, dv=128, io="bf16", page=64, order="heads", window=0,
             lse=False, fused=False)
    return [
        # a short prompt in full precision: latency
        dict(r, name="rope_short", N=1, T=256, Hq=2, Hk=2, d=64, io="fp32", rot=64),
        # the forward of a training step
        dict(r, name="rope_train", Hk=8, fused=True),
        # the gradients of a step on long documents: neighbouring pairs, half of the head, scaled far positions
        dict(r, name="rope_grads", Hq=32, Hk=8, rot=64, pairs="next", scaled="parts", at=126976, back=True),
        # one user's next token: latency
        dict(a, name="append_one", N=1, T=1, past=1000, Hq=16),
        # the next token of a full batch, no rotation, pages with the cells first
        dict(a, name="append_batch", N=256, T=1, ragged=3, past=2048, order="cells", page=16, rot=0),
        # ragged prompts packed into one row, slices of one projection, half of the head rotated
        dict(a, name="append_prompts", N=64, T=4096, ragged=1, rot=64, scaled="linear", fused=True),
        # one user's next token after an odd number of cells, in full precision: latency
        dict(s, name="attn_one", N=1, T=1, past=1001, Hq=4, Hk=2, dk=64, dv=64, io="fp32", page=16),
        # the decode step of a batch of ragged contexts: the cache's traffic
        dict(s, name="attn_batch", N=64, T=1, ragged=4, past=8192),
        # one very long context
        dict(s, name="attn_long", N=1, T=1, past=131071, order="cells", page=256),
        # drafted tokens checked at once, the last 1,024 cells in sight
        dict(s, name="attn_draft", N=96, T=4, past=3001, page=16, window=1024, Hq=16, lse=True),
        # whole prompts
        dict(s, name="attn_prompts", N=4, T=4096, Hq=32, fused=True),
        # a serving step: chunks of long prompts beside other users' single tokens
        dict(s, name="attn_chunks", N=12, T=1024, ragged=5, single=8, past=32768, Hq=16, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn"])
    hk = rng.choice([1, 2, 3, 4, 8])
    hq = hk * rng.choice([1, 2, 4, 5, 8] if hk < 8 else [1, 2, 4])
    io = rng.choice(["bf16", "bf16", "fp32"])
    c = dict(op=op, Hq=hq, Hk=hk, io=io, fused=rng.random() < 0.5)
    turn = dict(pairs=rng.choice(["half", "next"]), scaled=rng.choice(["none", "linear", "parts"]))
    if op == "rope":
        d = rng.choice([64, 128])
        return dict(c, N=rng.randint(1, 4), T=_log(rng, 1, 4096), d=d, rot=rng.choice([d, d // 2, 48]), at=rng.choice([0, _log(rng, 1, 1 << 20)]),
                    back=rng.random() < 0.5, **turn)
    c |= dict(dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128, 256]),
              order=rng.choice(["heads", "cells"]), ragged=rng.choice([0, rng.randrange(1, 1000)]), single=0)
    if op == "append":
        return dict(c, N=_log(rng, 1, 64), T=rng.choice([1, _log(rng, 1, 2048)]), past=_log(rng, 1, 2048),
                    rot=rng.choice([0, 16, 48, c["dk"]]), **turn)
    c |= dict(window=rng.choice([0, 0, _log(rng, 1, 2048)]), lse=rng.random() < 0.5)
    kind = rng.choice(["single", "few", "chunks"])
    if kind == "chunks":
        n = rng.randint(1, 6)
        return dict(c, N=n, T=_log(rng, 16, 1024), past=rng.choice([0, _log(rng, 1, 16384)]), single=rng.choice([0, n // 2]))
    return dict(c, N=_log(rng, 1, 64), T=1 if kind == "single" else rng.randint(2, 9), past=_log(rng, 1, 8192))


def _seqs(case):
    """New tokens and cells (with those) of each sequence."""
    n, gen = case["N"], torch.Generator().manual_seed(case["ragged"])
    if not case["ragged"]:
        new, past = [case["T"]] * n, [case["past"]] * n
    else:
        new = torch.randint(1, case["T"] + 1, (n,), generator=gen).tolist()
        past = torch.randint(case["past"] // 16, case["past"] + 1, (n,), generator=gen).tolist()
    new[: case["single"]] = [1] * case["single"]
    return new, [a + b for a, b in zip(new, past)]


def _frequencies(rot, scaled):
    """Rotations per position of each pair, in 64 bits, and the amplitude that goes with them."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    if scaled == "linear":  # positions squeezed into a quarter
        return f / 4, 1.0
    if scaled == "parts":  # pairs that turn less than once in 4,096 positions are squeezed, those above 32 turns kept
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * (keep + (1 - keep) / 32), 0.1 * math.log(32) + 1
    return f, 1.0


# ------------------------------------------------------------------------------------ inputs --
def _heads(rows, widths, dt, fused, gen):
    """Tensors [*rows, heads, d] for (heads, d) in widths; `fused`: views of one projection's output."""
    x = [torch.randn(*rows, h, d, generator=gen, device=DEV).to(dt) for h, d in widths]
    if not fused:
        return x
    parts = torch.cat([t.flatten(-2) for t in x], -1).split([h * d for h, d in widths], -1)
    return [t.unflatten(-1, w) for t, w in zip(parts, widths)]


def _pool(pages, heads, cells, d, case, gen):
    """Pages [pages, heads, cells, d], in memory in the case's order, holding what earlier sequences left there."""
    shape = (pages, heads, cells, d) if case["order"] == "heads" else (pages, cells, heads, d)
    x = torch.randn(*shape, generator=gen, device=DEV, dtype=_DT[case["io"]])
    return x if case["order"] == "heads" else x.transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, hq, hk = _DT[case["io"]], case["Hq"], case["Hk"]
    st = dict(case=case)
    if case.get("rot"):
        f, st["amplitude"] = _frequencies(case["rot"], case["scaled"])
        st["freq"] = f.float().to(DEV)
    if case["op"] == "rope":
        rows = (case["N"], case["T"])
        st["q"], st["k"] = _heads(rows, [(hq, case["d"]), (hk, case["d"])], dt, case["fused"], gen)
        st["pos"] = (case["at"] + torch.arange(case["T"], dtype=torch.int32)).expand(rows).contiguous().to(DEV)
        return st
    new, cells = _seqs(case)
    rows = (1, sum(new)) if case["ragged"] or case["single"] else (case["N"], case["T"])
    st["cu"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV) if case["ragged"] or case["single"] else None
    st["lens"] = torch.tensor(cells, dtype=torch.int32).to(DEV)
    dk, dv, page = case["dk"], case["dv"], case["page"]
    st["q"], st["k"], st["v"] = _heads(rows, [(hq, dk), (hk, dk), (hk, dv)], dt, case["fused"], gen)
    need = [-(-c // page) for c in cells]
    free = torch.randperm(sum(need) + 3, generator=gen, device=DEV).to(torch.int32)
    table, at = torch.zeros(case["N"], max(need) + 2, dtype=torch.int32, device=DEV), 0
    for n, m in enumerate(need):
        table[n, :m] = free[at:at + m]
        at += m
    st["table"] = table
    st["kp"], st["vp"] = (_pool(len(free), hk, page, d, case, gen) for d in (dk, dv))
    return st


# -------------------------------------------------------------------------------- plain forms --
def _turned(x, pos, st, back=False):
    """x [..., heads, d] in 32 bits with its leading channels rotated; pos [...]."""
    case, x = st["case"], x.float()
    rot = case.get("rot", 0)
    if not rot:
        return x
    t = pos.double()[..., None, None] * st["freq"].double()
    c, s = t.cos().float() * st["amplitude"], t.sin().float() * st["amplitude"]
    if back:
        s = -s
    y, rest = x[..., :rot], x[..., rot:]
    if case["pairs"] == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _places(st, tokens):
    """Sequence and position of each of the batch's tokens."""
    at = torch.arange(tokens, device=DEV)
    if st["cu"] is None:
        T = st["case"]["T"]
        n = at // T
        return n, st["lens"].long()[n] - T + at % T
    cu = st["cu"].long()
    n = torch.searchsorted(cu[1:], at, right=True)
    return n, st["lens"].long()[n] - cu[n + 1] + at


def _plain_attn(st):
    case = st["case"]
    hq, hk, page = case["Hq"], case["Hk"], case["page"]
    new, cells = _seqs(case)
    q = st["q"].flatten(0, 1)
    outs, lses, at = [], [], 0
    for n, (t, c) in enumerate(zip(new, cells)):
        p = st["table"][n, : -(-c // page)].long()
        k, v = (x[p].transpose(0, 1).flatten(1, 2)[:, :c].float() for x in (st["kp"], st["vp"]))  # [Hk, cells, d]
        x = q[at:at + t].float().unflatten(1, (hk, hq // hk)).permute(1, 2, 0, 3).flatten(1, 2)  # [Hk, G new, dk]
        s = (x @ k.mT * case["dk"] ** -0.5).unflatten(1, (hq // hk, t))
        pos, j = c - t + torch.arange(t, device=DEV)[:, None], torch.arange(c, device=DEV)
        hidden = j > pos
        if case["window"]:
            hidden = hidden | (j <= pos - case["window"])
        s = s.masked_fill_(hidden, -math.inf)
        m = s.amax(-1, keepdim=True)
        s = s.sub_(m).exp_()
        z = s.sum(-1, keepdim=True)
        o = (s.flatten(1, 2) @ v).unflatten(1, (hq // hk, t)) / z
        outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
        lses.append((m + z.log())[..., 0].permute(2, 0, 1).flatten(1))
        at += t
    rows = st["q"].shape[:2]
    out = torch.cat(outs).unflatten(0, rows).to(st["q"].dtype)
    return (out, torch.cat(lses).unflatten(0, rows)) if case["lse"] else out


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    if case["op"] == "rope":
        return [_turned(st[n], st["pos"], st, case["back"]).to(st[n].dtype) for n in ("q", "k")]
    if case["op"] == "attn":
        return _plain_attn(st)
    rows, dt = st["q"].shape[:2], st["q"].dtype
    n, pos = _places(st, rows[0] * rows[1])
    turned = [_turned(st[x].flatten(0, 1), pos, st).to(dt) for x in ("q", "k")]
    page, cell = st["table"][n, pos // case["page"]].long(), pos % case["page"]
    st["kp"][page, :, cell] = turned[1]
    st["vp"][page, :, cell] = st["v"].flatten(0, 1)
    return turned[0].unflatten(0, rows) if case["rot"] else None, st["kp"], st["vp"]


def _run_own(st):
    import gated_delta_rule_45_amd as kda

    case = st["case"]
    turn = {}
    if case.get("rot"):
        turn = dict(inv_freq=st["freq"], interleaved=case["pairs"] == "next", amplitude=st["amplitude"])
    if case["op"] == "rope":
        return (kda.rope_bwd if case["back"] else kda.rope)(st["q"], st["k"], positions=st["pos"], **turn)
    if case["op"] == "append":
        q = st["q"] if case["rot"] else None
        return kda.paged_append(st["k"], st["v"], st["kp"], st["vp"], st["table"], st["lens"], st["cu"], q=q, **turn), st["kp"], st["vp"]
    return kda.paged_attention(st["q"], st["kp"], st["vp"], st["table"], st["lens"], st["cu"], scale=case["dk"] ** -0.5,
                               window=case["window"], return_lse=case["lse"])


# ------------------------------------------------------------------------------------- work --
def work(case):
    e, hq, hk = (2 if case["io"] == "bf16" else 4), case["Hq"], case["Hk"]
    if case["op"] == "rope":
        n = case["N"] * case["T"]
        return {"bytes": 2 * n * (hq + hk) * case["d"] * e + 4 * n, "flops": 3 * n * (hq + hk) * case["rot"]}
    new, cells = _seqs(case)
    dk, dv, n = case["dk"], case["dv"], sum(new)
    if case["op"] == "append":
        q = hq * dk if case["rot"] else 0
        return {"bytes": 2 * n * (q + hk * (dk + dv)) * e, "flops": 3 * n * (hq + hk) * case["rot"]}
    w, pairs, read = case["window"], 0, 0
    for t, c in zip(new, cells):
        first = c - t + 1  # cells that the first new token sees, without the window
        pairs += sum(min(first + i, w) for i in range(t)) if w else t * first + t * (t - 1) // 2
        read += min(c, w + t - 1) if w else c
    return {"bytes": n * hq * (dk + dv) * e + read * hk * (dk + dv) * e + (4 * n * hq if case["lse"] else 0),
            "flops": 2 * pairs * hq * (dk + dv)}


# ------------------------------------------------------------------------------------ exact --
def _wheel(x, pos, st, back=False):
    """The rotation as a product of complex numbers in 64 bits."""
    case, x = st["case"], x.double()
    rot = case.get("rot", 0)
    if not rot:
        return x
    half = case["pairs"] == "half"
    z = x[..., :rot].unflatten(-1, (2, -1) if half else (-1, 2))
    z = torch.complex(*z.unbind(-2 if half else -1))
    t = pos.double()[..., None] * st["freq"].double() * (-1 if back else 1)
    z = torch.view_as_real(z * torch.polar(torch.full_like(t, st["amplitude"]), t).unsqueeze(-2))
    return torch.cat([(z.transpose(-1, -2) if half else z).flatten(-2), x[..., rot:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return [_wheel(st[n], st["pos"], st, case["back"]) for n in ("q", "k")]
    new, cells = _seqs(case)
    rows, table, page = st["q"].shape[:2], st["table"].tolist(), case["page"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(c - t, c) for t, c in zip(new, cells)]).to(DEV)
        q, k = (_wheel(st[x].flatten(0, 1), pos, st) for x in ("q", "k"))
        kp, vp = st["kp"].double(), st["vp"].double()
        v, at = st["v"].flatten(0, 1).double(), 0
        for n, (t, c) in enumerate(zip(new, cells)):
            a = c - t
            while a < c:  # page by page
                b = min(c, (a // page + 1) * page)
                x = at + a - (c - t)
                kp[table[n][a // page], :, a % page: a % page + b - a] = k[x:x + b - a].transpose(0, 1)
                vp[table[n][a // page], :, a % page: a % page + b - a] = v[x:x + b - a].transpose(0, 1)
                a = b
            at += t
        return q.unflatten(0, rows) if case["rot"] else None, kp, vp
    hq, hk, dv = case["Hq"], case["Hk"], case["dv"]
    q = st["q"].flatten(0, 1)
    out = q.new_empty(len(q), hq, dv, dtype=torch.float64)
    lse = q.new_empty(len(q), hq, dtype=torch.float64)
    at = 0
    for n, (t, c) in enumerate(zip(new, cells)):
        for h in range(hk):
            cell = torch.arange(c, device=DEV)
            p = st["table"][n].long()[cell // page]
            k, v = (x[p, h, cell % page].double() for x in (st["kp"], st["vp"]))
            for a in range(0, t, 512):  # a few tokens and one group of heads at a time
                b = min(t, a + 512)
                pos = torch.arange(c - t + a, c - t + b, device=DEV)[:, None, None]
                see = (cell <= pos) & ((cell > pos - case["window"]) if case["window"] else True)
                g = slice(h * (hq // hk), (h + 1) * (hq // hk))
                x = torch.einsum("tgd,cd->tgc", q[at + a:at + b, g].double(), k) / math.sqrt(case["dk"])
                z = torch.logsumexp(torch.where(see, x, -math.inf), -1)
                out[at + a:at + b, g] = torch.where(see, (x - z[..., None]).exp(), 0.0) @ v
                lse[at + a:at + b, g] = z
        at += t
    out, lse = out.unflatten(0, rows), lse.unflatten(0, rows)
    return (out, lse) if case["lse"] else out
