"""Rotary positions and the paged key-value cache of a hybrid's full-attention layers: argument checks and marshalling
for the kda_rope* and kda_paged_* entry points of libkda.so.

    rope            pairs of a head's leading channels turned by position * frequency (rope_bwd: back)
    paged_append    new tokens' keys and values into the pages of their sequences, turned on the way
    paged_attention softmax attention of the new tokens, one or many per sequence, over those pages

Query head h of Hq reads key-value head h // (Hq // Hkv).  Pages: [num_pages, Hkv, page_size, d], a view of any order
in memory whose last axis is dense (pages that hold cells first: pages.transpose(1, 2); keys and values may be slices of one
tensor), page_size a power of two from 16 on.  block_table: int32 [N, max_pages]; cell p of sequence n is cell p % page_size of page block_table[n, p //
page_size].  kv_lens: int32 [N], the cells of each sequence WITH its new tokens, for both calls: the i-th of `new`
tokens is cell kv_lens[n] - new + i.  A plain batch is q, k, v [N, T, heads, d], T new tokens each; a packed one
[1, tokens, heads, d] with cu_seqlens int32 [N + 1].  q, k and v may be slices of one projection's output.

Rows that no sequence owns, and appended tokens whose cell would be negative (padding), are not written: in tensors
allocated here they hold whatever the memory held.  Attention gives 0 to a row without cells.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _P, _check, _io_code, library
from .gdn import _dense, _host_i32, _Launch, _ptr, _room, _rows, _want

__all__ = ["rope", "rope_bwd", "rope_frequencies", "paged_append", "paged_attention"]

_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


class RopeProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "seq_len", "num_heads_q", "num_heads_k", "head_dim", "io_dtype",
                                              "rot_dim", "interleaved", "inverse")] + \
        [("amplitude", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("stride_q", "stride_k", "stride_q_out", "stride_k_out")]


class PagedProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "seq_len", "num_seqs", "num_heads_q", "num_heads_kv", "head_dim_k",
                                              "head_dim_v", "io_dtype", "page_size", "max_pages")] + \
        [(n, ctypes.c_int64) for n in ("num_pages", "stride_table", "stride_q", "stride_k", "stride_v", "k_page_stride",
                                       "k_head_stride", "k_cell_stride", "v_page_stride", "v_head_stride", "v_cell_stride")]


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float), ("inv_freq", _P),
                ("positions", _P)]


def declare(lib: ctypes.CDLL) -> None:
    size, prob, status = ctypes.c_size_t, ctypes.POINTER(PagedProblem), ctypes.c_int
    lib.kda_rope.argtypes = [ctypes.POINTER(RopeProblem)] + [_P] * 7
    lib.kda_rope_frequencies.argtypes = [ctypes.c_int32, ctypes.c_double, ctypes.c_int32, ctypes.c_double, ctypes.c_int64,
                                         ctypes.c_double, ctypes.c_double, _P, _P]
    lib.kda_paged_append.argtypes = [prob] + [_P] * 3 + [ctypes.POINTER(Rope)] + [_P] * 8
    lib.kda_paged_attn.argtypes = [prob] + [_P] * 7 + [ctypes.c_float, ctypes.c_int32] + [_P] * 3 + [size, _P]
    lib.kda_paged_attn_workspace.argtypes = [prob, ctypes.POINTER(size)]
    for f in (lib.kda_rope, lib.kda_rope_frequencies, lib.kda_paged_append, lib.kda_paged_attn, lib.kda_paged_attn_workspace):
        f.restype = status


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, slow: float = 1.0, fast: float = 32.0, device=None):
    """Frequencies (fp32 [rot_dim / 2]) and the amplitude that goes with them.  scaling: "none"; "linear" (positions
    squeezed by factor); "base" (a larger base, the slowest pair squeezed by factor); "parts" (pairs that turn less than
    `slow` times in original_len positions squeezed by factor, those above `fast` times kept, a ramp in between).  device: None
    for the CPU."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling is {scaling!r}, expected one of {sorted(_SCALINGS)}")
    freq, amplitude = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float32, device="cpu"), ctypes.c_float(1.0)
    _check(library().kda_rope_frequencies(rot_dim, base, _SCALINGS[scaling], factor, original_len, slow, fast, _ptr(freq),
                                          ctypes.addressof(amplitude)))
    return freq.to(device) if device is not None else freq, amplitude.value


def _rotation(inv_freq, positions, rows, like):
    """Rotated channels, after the checks of the tensors."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a tensor of one axis")
    _want(inv_freq, "inv_freq", torch.float32, inv_freq.shape, like)
    if positions is not None:
        _want(positions, "positions", torch.int32, rows, like)
    return 2 * inv_freq.shape[0]


def _turn(q, k, inv_freq, positions, interleaved, amplitude, inverse, out, stream):
    shape = q.shape
    if len(shape) != 4 or (k is not None and len(k.shape) != 4):
        raise ValueError("q and k must be [B, T, heads, d]")
    B, T, Hq, d = shape
    Hk, dt = (0 if k is None else k.shape[2]), q.dtype
    io = _io_code(dt)
    lq = 0 if q.is_contiguous() else _rows(q, "q", dt, shape, q.device)
    lk = 0 if k is None or _dense(k, dt, (B, T, Hk, d), q) else _rows(k, "k", dt, (B, T, Hk, d), q.device)
    rot = _rotation(inv_freq, positions, (B, T), q)
    with _Launch(q.device, stream) as handle:
        lqo = lko = 0
        if out is None:
            qo, ko = q.new_empty(shape), None if k is None else k.new_empty(k.shape)
        else:
            qo, ko = out
            lqo = 0 if _dense(qo, dt, shape, q) else _rows(qo, "q_out", dt, shape, q.device)
            if k is not None:
                lko = 0 if _dense(ko, dt, k.shape, q) else _rows(ko, "k_out", dt, k.shape, q.device)
        p = RopeProblem(B, T, Hq, Hk, d, io, rot, interleaved, inverse, amplitude, lq, lk, lqo, lko)
        _check(library().kda_rope(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(positions), _ptr(inv_freq), _ptr(qo),
                                  _ptr(ko) if k is not None else None, handle))
    return qo, ko


def rope(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor, positions: Optional[torch.Tensor] = None, *,
         interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Rotary positions.  q: [B, T, Hq, d], k: [B, T, Hk, d] or None (bf16 or fp32); inv_freq: fp32, half as many as the
    leading channels that turn (a multiple of 16 of them); positions: int32 [B, T] or None (0 .. T - 1); interleaved:
    neighbouring channels are a pair, else channel i and i + len(inv_freq); out: (q_out, k_out), which may be (q, k).
    Returns (q_out, k_out)."""
    return _turn(q, k, inv_freq, positions, bool(interleaved), amplitude, 0, out, stream)


def rope_bwd(d_q: torch.Tensor, d_k: Optional[torch.Tensor], inv_freq: torch.Tensor, positions: Optional[torch.Tensor] = None,
             *, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Gradients of rope: those of its results, turned back.  Returns (d_q, d_k) with respect to its arguments."""
    return _turn(d_q, d_k, inv_freq, positions, bool(interleaved), amplitude, 1, out, stream)


def _pool(t, name: str, like: torch.Tensor):
    """A pool's shape and strides (the checks in one go first, as in _dense)."""
    if isinstance(t, torch.Tensor) and t.dtype == like.dtype and t.get_device() == like.get_device() and t.dim() == 4:
        s = t.stride()
        if s[3] == 1 and s[0] > 0 and s[1] > 0 and s[2] > 0:
            return t.shape, s
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.get_device() != like.get_device() or t.device.type != like.device.type:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [pages, heads, page_size, d]")
    s = t.stride()
    if s[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: the last axis must be dense (strides {s})")
    if any(a == 0 and b > 1 for a, b in zip(s, t.shape)):
        raise ValueError(f"{name}: cells share memory (strides {s})")
    return t.shape, s


def _shared(block_table) -> bool:
    """Sequences that share one row of the table (an expanded one)."""
    return block_table.shape[0] > 1 and block_table.shape[1] > 0 and block_table.stride(0) == 0


def _paged(like, B, T, Hq, k_pages, v_pages, block_table, kv_lens, cu_seqlens, lq, lk, lv):
    (pages, Hk, cells, dk), ks = _pool(k_pages, "k_pages", like)
    vshape, vs = _pool(v_pages, "v_pages", like)
    if vshape[:3] != k_pages.shape[:3]:
        raise ValueError(f"v_pages has shape {tuple(vshape)}, expected {(pages, Hk, cells)} and d_v")
    n = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("a packed batch (cu_seqlens) needs B == 1")
        n = cu_seqlens.numel() - 1
        if n < 0:
            raise ValueError("cu_seqlens needs at least one entry")
        _want(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), like)
    _want(kv_lens, "kv_lens", torch.int32, (n,), like)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [sequences, pages]")
    most = block_table.shape[1]
    lt = 0
    if not _dense(block_table, torch.int32, (n, most), like):
        if block_table.shape[0] != n or block_table.dtype != torch.int32 or block_table.device != like.device or \
                (most > 1 and block_table.stride(1) != 1):
            _want(block_table, "block_table", torch.int32, (n, most), like)
        lt = block_table.stride(0) if n > 1 else 0  # (0, sequences that share a row: the caller's to settle, as C reads it as dense)
    p = PagedProblem(B, T, n if cu_seqlens is not None else 0, Hq, Hk, dk, vshape[3], _io_code(like.dtype), cells, most, pages, lt,
                     lq, lk, lv, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
    return p, n


def _in_place(out, x: torch.Tensor) -> bool:
    return out is x or (isinstance(out, torch.Tensor) and out.data_ptr() == x.data_ptr() and out.dtype == x.dtype
                        and out.shape == x.shape and out.stride() == x.stride() and out.get_device() == x.get_device())


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                 kv_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *, q: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, interleaved: bool = False,
                 amplitude: float = 1.0, q_out: Optional[torch.Tensor] = None, cu_seqlens_host=None, stream=None):
    """Store the new tokens' k [B, T, Hkv, d_k] and v [B, T, Hkv, d_v] in their sequences' pages (written in place).
    With inv_freq (and positions, interleaved, amplitude as for rope; positions None: the token's cell) the keys are
    turned on the way, and the queries q [B, T, Hq, d_k] with them, into q_out (allocated here when None; may be q).
    A token whose page is not in the pool is not stored.  Sequences that share a row of an expanded block_table are refused.
    Returns q_out, or None without q."""
    shape, dt = k.shape, k.dtype
    if len(shape) != 4 or len(v.shape) != 4:
        raise ValueError("k and v must be [B, T, heads, d]")
    B, T, Hk, dk = shape
    lk = 0 if k.is_contiguous() else _rows(k, "k", dt, shape, k.device)
    vs = (B, T, Hk, v.shape[3])
    lv = 0 if _dense(v, dt, vs, k) else _rows(v, "v", dt, vs, k.device)
    Hq, lq, turn = Hk, 0, None
    if inv_freq is not None:
        turn = Rope(_rotation(inv_freq, positions, (B, T), k), bool(interleaved), amplitude, _ptr(inv_freq), _ptr(positions))
    elif positions is not None or q is not None:
        raise ValueError("q and positions are for a rotation: inv_freq is needed")
    if q is not None:
        if len(q.shape) != 4:
            raise ValueError("q must be [B, T, heads, d]")
        Hq = q.shape[2]
        lq = 0 if _dense(q, dt, (B, T, Hq, dk), k) else _rows(q, "q", dt, (B, T, Hq, dk), k.device)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    p, n = _paged(k, B, T, Hq, k_pages, v_pages, block_table, kv_lens, cu_seqlens, lq, lk, lv)
    if _shared(block_table):
        raise ValueError("block_table: sequences share a row, their tokens would share cells")
    if (p.num_heads_kv, p.head_dim_k, p.head_dim_v) != (Hk, dk, v.shape[3]):
        raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} do not fit pages of {p.num_heads_kv} heads of "
                         f"{p.head_dim_k} and {p.head_dim_v}")
    host = _host_i32(cu_seqlens_host, n + 1, "cu_seqlens_host")
    with _Launch(k.device, stream) as handle:
        if q is not None and q_out is None:
            q_out = q.new_empty(q.shape)
        elif q is not None and not _in_place(q_out, q):
            _want(q_out, "q_out", dt, q.shape, k)
            if q_out.data_ptr() == q.data_ptr() and not q.is_contiguous():  # (C would take it for q in place)
                raise ValueError("q_out starts where q does, but its tokens lie elsewhere")
        _check(library().kda_paged_append(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(q), ctypes.byref(turn) if turn else None,
                                          _ptr(block_table), _ptr(kv_lens), _ptr(cu_seqlens), _ptr(host), _ptr(k_pages),
                                          _ptr(v_pages), _ptr(q_out), handle))
    return q_out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    kv_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                    window: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    return_lse: bool = False, cu_seqlens_host=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the new tokens q [B, T, Hq, d_k] over their sequences' pages, each token over the cells up to its own
    (the last `window` of them, 0: all).  scale: None for d_k ** -0.5.  block_table may be one row expanded to all sequences
    (it is copied then).  workspace: uint8, as long as
    kda_paged_attn_workspace says (allocated here when None and needed).  Returns out [B, T, Hq, d_v]; with return_lse, or
    an lse to write, (out, lse [B, T, Hq] fp32: the logarithm of the summed weights, -inf for a row without cells)."""
    shape, dt = q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError("q must be [B, T, heads, d]")
    B, T, Hq, dk = shape
    if not 0 <= window < 1 << 31:  # (ctypes would cut it to 32 bits)
        raise ValueError(f"window {window} is not in 0 .. 2^31 - 1")
    lq = 0 if q.is_contiguous() else _rows(q, "q", dt, shape, q.device)
    p, n = _paged(q, B, T, Hq, k_pages, v_pages, block_table, kv_lens, cu_seqlens, lq, 0, 0)
    if p.head_dim_k != dk:
        raise ValueError(f"q has heads of {dk}, the pages keys of {p.head_dim_k}")
    host, lib, want = _host_i32(cu_seqlens_host, n + 1, "cu_seqlens_host"), library(), (B, T, Hq, p.head_dim_v)
    with _Launch(q.device, stream) as handle:
        if _shared(block_table):
            block_table = block_table.contiguous()
        if out is None:
            out = q.new_empty(want)
        else:
            _want(out, "out", dt, want, q)
        if lse is not None:
            _want(lse, "lse", torch.float32, (B, T, Hq), q)
        elif return_lse:
            lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
        if workspace is None:
            need = ctypes.c_size_t(0)
            _check(lib.kda_paged_attn_workspace(ctypes.byref(p), ctypes.byref(need)))
            workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device) if need.value else None
        room, size = _room(workspace, q.device)
        _check(lib.kda_paged_attn(ctypes.byref(p), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(kv_lens),
                                  _ptr(cu_seqlens), _ptr(host), dk ** -0.5 if scale is None else scale, window, _ptr(out), _ptr(lse),
                                  room, size, handle))
    return (out, lse) if lse is not None else out
