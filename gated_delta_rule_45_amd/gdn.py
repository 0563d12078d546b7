"""Scalar-gate delta rule (one log-gate per token and value head, grouped heads) and the gradients of the
output epilogue: argument checks and marshalling for the kda_gdn_* and kda_norm_gate_bwd entry points
of libkda.so.

    S_t = (I - beta_t k_t k_t^T) exp(g_t) S_{t-1} + beta_t k_t v_t^T,     o_t = scale * S_t^T q_t

q, k have Hk heads, v, g, beta, out and the states Hv (a multiple of Hk); value head h reads key head
h // (Hv // Hk).  q, k and v may be slices of one projection's output: the heads of a token dense, the
tokens a constant multiple of 16 bytes apart.  g and beta are both fp32 or both bf16, states fp32 or bf16.

Rows that no sequence of cu_seqlens owns (a padded packed batch) and the rows of padded slots are not written: in
tensors allocated here they hold whatever the memory held.  Where they are read later (a weight's gradient
sums over all rows of dq, dk and dv), pass `out` with what they are to hold, zeros for instance.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _P, _check, _io_code, _need, library

__all__ = ["gdn_chunk_fwd", "gdn_chunk_bwd", "gdn_decode", "norm_gate_bwd"]


class GdnProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "seq_len", "num_seqs", "num_heads_k", "num_heads_v", "head_dim_k",
                                              "head_dim_v", "io_dtype", "gate_dtype", "state_dtype")] + \
        [("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("stride_q", "stride_k", "stride_v")]


def declare(lib: ctypes.CDLL) -> None:
    prob = ctypes.POINTER(GdnProblem)
    lib.kda_gdn_chunk_fwd.argtypes = [prob] + [_P] * 11 + [ctypes.c_size_t, _P]
    lib.kda_gdn_chunk_fwd_workspace.argtypes = [prob, ctypes.POINTER(ctypes.c_size_t)]
    lib.kda_gdn_decode.argtypes = [prob] + [_P] * 6 + [ctypes.c_int64] + [_P] * 6
    lib.kda_norm_gate_bwd.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_float] + [_P] * 8 + \
        [ctypes.c_size_t, _P]
    lib.kda_norm_gate_bwd_workspace.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
    lib.kda_norm_gate_bwd_workspace.restype = ctypes.c_size_t
    lib.kda_gdn_chunk_bwd.argtypes = [prob] + [_P] * 17 + [ctypes.c_size_t, _P]
    lib.kda_gdn_chunk_bwd_workspace.argtypes = [prob, ctypes.POINTER(ctypes.c_size_t)]
    for f in (lib.kda_gdn_chunk_bwd, lib.kda_gdn_chunk_bwd_workspace, lib.kda_gdn_chunk_fwd, lib.kda_gdn_chunk_fwd_workspace,
              lib.kda_gdn_decode, lib.kda_norm_gate_bwd):
        f.restype = ctypes.c_int


def _current_handle(index: int) -> int:
    """The current stream's handle on a device: alone, where this torch has a function for that, since a Stream object around
    it costs 1.7 us, a good part of a small call."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


class _Launch:
    """The device and the stream of a call: what is allocated inside belongs to that stream, and the
    launch happens with that device current."""

    def __init__(self, device: torch.device, stream):
        if device.type != "cuda":
            raise ValueError(f"tensors must be on a GPU, got {device}")
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, expected {device}")
        self.other = None
        if stream is None:
            self.handle = _current_handle(device.index)
        else:
            self.handle = stream.cuda_stream
            if stream != torch.cuda.current_stream(device):
                self.other = torch.cuda.stream(stream)
                return
        if device.index != torch.cuda.current_device():
            self.other = torch.cuda.device(device)

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dense(t, dtype, shape, like: torch.Tensor) -> bool:
    """The checks of a call in one go (a few us of host time are most of a small call); what fails here is
    named by the slower ones."""
    return (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == like.get_device()
            and t.is_contiguous())


def _want(t, name: str, dtype, shape, like: torch.Tensor) -> None:
    if not _dense(t, dtype, shape, like):
        _need(t, name, dtype, shape, like.device)


def _rows(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Check one of q, k, v ([B, T, H, d]) and return the elements between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    B, T, H, d = shape
    if t.is_contiguous():
        return H * d
    sb, st, sh, sd = t.stride()
    ld = st if T > 1 else sb if B > 1 else H * d
    if sd != 1 or (H > 1 and sh != d) or (B > 1 and T > 1 and sb != T * st) or ld < H * d:
        raise ValueError(f"{name}: the heads of a token must be dense and the tokens evenly spaced (strides {t.stride()})")
    return ld


def _room(workspace, device):
    """A workspace's pointer and bytes."""
    if workspace is None or workspace.numel() == 0:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def _host_i32(x, n: int, name: str):
    if x is None:
        return None
    h = torch.as_tensor(x, dtype=torch.int32).contiguous().cpu()
    if h.numel() != n:
        raise ValueError(f"{name} has the wrong length")
    return h


def _problem(q, k, v, g, beta, cu_seqlens, state_dtype, scale):
    """Checks of the inputs that every call shares."""
    qs, vs, gate = q.shape, v.shape, g.dtype
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError("q, k and v must be [B, T, heads, d]")
    B, T, Hk, dk = qs
    Hv, dv = vs[2], vs[3]
    dt = q.dtype
    io = _io_code(dt)
    # 0: dense
    lq = 0 if q.is_contiguous() else _rows(q, "q", dt, qs, q.device)
    lk = 0 if _dense(k, dt, qs, q) else _rows(k, "k", dt, qs, q.device)
    lv = 0 if _dense(v, dt, (B, T, Hv, dv), q) else _rows(v, "v", dt, (B, T, Hv, dv), q.device)
    _want(g, "g", gate, (B, T, Hv), q)
    _want(beta, "beta", gate, (B, T, Hv), q)
    n = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("a packed batch (cu_seqlens) needs B == 1")
        n = cu_seqlens.numel() - 1
        if n < 0:
            raise ValueError("cu_seqlens needs at least one entry")
        _want(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), q)
    p = GdnProblem(B, T, n if cu_seqlens is not None else 0, Hk, Hv, dk, dv, io, _io_code(gate),
                   _io_code(state_dtype), scale, lq, lk, lv)
    return p, n


def gdn_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                  cu_seqlens_host=None, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  state_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Chunkwise forward.  q, k: [B, T, Hk, d_k]; v: [B, T, Hv, d_v] (bf16 or fp32); g, beta: [B, T, Hv]
    (fp32 or bf16); initial_state: [N, Hv, d_k, d_v] (fp32 or bf16) or None; cu_seqlens: int32 [N+1]
    (B == 1) or None.  The states' dtype is that of the state given, else state_dtype, else fp32;
    final_state may be initial_state.  workspace: uint8, as long as kda_gdn_chunk_fwd_workspace says, for long
    sequences on few heads (allocated here when None and needed; an empty tensor: do without), of which a packed
    batch makes no use.  Returns (out, final_state)."""
    given = initial_state if initial_state is not None else final_state
    sdt = given.dtype if given is not None else state_dtype or torch.float32
    p, n = _problem(q, k, v, g, beta, cu_seqlens, sdt, scale)
    dev, shape, states = q.device, v.shape, (n, v.shape[2], q.shape[3], v.shape[3])
    if initial_state is not None:
        _want(initial_state, "initial_state", sdt, states, q)
    host = _host_i32(cu_seqlens_host, n + 1, "cu_seqlens_host")
    with _Launch(dev, stream) as handle:
        if out is None:
            out = q.new_empty(shape)
        else:
            _want(out, "out", q.dtype, shape, q)
        if final_state is not None:
            _want(final_state, "final_state", sdt, states, q)
        elif output_final_state:
            final_state = torch.empty(states, dtype=sdt, device=dev)
        if workspace is None and cu_seqlens is None and q.shape[1] >= _SPLIT_TOKENS:
            need = _fwd_workspace(p)
            workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        room, size = _room(workspace, dev)
        _check(library().kda_gdn_chunk_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                           _ptr(initial_state), _ptr(cu_seqlens), _ptr(host), _ptr(out),
                                           _ptr(final_state), room, size, handle))
    return out, final_state


_SPLIT_TOKENS = 225  # the library splits no shorter sequence: a small call is spared the question


def _fwd_workspace(p: GdnProblem) -> int:
    n = ctypes.c_size_t(0)
    _check(library().kda_gdn_chunk_fwd_workspace(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def gdn_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  d_out: torch.Tensor, initial_state: Optional[torch.Tensor] = None,
                  d_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                  cu_seqlens_host=None, scale: float = 1.0, need_d_initial_state: bool = True,
                  workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """Gradients of gdn_chunk_fwd for L = sum(d_out * out) + sum(d_final_state * final_state).  d_out: out's
    shape and dtype; d_final_state: as the states, or None (zero).  Returns dict(dq, dk [B, T, Hk, d_k],
    dv [B, T, Hv, d_v] (io dtype), dg, dbeta [B, T, Hv] (g's dtype), d_initial_state [N, Hv, d_k, d_v]
    (the states' dtype, fp32 where no state is given, or None)), all dense; `out` (a dict returned by an
    earlier call of the same shape) is written in place."""
    given = initial_state if initial_state is not None else d_final_state
    sdt = given.dtype if given is not None else torch.float32
    p, n = _problem(q, k, v, g, beta, cu_seqlens, sdt, scale)
    dev, states = q.device, (n, v.shape[2], q.shape[3], v.shape[3])
    _want(d_out, "d_out", q.dtype, v.shape, q)
    if initial_state is not None:
        _want(initial_state, "initial_state", sdt, states, q)
    if d_final_state is not None:
        _want(d_final_state, "d_final_state", sdt, states, q)
    host = _host_i32(cu_seqlens_host, n + 1, "cu_seqlens_host")
    lib = library()
    want = {"dq": (q.shape, q.dtype), "dk": (q.shape, q.dtype), "dv": (v.shape, q.dtype), "dg": (g.shape, g.dtype),
            "dbeta": (g.shape, g.dtype), "d_initial_state": (states, sdt)}
    with _Launch(dev, stream) as handle:
        if out is None:
            out = {name: torch.empty(s, dtype=t, device=dev) if name != "d_initial_state" or need_d_initial_state else None
                   for name, (s, t) in want.items()}
        else:
            for name, (s, t) in want.items():
                if name != "d_initial_state" or out.get(name) is not None:
                    _want(out[name], name, t, s, q)
        if workspace is None:
            need = ctypes.c_size_t(0)
            _check(lib.kda_gdn_chunk_bwd_workspace(ctypes.byref(p), ctypes.byref(need)))
            workspace = torch.empty(need.value, dtype=torch.uint8, device=dev)
        room, size = _room(workspace, dev)
        _check(lib.kda_gdn_chunk_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                     _ptr(cu_seqlens), _ptr(host), _ptr(d_out), _ptr(d_final_state), _ptr(out["dq"]),
                                     _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
                                     _ptr(out.get("d_initial_state")), room, size, handle))
    return out


def gdn_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
               state: torch.Tensor, state_slots: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, *, state_slots_host=None, cu_seqlens_host=None,
               scale: float = 1.0, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One or a few new tokens per sequence.  q, k: [N, T, Hk, d_k]; v: [N, T, Hv, d_v]; g, beta: [N, T, Hv]
    (with cu_seqlens: [1, tokens, ...], ragged); state: [slots, Hv, d_k, d_v] fp32 or bf16, updated in
    place; state_slots: int32 [N], the slot of each sequence (None: sequence n has slot n), each at
    most once; a slot outside the pool marks a padded row, whose outputs are not written.  Returns out."""
    p, n = _problem(q, k, v, g, beta, cu_seqlens, state.dtype, scale)
    dev, shape = q.device, v.shape
    _want(state, "state", state.dtype, (state.shape[0], shape[2], q.shape[3], shape[3]), q)
    if state_slots is not None:
        _want(state_slots, "state_slots", torch.int32, (n,), q)
    host = _host_i32(cu_seqlens_host, n + 1, "cu_seqlens_host")
    slots_host = _host_i32(state_slots_host, n, "state_slots_host")
    with _Launch(dev, stream) as handle:
        if out is None:
            out = q.new_empty(shape)
        else:
            _want(out, "out", q.dtype, shape, q)
        _check(library().kda_gdn_decode(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                        state.shape[0], _ptr(state_slots), _ptr(slots_host), _ptr(cu_seqlens),
                                        _ptr(host), _ptr(out), handle))
    return out


def norm_gate_bwd(o: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, d_out: torch.Tensor, *, eps: float = 1e-6,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of norm_gate (o: its input) for L = sum(d_out * out).  o, gate, d_out: same shape and dtype
    (bf16 or fp32), contiguous; weight: fp32 [d].  Returns (d_o, d_gate, d_weight)."""
    dev, d, shape = o.device, o.shape[-1], o.shape
    _want(o, "o", o.dtype, shape, o)
    _want(gate, "gate", o.dtype, shape, o)
    _want(d_out, "d_out", o.dtype, shape, o)
    _want(weight, "weight", torch.float32, (d,), o)
    rows, io, lib = o.numel() // d if d else 0, _io_code(o.dtype), library()
    need = lib.kda_norm_gate_bwd_workspace(rows, d, io)
    with _Launch(dev, stream) as handle:
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        room, size = _room(workspace, dev)
        d_o, d_gate, d_weight = torch.empty_like(o), torch.empty_like(o), torch.empty_like(weight)
        _check(lib.kda_norm_gate_bwd(rows, d, io, eps, _ptr(o), _ptr(gate), _ptr(weight), _ptr(d_out), _ptr(d_o),
                                     _ptr(d_gate), _ptr(d_weight), room, size, handle))
    return d_o, d_gate, d_weight
