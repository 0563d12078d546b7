"""Plain token-by-token reference of the scalar-gate delta rule and of the output epilogue, in fp64
torch (differentiable; shares no code with the library):

    S_t = (I - beta_t k_t k_t^T) e^{g_t} S_{t-1} + beta_t k_t v_t^T,     o_t = scale S_t^T q_t
"""
import torch


def lens_of(cu, B, T):
    return [T] * B if cu is None else [int(b - a) for a, b in zip(cu[:-1], cu[1:])]


def delta_rule(q, k, v, g, beta, s0=None, cu=None, scale=1.0):
    """q, k [B, T, Hk, dk], v [B, T, Hv, dv], g, beta [B, T, Hv], s0 [N, Hv, dk, dv], any dtype.
    Returns (out, final) in fp64."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    rep = Hv // Hk
    q, k, v, g, beta = (x.double().flatten(0, 1) for x in (q, k, v, g, beta))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    lens = lens_of(cu, B, T)
    N, L = len(lens), max(lens, default=0)
    S = q.new_zeros(N, Hv, dk, dv) if s0 is None else s0.double()
    start = torch.tensor([0] + lens).cumsum(0)[:-1].to(q.device)
    if cu is not None and len(cu):
        start = cu[:-1].long().to(q.device)
    n = torch.tensor(lens, device=q.device)
    outs, where = [], []
    for t in range(L):
        live = n > t
        at = (start + t)[live]
        a = g[at].exp()[..., None, None]
        Sl = S[live] * a
        res = v[at] - torch.einsum("nhk,nhkv->nhv", k[at], Sl)
        Sl = Sl + torch.einsum("nhk,nhv->nhkv", k[at], beta[at][..., None] * res)
        outs.append(scale * torch.einsum("nhk,nhkv->nhv", q[at], Sl))
        where.append(at)
        S = S.clone()
        S[live] = Sl
    out = q.new_zeros(B * T, Hv, dv)
    if outs:
        out = out.index_copy(0, torch.cat(where), torch.cat(outs))
    return out.view(B, T, Hv, dv), S


def delta_rule_grads(q, k, v, g, beta, d_out, s0=None, d_final=None, cu=None, scale=1.0):
    """Gradients of sum(d_out * out) + sum(d_final * final), by autograd, in fp64."""
    x = [t.double().detach().requires_grad_() for t in (q, k, v, g, beta)]
    n = len(lens_of(cu, q.shape[0], q.shape[1]))
    s = torch.zeros(n, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64, device=q.device) if s0 is None else s0.double().detach()
    s.requires_grad_()
    out, fin = delta_rule(*x, s, cu, scale)
    loss = (d_out.double() * out).sum() + (0 if d_final is None else (d_final.double() * fin).sum())
    grads = torch.autograd.grad(loss, x + [s], allow_unused=True)
    return {n: torch.zeros_like(t) if d is None else d
            for n, t, d in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial_state"), x + [s], grads)}


def norm_gate(o, z, w, eps=1e-6):
    o, z, w = o.double(), z.double(), w.double()
    return o / ((o * o).mean(-1, keepdim=True) + eps).sqrt() * w * torch.sigmoid(z)


def inputs(B, T, Hk, Hv, dk, dv, io=torch.bfloat16, gates=None, mu=-2.0, seed=0, device="cpu"):
    """q, k of unit norm, v normal, g = -softplus(normal + mu), beta = sigmoid(normal)."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    gates = gates or io
    q, k, v = unit(rnd(B, T, Hk, dk)), unit(rnd(B, T, Hk, dk)), rnd(B, T, Hv, dv)
    g, beta = -torch.nn.functional.softplus(rnd(B, T, Hv) + mu), torch.sigmoid(rnd(B, T, Hv))
    return [x.to(t).to(device) for x, t in ((q, io), (k, io), (v, io), (g, gates), (beta, gates))]


def packed(lens, device="cpu"):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(device)
