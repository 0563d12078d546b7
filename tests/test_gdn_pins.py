"""The reference of the scalar-gate delta rule's GPU tests against the C oracle (the per-channel rule with the
gate the same in every channel) and its gradients against the oracle's and against differences."""
import numpy as np
import pytest
import torch

import gdn_reference as ref
import oracle


def _np(x):
    return x.float().numpy()


@pytest.mark.parametrize("lens", [None, [0, 5, 1, 0, 9]])
def test_reference_matches_the_oracle(lens):
    B, T = (2, 7) if lens is None else (1, sum(lens))
    q, k, v, g, b = ref.inputs(B, T, 2, 4, 8, 6, io=torch.float32, seed=1)
    cu = None if lens is None else ref.packed(lens)
    n = B if lens is None else len(lens)
    s0, dsf, do = (torch.randn(*s) for s in ((n, 4, 8, 6), (n, 4, 8, 6), (B, T, 4, 6)))
    wide = lambda x: _np(x.repeat_interleave(2, 2))  # noqa: E731
    gw = _np(g[..., None].expand(*g.shape, 8).contiguous())
    cun = None if cu is None else cu.numpy()
    o, f = oracle.fwd(wide(q), wide(k), _np(v), gw, _np(b), initial_state=_np(s0), cu_seqlens=cun, scale=0.7)
    out, fin = ref.delta_rule(q, k, v, g, b, s0, cu, 0.7)
    assert np.abs(out.numpy() - o).max() < 1e-12 and np.abs(fin.numpy() - f).max() < 1e-12
    want = oracle.bwd(wide(q), wide(k), _np(v), gw, _np(b), _np(do), initial_state=_np(s0), d_final_state=_np(dsf),
                      cu_seqlens=cun, scale=0.7)
    got = ref.delta_rule_grads(q, k, v, g, b, do, s0, dsf, cu, 0.7)
    group = lambda x: x.reshape(B, T, 2, 2, 8).sum(3)  # noqa: E731
    for key, w in (("dq", group(want["dq"])), ("dk", group(want["dk"])), ("dv", want["dv"]),
                   ("dg", want["dg"].sum(-1)), ("dbeta", want["dbeta"]), ("d_initial_state", want["d_initial_state"])):
        assert np.abs(got[key].numpy() - w).max() < 1e-11, key


def test_reference_gradients_match_differences():
    q, k, v, g, b = [x.double() for x in ref.inputs(1, 6, 1, 2, 4, 3, io=torch.float32, seed=2)]
    s0, dsf, do = (torch.randn(*s, dtype=torch.float64) for s in ((1, 2, 4, 3), (1, 2, 4, 3), (1, 6, 2, 3)))
    x = dict(dq=q, dk=k, dv=v, dg=g, dbeta=b, d_initial_state=s0)
    grads = ref.delta_rule_grads(q, k, v, g, b, do, s0, dsf)

    def loss(x):
        o, f = ref.delta_rule(x["dq"], x["dk"], x["dv"], x["dg"], x["dbeta"], x["d_initial_state"])
        return float((do * o).sum() + (dsf * f).sum())

    for key in x:
        d = torch.randn_like(x[key])
        h = 1e-5
        num = (loss({**x, key: x[key] + h * d}) - loss({**x, key: x[key] - h * d})) / (2 * h)
        assert abs(num - float((grads[key] * d).sum())) < 1e-7 * max(1.0, abs(num)), key


def test_a_planted_mistake_is_caught():
    """Undecayed correction (the residual against S before the gate) differs from the reference."""
    q, k, v, g, b = [x.double() for x in ref.inputs(1, 5, 1, 1, 4, 3, io=torch.float32, seed=3)]
    S, outs = torch.zeros(4, 3, dtype=torch.float64), []
    for t in range(5):
        res = v[0, t, 0] - k[0, t, 0] @ S
        S = g[0, t, 0].exp() * S + torch.outer(k[0, t, 0], b[0, t, 0] * res)
        outs.append(q[0, t, 0] @ S)
    out, _ = ref.delta_rule(q, k, v, g, b)
    assert (out[0, :, 0] - torch.stack(outs)).abs().max() > 1e-3
