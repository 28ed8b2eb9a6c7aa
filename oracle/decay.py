"""Linear attention with a decay per head, written out token by token in fp64:
S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t (scale q_t), and its reverse mode.

Shapes: q, k [B,T,Hk,dk]; v, dO [B,T,H,dv]; g [B,T,H]; states [B,H,dv,dk].
Value head h reads key head h // (H // Hk)."""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else x.detach().double().cpu()


def forward(q, k, v, g, h0=None, scale=1.0):
    """(o, hT, the states after every token)."""
    q, k, v, g, h0 = map(_f64, (q, k, v, g, h0))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    head = torch.arange(H) // (H // Hk)
    S = torch.zeros(B, H, dv, dk, dtype=torch.float64) if h0 is None else h0.clone()
    o, states = torch.zeros(B, T, H, dv, dtype=torch.float64), []
    for t in range(T):
        S = S * torch.exp(g[:, t])[..., None, None] + v[:, t, :, :, None] * k[:, t, head, None, :]
        o[:, t] = scale * (S * q[:, t, head, None, :]).sum(-1)
        states.append(S)
    return o, S, states


def backward(q, k, v, g, dO, h0=None, dhT=None, scale=1.0):
    """Gradients of <dO, o> + <dhT, hT>: dict with dq, dk, dv, dg, dh0."""
    _, _, states = forward(q, k, v, g, h0, scale)
    q, k, v, g, h0, dO, dhT = map(_f64, (q, k, v, g, h0, dO, dhT))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    head = torch.arange(H) // (H // Hk)
    zero = torch.zeros(B, H, dv, dk, dtype=torch.float64)
    dS = zero.clone() if dhT is None else dhT.clone()
    r = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dg=torch.zeros_like(g))
    for t in reversed(range(T)):
        r["dq"][:, t].index_add_(1, head, scale * (states[t] * dO[:, t, :, :, None]).sum(-2))
        dS = dS + scale * dO[:, t, :, :, None] * q[:, t, head, None, :]
        r["dv"][:, t] = (dS * k[:, t, head, None, :]).sum(-1)
        r["dk"][:, t].index_add_(1, head, (dS * v[:, t, :, :, None]).sum(-2))
        before = states[t - 1] if t else (zero if h0 is None else h0)
        a = torch.exp(g[:, t])
        r["dg"][:, t] = a * (dS * before).sum((-1, -2))
        dS = dS * a[..., None, None]
    r["dh0"] = dS
    return r


def packed(fn, cu, q, k, v, g, *rest, scale=1.0):
    """fn (forward or backward) on each sequence of a packed row; token rows of no
    sequence are zero.  rest: dO (backward only), then the state arguments."""
    grad = fn is backward
    dO = rest[0] if grad else None
    h0, more = (rest[1], rest[2]) if grad else (rest[0], None)
    one = lambda x, s: None if x is None else x[s:s + 1]  # noqa: E731
    parts, outs = [], None
    for s in range(len(cu) - 1):
        w = slice(cu[s], cu[s + 1])
        args = (q[:, w], k[:, w], v[:, w], g[:, w])
        if grad:
            parts.append((w, fn(*args, dO[:, w], one(h0, s), one(more, s), scale=scale)))
        else:
            parts.append((w, fn(*args, one(h0, s), scale=scale)))
    if grad:
        outs = {n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
        for w, r in parts:
            for n in outs:
                outs[n][:, w] = r[n]
        outs["dh0"] = torch.cat([r["dh0"] for _, r in parts])
        return outs
    o = torch.zeros(v.shape, dtype=torch.float64)
    for w, r in parts:
        o[:, w] = r[0]
    return o, torch.cat([r[1] for _, r in parts])
