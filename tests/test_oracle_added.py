"""Pins of the fp64 oracles of the per-head decay recurrence, the draft-tree
attention and the output norm: closed forms, library functions used once, and
central differences."""
import math

import pytest
import torch

from oracle import decay, gated_norm, tree_attn


def _inputs(B=2, T=9, H=4, Hk=2, dk=5, dv=3, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    return dict(q=r(B, T, Hk, dk), k=r(B, T, Hk, dk), v=r(B, T, H, dv), g=-r(B, T, H).abs() * 0.3,
                h0=r(B, H, dv, dk), dO=r(B, T, H, dv), dhT=r(B, H, dv, dk))


def test_decay_is_the_masked_product():
    x = _inputs()
    o, hT, _ = decay.forward(x["q"], x["k"], x["v"], x["g"], x["h0"], scale=0.7)
    T, rep = 9, 2
    G = x["g"].cumsum(1)
    D = torch.exp(G[:, :, None] - G[:, None]) * torch.ones(T, T).tril()[None, :, :, None]
    A = torch.einsum("bihd,bjhd->bijh", x["q"], x["k"]).repeat_interleave(rep, -1) * D * 0.7
    ref = torch.einsum("bijh,bjhv->bihv", A, x["v"])
    ref += 0.7 * torch.exp(G)[..., None] * torch.einsum("bhvk,bihk->bihv", x["h0"], x["q"].repeat_interleave(rep, 2))
    assert torch.allclose(o, ref, atol=1e-12)
    end = torch.exp(G[:, -1:] - G)[..., None] * x["k"].repeat_interleave(rep, 2)
    assert torch.allclose(hT, torch.einsum("bthv,bthk->bhvk", x["v"], end) +
                          torch.exp(G[:, -1])[..., None, None] * x["h0"], atol=1e-12)


def test_decay_gradients_are_the_differences():
    x = _inputs(B=1, T=5, H=2, Hk=1, dk=3, dv=2, seed=1)
    names = ("q", "k", "v", "g", "h0")
    r = decay.backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dhT"], scale=0.9)

    def loss(y):
        o, hT, _ = decay.forward(y["q"], y["k"], y["v"], y["g"], y["h0"], scale=0.9)
        return float((o * x["dO"]).sum() + (hT * x["dhT"]).sum())

    step = 1e-5
    for n in names:
        got = r["d" + n].reshape(-1)
        for i in range(x[n].numel()):
            up, dn = (dict(x, **{n: x[n].clone()}) for _ in range(2))
            up[n].reshape(-1)[i] += step
            dn[n].reshape(-1)[i] -= step
            assert abs((loss(up) - loss(dn)) / (2 * step) - float(got[i])) < 1e-7, (n, i)


def test_decay_reset_and_packing():
    x = _inputs(B=1, T=8, seed=2)
    x["g"][0, 4] = -math.inf
    o, hT, _ = decay.forward(x["q"], x["k"], x["v"], x["g"], x["h0"])
    o2, h2, _ = decay.forward(*(x[n][:, 4:] for n in ("q", "k", "v", "g")))
    assert torch.allclose(o[:, 4:], o2) and torch.allclose(hT, h2)
    cu = [0, 3, 3, 8]
    h = torch.randn(3, 4, 3, 5, dtype=torch.float64)
    po, ph = decay.packed(decay.forward, cu, x["q"], x["k"], x["v"], x["g"], h)
    assert torch.equal(ph[1], h[1])
    assert torch.equal(po[:, :3], decay.forward(*(x[n][:, :3] for n in ("q", "k", "v", "g")), h[:1])[0])


@pytest.mark.parametrize("window", [0, 1, 4])
def test_tree_chain_is_causal_attention(window):
    """A chain over a cache is causal attention of the sequence cache + nodes."""
    gen = torch.Generator().manual_seed(3)
    L, M, d, page = 7, 5, 4, 2
    kv = torch.randn(2, L + M, 1, d, generator=gen)
    q = torch.randn(1, M, 1, d, generator=gen)
    cache = torch.zeros(2, 4, page, 1, d)
    table = torch.tensor([[2, 0, 3, 1]])
    for p in range(L):
        cache[:, table[0, p // page], p % page] = kv[:, p]
    parent = torch.arange(M)[None] - 1
    o, _ = tree_attn.attend(parent, q, kv[0][None, L:], kv[1][None, L:], cache[0], cache[1], table,
                            torch.tensor([L]), 0.5, window)
    i, j = torch.arange(M)[:, None] + L, torch.arange(L + M)[None]
    seen = (j <= i) & ((i - j < window) if window else True)
    s = (0.5 * q[0, :, 0].double() @ kv[0, :, 0].double().T).masked_fill(~seen, -math.inf)
    assert torch.allclose(o[0, :, 0], torch.softmax(s, -1) @ kv[1, :, 0].double(), atol=1e-12)
    kc, vc, new = tree_attn.append(parent, torch.tensor([0]), kv[0][None, L:], kv[1][None, L:], cache[0], cache[1],
                                   table, torch.tensor([L]))
    assert int(new[0]) == L + 1 and torch.equal(kc[1, 1], kv[0, L]) and torch.equal(vc[1, 1], kv[1, L])


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_against_library_and_differences(center, shared):
    gen = torch.Generator().manual_seed(4)
    x, z, dy = (torch.randn(3, 2, 6, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.randn(6, generator=gen, dtype=torch.float64) if shared else torch.randn(2, 6, generator=gen, dtype=torch.float64)
    y = gated_norm.forward(x, z, w, 1e-3, center)
    F = torch.nn.functional
    n = F.layer_norm(x, (6,), eps=1e-3) if center else F.rms_norm(x, (6,), eps=1e-3)
    assert torch.allclose(y, n * w * F.silu(z), atol=1e-12)
    got = gated_norm.backward(x, z, w, dy, 1e-3, center)[:3]
    step = 1e-5
    for t, g in zip((x, z, w), got):
        for i in range(t.numel()):
            old = float(t.reshape(-1)[i])
            vals = []
            for s in (step, -step):
                t.reshape(-1)[i] = old + s
                vals.append(float((gated_norm.forward(x, z, w, 1e-3, center) * dy).sum()))
            t.reshape(-1)[i] = old
            assert abs((vals[0] - vals[1]) / (2 * step) - float(g.reshape(-1)[i])) < 1e-7
