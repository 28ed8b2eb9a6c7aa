"""The states that gdn_decay_* returns are fp32 sums of products that are exact to fp32, with
bf16 inputs too.  Few tokens are not zero, so that the sums are short and the bound is
tight enough to tell: with v (or dO) decayed and then taken as two bf16 terms, and not
three, the errors are beyond it.

Bound, in units of 2^-24 relative to the terms' absolute sum.  The decay of a pair of tokens:
4 for the exponential (2^-22), D = |log2 of it| for the difference that goes in, 2 for the
products that scale it.  Its product with v: 1; the three terms: 1/8.  Sums of up to 3
tokens in the tensor core, which may drop up to a step per product: 6, and 3 for the sums
with the state, whose own decay takes 6 + D.  24 + D covers either."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

U = 2.0 ** -24
DIMS = [(64, 64), (128, 64), (64, 128), (128, 128)]


def exact(k, v, g, h0, tokens, scale=1.0, back=False):
    """Sum over `tokens` of decay v k^T + decay h0, its absolute terms, and the largest D."""
    k, v, g, h0 = (t.double() for t in (k, v, g, h0))
    G = g.cumsum(0)                                     # [T, H]
    w = G[tokens] if back else G[-1] - G[tokens]        # [n, H]
    e = scale * torch.exp(w)
    end = torch.exp(G[-1])[:, None, None]
    ref = torch.einsum("nh,nhv,nhk->hvk", e, v[tokens], k[tokens]) + end * h0
    mag = torch.einsum("nh,nhv,nhk->hvk", e.abs(), v[tokens].abs(), k[tokens].abs()) + end * h0.abs()
    return ref, mag, float(w.abs().max().maximum(G[-1].abs().max())) * 1.4427


def make(T, H, dk, dv, tokens, seed, gates):
    gen = torch.Generator().manual_seed(seed)
    x = dict(k=torch.zeros(T, H, dk), v=torch.zeros(T, H, dv), g=torch.zeros(T, H))
    for n in ("k", "v"):
        x[n][tokens] = torch.randn(len(tokens), H, x[n].shape[2], generator=gen)
        x[n] = x[n].bfloat16()
    for t in gates:
        x["g"][t] = -torch.rand(H, generator=gen) - 0.05
    return x


def close(got, ref, mag, D):
    return bool(((got.double().cpu() - ref).abs() <= (24 + D) * U * mag).all())


CASES = [(3, [0, 1, 2], [0, 1, 2]), (130, [1, 77, 129], [0, 40, 100, 129]), (3000, [10], [20]), (3000, [1400], [1403]),
         (3000, [2990], [2991, 2995])]


@pytest.mark.parametrize("dk,dv", DIMS)
def test_two_terms_are_not_enough(dk, dv):
    """The same sums with the decayed v as two bf16 terms are beyond the bound."""
    T, tokens, gates = CASES[0]
    x = make(T, 4, dk, dv, tokens, 111, gates)
    ref, mag, D = exact(x["k"], x["v"], x["g"], torch.zeros(4, dv, dk), tokens)
    G = x["g"].double().cumsum(0)
    y = torch.exp(G[-1] - G)[..., None] * x["v"].double()
    for terms, fine in ((3, True), (2, False)):
        rest, total = y.clone(), torch.zeros_like(y)
        for _ in range(terms):
            t = rest.bfloat16().double()
            total += t
            rest -= t
        assert close(torch.einsum("nhv,nhk->hvk", total, x["k"].double()), ref, mag, D) == fine


@pytest.mark.gpu
@pytest.mark.parametrize("T,tokens,gates", CASES)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_last_state_and_gradient_of_the_first(dev, dk, dv, T, tokens, gates):
    H = 8 if T < 1000 else 1  # one head's chain is cut into runs
    x = make(T, H, dk, dv, tokens, 112 + T, gates)
    gen = torch.Generator().manual_seed(5)
    h0 = torch.randn(H, dv, dk, generator=gen) if T < 1000 else torch.zeros(H, dv, dk)
    d = {n: t[None].to(dev) for n, t in x.items()}
    h = h0[None].to(dev)
    zero = torch.zeros_like(d["k"])
    _, hT = gdn.gdn_decay_fwd(zero, d["k"], d["v"], d["g"], h)
    ref, mag, D = exact(x["k"], x["v"], x["g"], h0, tokens)
    assert close(hT[0], ref, mag, D)
    # the gradient's state takes q and dO in their place, decayed from the start
    r = gdn.gdn_decay_bwd(d["k"], zero, torch.zeros_like(d["v"]), d["g"], d["v"], h, h, scale=0.3)
    ref, mag, D = exact(x["k"], x["v"], x["g"], h0, tokens, float(torch.tensor(0.3)), back=True)
    assert close(r["dh0"][0], ref, mag, D)
