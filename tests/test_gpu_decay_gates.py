"""The gate's gradient of gdn_decay_bwd to fp32, with bf16 inputs: what one token leaves in
the state and another takes from it, chunks apart, so that it passes through the states
that the backward keeps.

One key channel and one value channel per head, so that nearly nothing is summed and the
bound is tight enough to tell: states taken as two bf16 terms, and not three, are beyond it.
In units of 2^-24 of the value: 4 for each of four exponentials and D = |log2 of the decay| in
all for what goes into them, 2 for the products that scale each, 6 for the sums of the
terms in the tensor core, and 2 for the products with q and dO: 32 + D."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

U = 2.0 ** -24
DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]
H, T = 32, 400
SCALE = float(torch.tensor(0.3))


def make(dk, dv, seed, j, i):
    """Token j's k and v, token i's q and dO, a gate in each chunk, and the channels."""
    gen = torch.Generator().manual_seed(seed)
    x = dict(q=torch.zeros(T, H, dk), k=torch.zeros(T, H, dk), v=torch.zeros(T, H, dv), dO=torch.zeros(T, H, dv),
             g=torch.zeros(T, H))
    c, e = torch.randint(0, dk, (H,), generator=gen), torch.randint(0, dv, (H,), generator=gen)
    for n, t, at in (("q", i, c), ("k", j, c), ("v", j, e), ("dO", i, e)):
        x[n][t, torch.arange(H), at] = torch.randn(H, generator=gen).abs() + 0.1
        x[n] = x[n].bfloat16()
    for t in (20, 60, 200, 270, 390):
        x["g"][t] = -torch.rand(H, generator=gen) - 0.05
    return x, c, e


def values(x, j, i):
    """dg of the tokens from j + 1 to i, per head, what the state held, and D."""
    G = x["g"].double().cumsum(0)
    held = torch.exp(G[i] - G[j]) * x["v"][j].double().sum(-1)
    return SCALE * held * x["k"][j].double().sum(-1) * x["q"][i].double().sum(-1) * x["dO"][i].double().sum(-1), held, \
        float((G[j] - G[i]).max()) * 1.4427


def test_two_terms_are_not_enough():
    x, _, _ = make(64, 64, 121, 37, 300)
    ref, held, D = values(x, 37, 300)
    for terms, fine in ((3, True), (2, False)):
        rest, total = held.clone(), torch.zeros_like(held)
        for _ in range(terms):
            t = rest.bfloat16().double()
            total += t
            rest -= t
        assert bool(((ref / held * total - ref).abs() <= (32 + D) * U * ref.abs()).all()) == fine


@pytest.mark.gpu
@pytest.mark.parametrize("j,i", [(37, 300), (130, 300), (0, 256), (127, 128)])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_between_two_tokens(dev, dk, dv, j, i):
    """j's own chunk, the chunks between, i's own chunk; zero outside."""
    x, _, _ = make(dk, dv, 121 + j, j, i)
    d = {n: t[None].to(dev) for n, t in x.items()}
    r = gdn.gdn_decay_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], scale=SCALE)
    ref, _, D = values(x, j, i)
    dg = r["dg"][0].double().cpu()
    assert bool(((dg[j + 1:i + 1] - ref).abs() <= (32 + D) * U * ref.abs()).all())
    assert not bool(dg[:j + 1].any()) and not bool(dg[i + 1:].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", DIMS)
def test_from_the_first_state_and_to_the_last(dev, dk, dv):
    """h0 takes j's part, and in turn dhT takes i's."""
    x, c, e = make(dk, dv, 131, 0, 300)
    gen = torch.Generator().manual_seed(7)
    G = x["g"].double().cumsum(0)
    heads, h = torch.arange(H), torch.randn(H, generator=gen).abs() + 0.1
    state = torch.zeros(1, H, dv, dk)
    state[0, heads, e, c] = h
    zero = {n: torch.zeros_like(t[None]).to(dev) for n, t in x.items()}
    d = {n: t[None].to(dev) for n, t in x.items()}
    s, none = state.to(dev), torch.zeros_like(state).to(dev)
    r = gdn.gdn_decay_bwd(d["q"], zero["k"], zero["v"], d["g"], d["dO"], s, none, scale=SCALE)
    ref = SCALE * torch.exp(G[300]) * h * x["q"][300].double().sum(-1) * x["dO"][300].double().sum(-1)
    dg, D = r["dg"][0].double().cpu(), float(-G[-1].min()) * 1.4427
    assert bool(((dg[:301] - ref).abs() <= (32 + D) * U * ref.abs()).all()) and not bool(dg[301:].any())
    r = gdn.gdn_decay_bwd(zero["q"], d["k"], d["v"], d["g"], zero["dO"], none, s, scale=SCALE)
    ref = torch.exp(G[-1] - G[0]) * h * x["k"][0].double().sum(-1) * x["v"][0].double().sum(-1)
    dg = r["dg"][0].double().cpu()
    assert bool(((dg[1:] - ref).abs() <= (32 + D) * U * ref.abs()).all()) and not bool(dg[:1].any())
    r = gdn.gdn_decay_bwd(zero["q"], zero["k"], zero["v"], d["g"], zero["dO"], s, s, scale=SCALE)
    ref = torch.exp(G[-1]) * h * h
    dg = r["dg"][0].double().cpu()
    assert bool(((dg - ref).abs() <= (32 + D) * U * ref.abs()).all())
