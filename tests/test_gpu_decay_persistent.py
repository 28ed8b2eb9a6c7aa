"""gdn_decay_* on tensor cores with more chunks than CTAs, so that every CTA of the backward
goes through several, and batches cut into runs: against the definition as masked products
of whole sequences in fp64 (the token loop of the oracle would hold a state per token),
gradients by automatic differentiation.  The bounds are those of test_gpu_decay.py."""
import math

import pytest
import torch

import gated_delta_rule_153_b200 as gdn
from oracle import decay

from . import test_gpu_decay as base

NAMES = ("q", "k", "v", "g", "h0")


def whole(x, scale, cu=None):
    """Outputs and gradients of <dO, o> + <dhT, hT>, by name, sequence by sequence in fp64."""
    leaf = {n: x[n].detach().double().requires_grad_(True) for n in NAMES}
    B, T, Hk, _ = x["q"].shape
    rep = x["v"].shape[2] // Hk
    spans = [(b, 0, T) for b in range(B)] if cu is None else [(0, a, b) for a, b in zip(cu, cu[1:])]
    o, hT = torch.zeros_like(leaf["v"]), []
    rows = []
    for i, (b, lo, hi) in enumerate(spans):
        q, k = (leaf[n][b, lo:hi].repeat_interleave(rep, 1).transpose(0, 1) for n in ("q", "k"))  # [H, T, dk]
        v, G = leaf["v"][b, lo:hi].transpose(0, 1), leaf["g"][b, lo:hi].cumsum(0).T
        S = leaf["h0"][i]
        keep = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device=q.device).tril()
        D = (G[:, :, None] - G[:, None]).masked_fill(~keep, -math.inf).exp()
        y = scale * (((q @ k.transpose(1, 2)) * D) @ v + G.exp()[..., None] * (q @ S.transpose(1, 2)))
        last = G[:, -1:] if hi > lo else torch.zeros_like(S[:, 0, :1])
        hT.append(last.exp()[..., None] * S + v.transpose(1, 2) @ ((last - G).exp()[..., None] * k))
        rows.append(((b, lo, hi), y.transpose(0, 1)))
    loss = sum((y * x["dO"][b, lo:hi].double()).sum() for (b, lo, hi), y in rows)
    hT = torch.stack(hT)
    loss = loss + (hT * x["dhT"].double()).sum()
    grads = torch.autograd.grad(loss, [leaf[n] for n in NAMES])
    o = torch.zeros_like(leaf["v"].detach())
    for (b, lo, hi), y in rows:
        o[b, lo:hi] = y.detach()
    return dict(o=o, hT=hT.detach(), **{"d" + n: t for n, t in zip(NAMES, grads)})


def check(got, x, scale=1.0, cu=None):
    x = {n: t.cuda() for n, t in x.items()} if torch.cuda.is_available() else x
    ref, mag = whole(x, scale, cu), whole(base.absolute(x), abs(scale), cu)
    T = x["q"].shape[1] if cu is None else max(b - a for a, b in zip(cu, cu[1:]))
    own = (x["q"].double().abs() * mag["dq"] + x["k"].double().abs() * mag["dk"]).sum(-1)
    own = own.repeat_interleave(x["v"].shape[2] // own.shape[2], 2)
    run = torch.nn.functional.pad(own, (0, 0, 0, 128)).cumsum(1)  # over the 128 tokens from t on
    mag["dg"] = mag["dg"] + run[:, 127:-1] - torch.nn.functional.pad(run, (0, 0, 1, 0))[:, :own.shape[1]]
    for n, t in got.items():
        if t is None:
            continue
        err, lim = (t.detach().double() - ref[n]).abs(), base.tolerance(n, ref[n], mag[n], x, T)
        assert bool((err <= lim).all()), (n, float((err / lim).max()))


def test_whole_sequences_are_the_token_loop():
    """The reference here against the oracle."""
    cu = [0, 5, 5, 19]
    x = base.make(1, 19, 4, 2, 16, 32, "f32", seed=71, nstates=3)
    mine, ref = whole(x, 0.7, cu), base.oracle_both(x, cu, 0.7)
    for n in ref:
        assert torch.allclose(mine[n], ref[n], rtol=1e-10, atol=1e-12), n
    assert torch.allclose(whole(base.make(2, 9, 2, 1, 16, 16, "f32", seed=72), 1.0)["o"],
                          decay.forward(*(base.make(2, 9, 2, 1, 16, 16, "f32", seed=72)[n] for n in NAMES))[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_results_leave_whole_under_memory_traffic(dev, dk, dv):
    """dq, dk and dv leave through the same shared memory one after the other: each store has
    to have read its source before the next result comes.  Whole chunks, a key head per
    value head, copies on another stream that hold the stores up; every call the same."""
    B, T, H = 3, 640, 20
    x = base.make(B, T, H, H, dk, dv, "bf16", seed=73)
    d = {n: t.to(dev) for n, t in x.items()}
    a = [d[n] for n in ("q", "k", "v", "g", "dO", "h0", "dhT")]
    want = gdn.gdn_decay_bwd(*a, scale=0.5)
    torch.cuda.synchronize()
    check(want, x, 0.5)
    src, dst = (torch.empty(1 << 28, dtype=torch.uint8, device=dev) for _ in range(2))
    side = torch.cuda.Stream()
    got = []
    with torch.cuda.stream(side):
        for _ in range(40):
            dst.copy_(src)
    for _ in range(30):
        got.append(gdn.gdn_decay_bwd(*a, scale=0.5))
    torch.cuda.synchronize()
    for r in got:
        for n in want:
            assert torch.equal(r[n], want[n]), n


DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


def both(x, dev, cu=None):
    got = base.run(x, dev, cu, scale=0.5)
    again = base.run(x, dev, cu, scale=0.5)
    for n in got:
        assert torch.equal(got[n], again[n]), n
    check(got, x, 0.5, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [640, 645])
@pytest.mark.parametrize("Hk", [20, 5])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_several_chunks_per_cta(dev, dk, dv, Hk, T):
    """360 chunk-heads, whole chunks alone or with a chunk of 5 tokens at each sequence's end."""
    both(base.make(3, T, 20, Hk, dk, dv, "bf16", seed=74), dev)


@pytest.mark.gpu
@pytest.mark.parametrize("Hk", [24, 6])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_several_chunks_per_cta_packed(dev, dk, dv, Hk):
    """Sequences of all lengths: whole and short chunks in any order on a CTA, empty slots
    between them, tokens of no sequence around them."""
    cu = [7, 7, 8, 136, 400, 401, 657, 657, 700, 1213, 1500]
    x = base.make(1, 1510, 24, Hk, dk, dv, "bf16", seed=75, nstates=len(cu) - 1)
    d = {n: t.to(dev) for n, t in x.items()}
    c = torch.tensor(cu, dtype=torch.int32, device=dev)
    a = [d[n] for n in ("q", "k", "v", "g")]
    runs = []
    for _ in range(2):
        out = {n: torch.zeros_like(d[n[1:]]) for n in ("dq", "dk", "dv", "dg")}
        o, hT = gdn.gdn_decay_fwd(*a, d["h0"], cu_seqlens=c, scale=0.5, o=torch.zeros_like(d["v"]))
        r = gdn.gdn_decay_bwd(*a, d["dO"], d["h0"], d["dhT"], cu_seqlens=c, scale=0.5, out=out)
        runs.append(dict(o=o, hT=hT, **r))
    torch.cuda.synchronize()
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n
    check(runs[0], x, 0.5, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 64), ("bf16", 128, 128), ("f32", 64, 64), ("f32", 16, 32)])
def test_batches_in_runs(dev, dtype, dk, dv):
    """More than one sequence and few heads: every sequence of the batch is cut into runs."""
    both(base.make(2, 3001, 1, 1, dk, dv, dtype, seed=76, shift=-5.0), dev)
    both(base.make(3, 1100, 2, 1, dk, dv, dtype, seed=77, shift=-4.0), dev)
