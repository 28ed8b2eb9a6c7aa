"""gdn_decay_fwd / gdn_decay_bwd on tensor cores for sequences of up to 64 tokens, whose pair
products are two bf16 terms: where a row has few of them, one rounding would be the largest
error.

The bounds of test_gpu_decay.py with 2^-16 in place of 2^-8 for what a product's operand was
rounded to; a state enters o (only) in bf16, so o is taken without one."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

from . import test_gpu_decay as base

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 64), (64, 128), (128, 128)]


def check(got, x, names, cu=None, scale=1.0, keep=slice(None)):
    ref, mag = base.oracle_both(x, cu, scale), base.oracle_both(base.absolute(x), cu, abs(scale))
    T, dk, dv = x["q"].shape[1], x["q"].shape[-1], x["v"].shape[-1]
    c = (6 * T + 2 * dk + 2 * dv + 64) * 2.0 ** -24 + 2.0 ** -16
    for n in names:
        err = (got[n].double().cpu() - ref[n]).abs()[:, keep]
        lim = c * mag[n] + 2.0 ** -8 * (ref[n].abs() + c * mag[n]) + 1e-30
        assert bool((err <= lim[:, keep]).all()), (n, float((err / lim[:, keep]).max()))


@pytest.mark.parametrize("T", [1, 2, 3, 5, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_batches(dev, dk, dv, T):
    for H, Hk in ((4, 4), (4, 2)):
        x = base.make(3, T, H, Hk, dk, dv, "bf16", seed=151 + T, shift=1.0)
        check(base.run(x, dev, scale=0.7), x, ("dq", "dk", "dv"), scale=0.7)
        y = dict(x, h0=torch.zeros_like(x["h0"]))
        check(base.run(y, dev, scale=0.7), y, ("o",), scale=0.7)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_packed(dev, dk, dv):
    """One sequence longer than a chunk among short ones, ends around 64."""
    cu = [0, 64, 64, 65, 128, 193, 323, 327, 340, 341, 380]
    x = base.make(1, 380, 4, 4, dk, dv, "bf16", seed=161, nstates=10, shift=1.0)
    got = base.run(x, dev, cu, scale=0.7)
    base.check(got, x, cu, scale=0.7)
    short = [t for a, b in zip(cu, cu[1:]) if b - a <= 64 for t in range(a, b)]
    check(got, x, ("dq", "dk", "dv"), cu, 0.7, short)
    y = dict(x, h0=torch.zeros_like(x["h0"]))
    check(base.run(y, dev, cu, scale=0.7), y, ("o",), cu, 0.7, short)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_many_chunks_per_cta(dev, dk, dv):
    """More short sequences than SMs, rows behind them full of NaN, the same twice."""
    cu = [0]
    for n in range(40):
        cu.append(cu[-1] + (n * 17) % 62)
    x = base.make(1, cu[-1] + 9, 10, 10, dk, dv, "bf16", seed=162, nstates=40, shift=1.0)
    for n in ("q", "k", "v", "g", "dO"):
        x[n][:, cu[-1]:] = float("nan")
    a, b = base.run(x, dev, cu), base.run(x, dev, cu)
    y = {n: t if t.shape[0] == 40 else t[:, :cu[-1]].contiguous() for n, t in x.items()}
    rows = slice(0, cu[-1])
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(a[n][:, rows], b[n][:, rows]), n
    check({n: a[n][:, rows] for n in ("dq", "dk", "dv")}, y, ("dq", "dk", "dv"), cu)
    base.check({n: a[n] if n in ("hT", "dh0") else a[n][:, rows] for n in a}, y, cu)


def test_values_that_are_not_finite(dev):
    """The second half of a short chunk's v is a copy: it must not bring them back."""
    for T in (40, 64):
        x = base.make(2, T, 2, 2, 64, 64, "bf16", seed=163)
        o, _ = gdn.gdn_decay_fwd(*(x[n].to(dev) for n in ("q", "k", "v", "g", "h0")))
        for t, bad in ((0, float("nan")), (17, float("inf")), (T - 1, float("-inf"))):
            y = {n: a.clone() for n, a in x.items()}
            y["v"][1, t, 1, 9] = y["v"][1, t, 1, 20] = bad
            p, _ = gdn.gdn_decay_fwd(*(y[n].to(dev) for n in ("q", "k", "v", "g", "h0")))
            lost = torch.zeros(o.shape, dtype=torch.bool, device=dev)
            lost[1, t:, 1, 9] = lost[1, t:, 1, 20] = True
            assert torch.equal(p.isnan(), lost) and torch.equal(p[~lost], o[~lost]), (T, t)
