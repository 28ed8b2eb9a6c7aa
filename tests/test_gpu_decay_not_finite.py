"""Values that are not finite in gdn_decay_*: they reach what depends on them and nothing
else, bit for bit."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

from . import test_gpu_decay as base

pytestmark = pytest.mark.gpu

# (dtype, dk, dv): tensor cores, and CUDA cores with 16, 32 and 64 rows of the state per CTA
KINDS = [("bf16", 64, 64), ("bf16", 128, 64), ("bf16", 128, 128), ("bf16", 16, 32), ("bf16", 32, 128), ("f32", 64, 64),
         ("f32", 128, 128), ("f32", 16, 16), ("f32", 64, 32)]
BAD = [float("inf"), float("-inf"), float("nan")]


def forward(x, dev, cu=None):
    d = {n: t.to(dev) for n, t in x.items()}
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev)
    o, hT = gdn.gdn_decay_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], cu_seqlens=c, scale=0.5)
    torch.cuda.synchronize()
    return o.cpu(), hT.cpu()


@pytest.mark.parametrize("dtype,dk,dv", KINDS)
def test_values(dev, dtype, dk, dv):
    """One entry of v: its channel from its token on, in o and the last state."""
    x = base.make(2, 300, 4, 2, dk, dv, dtype, seed=101)
    o, hT = forward(x, dev)
    for i, t in enumerate((0, 5, 31, 32, 100, 127, 128, 255, 299)):
        y, h, c = {n: a.clone() for n, a in x.items()}, i % 4, (7 * i) % dv
        y["v"][1, t, h, c] = BAD[i % 3]
        po, ph = forward(y, dev)
        lost = torch.zeros(o.shape, dtype=torch.bool)
        lost[1, t:, h, c] = True
        assert torch.equal(po.isnan(), lost), t
        assert torch.equal(po[~lost], o[~lost]), t
        assert bool(ph[1, h, c].isnan().all())
        ph[1, h, c] = hT[1, h, c]
        assert torch.equal(ph, hT), t


@pytest.mark.parametrize("dtype,dk,dv", KINDS)
def test_several_values(dev, dtype, dk, dv):
    """A row of v, and entries before and behind it in the same and in other chunks."""
    x = base.make(1, 300, 2, 2, dk, dv, dtype, seed=102)
    o, _ = forward(x, dev)
    y = {n: a.clone() for n, a in x.items()}
    y["v"][0, 150, 1] = float("nan")
    y["v"][0, 140, 1, 3] = y["v"][0, 160, 1, 3] = float("inf")
    y["v"][0, 20, 1, 9] = y["v"][0, 21, 1, 8] = float("-inf")
    po, ph = forward(y, dev)
    lost = torch.zeros(o.shape, dtype=torch.bool)
    lost[0, 150:, 1] = lost[0, 140:, 1, 3] = lost[0, 20:, 1, 9] = lost[0, 21:, 1, 8] = True
    assert torch.equal(po.isnan(), lost) and torch.equal(po[~lost], o[~lost])
    assert bool(ph[0, 1].isnan().all()) and bool(ph[0, 0].isfinite().all())


@pytest.mark.parametrize("dtype,dk,dv", KINDS)
def test_keys_and_queries(dev, dtype, dk, dv):
    """k: every channel from its token on, for both value heads of the key head; q: its token."""
    x = base.make(2, 300, 4, 2, dk, dv, dtype, seed=103)
    o, hT = forward(x, dev)
    for i, t in enumerate((0, 31, 32, 127, 128, 299)):
        y = {n: a.clone() for n, a in x.items()}
        y["k"][0, t, 1, 3] = BAD[i % 3]
        po, ph = forward(y, dev)
        lost = torch.zeros(o.shape, dtype=torch.bool)
        lost[0, t:, 2:] = True
        assert torch.equal(po[~lost], o[~lost]) and not bool(po[lost].isfinite().any()), t
        assert torch.equal(ph[1], hT[1]) and torch.equal(ph[0, :2], hT[0, :2]) and not bool(ph[0, 2:, :, 3].isfinite().any())
        y = {n: a.clone() for n, a in x.items()}
        y["q"][0, t, 1, 3] = BAD[i % 3]
        po, ph = forward(y, dev)
        lost[0, t + 1:] = False
        assert torch.equal(po[~lost], o[~lost]) and not bool(po[lost].isfinite().any()), t
        assert torch.equal(ph, hT), t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_batch(dev, dtype):
    """Sequences of a batch that end early, with whatever the memory held behind them."""
    x = base.make(3, 290, 2, 1, 64, 64, dtype, seed=104)
    o, _ = forward(x, dev)
    y = {n: a.clone() for n, a in x.items()}
    for b, n in enumerate((290, 133, 40)):
        for name in ("q", "k", "v", "g"):
            y[name][b, n:] = float("nan")
    po, _ = forward(y, dev)
    for b, n in enumerate((290, 133, 40)):
        assert torch.equal(po[b, :n], o[b, :n]), b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_runs(dev, dtype):
    """A long chain, cut into runs: the runs before the value's, and those behind it."""
    x = base.make(1, 2500, 1, 1, 64, 64, dtype, seed=105, shift=-4.0)
    o, hT = forward(x, dev)
    for t in (3, 700, 1111, 2499):
        y = {n: a.clone() for n, a in x.items()}
        y["v"][0, t, 0, 5] = float("inf")
        po, ph = forward(y, dev)
        lost = torch.zeros(o.shape, dtype=torch.bool)
        lost[0, t:, 0, 5] = True
        assert torch.equal(po.isnan(), lost) and torch.equal(po[~lost], o[~lost]), t
        assert bool(ph[0, 0, 5].isnan().all())


@pytest.mark.parametrize("dtype,dk,dv", KINDS)
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_other_sequences(dev, dtype, dk, dv, packed):
    cu = [0, 140, 303, 303, 420] if packed else None
    x = base.make(1 if packed else 3, 420 if packed else 140, 4, 2, dk, dv, dtype, seed=106, nstates=4 if packed else 3)
    want = base.run(x, dev, cu)
    for name in ("q", "k", "v", "dO", "g"):
        y = {n: a.clone() for n, a in x.items()}
        rows = y[name][0, 140:303] if packed else y[name][1]
        rows[17] = rows[131] = float("nan")
        got = base.run(y, dev, cu)
        for n in want:
            a, b = got[n].cpu(), want[n].cpu()
            if n in ("hT", "dh0") or not packed:
                keep = [i for i in range(a.shape[0]) if i != 1]
                assert torch.equal(a[keep], b[keep]), (name, n)
            else:
                assert torch.equal(a[:, :140], b[:, :140]) and torch.equal(a[:, 303:], b[:, 303:]), (name, n)
