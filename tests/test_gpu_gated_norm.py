"""gdn_gated_norm_fwd / gdn_gated_norm_bwd against the fp64 oracle.

Bounds: with u = 2^-24, a row's statistics are sums of d terms ((d + 8) u of their
magnitude); exp is off by 2 steps (4 u), and the sigmoid, the root, the quotients
and the products add at most 24 u more: c = (d + 32) u relative to the factors.  A
centred row adds the rounding of its mean, (d + 8) u max|x| per element before the
division by the deviation.  dw is a sum of `rows` terms in at most three stages of
fp32 sums.  Results are rounded to their type once."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn
from oracle import gated_norm as oracle

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(shape, dtype, shared, seed=0, spread=2.0):
    gen = torch.Generator().manual_seed(seed + shape[0])
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    w = 1 + 0.2 * (r(shape[-1]) if shared else r(*shape[-2:]))
    return (spread * r(*shape) + 0.4).to(DT[dtype]), (2 * r(*shape)).to(DT[dtype]), w, r(*shape).to(DT[dtype])


def check(dev, x, z, w, dy, eps, center):
    X, Z, W, DY = (t.to(dev) for t in (x, z, w, dy))
    y = gdn.gdn_gated_norm_fwd(X, Z, W, eps=eps, center=center)
    dx, dz, dw = gdn.gdn_gated_norm_bwd(X, Z, W, DY, eps=eps, center=center)
    torch.cuda.synchronize()
    d = x.shape[-1]
    u, half = 2.0 ** -24, torch.finfo(x.dtype).eps / 2
    c = (d + 32) * u
    xd = x.double()
    cc = xd - xd.mean(-1, keepdim=True) if center else xd
    r = 1 / torch.sqrt((cc * cc).mean(-1, keepdim=True) + eps)
    off = (d + 8) * u * xd.abs().amax(-1, keepdim=True) * r if center else 0.0   # of h
    h, sz = cc * r, z.double() * torch.sigmoid(z.double())
    ry = oracle.forward(x, z, w, eps, center)
    lim = c * ry.abs() + off * (w * sz).abs()
    assert bool(((y.double().cpu() - ry).abs() <= lim + half * (ry.abs() + lim) + 1e-30).all()), "y"
    rx, rz, rw, mx, mw = oracle.backward(x, z, w, dy, eps, center)
    e = (dy.double() * w * sz).abs()
    lim = 3 * c * mx + off * r * (3 * (e * h.abs()).mean(-1, keepdim=True) + 3 * h.abs() * e.mean(-1, keepdim=True) + e)
    assert bool(((dx.double().cpu() - rx).abs() <= lim + half * (rx.abs() + lim) + 1e-30).all()), "dx"
    sg = torch.sigmoid(z.double())
    lim = (c * h.abs() + off) * (dy.double() * w).abs() * sg * (1 + z.double().abs())
    assert bool(((dz.double().cpu() - rz).abs() <= lim + half * (rz.abs() + lim) + 1e-30).all()), "dz"
    rows = x.numel() // d
    # a unit sums at most rows / units + 1 terms, the second kernel at most units / 32 + 32
    terms = min(rows, 2 * (rows // 1000) + 700)
    dims = tuple(range(x.dim() - (1 if w.dim() == 1 else 2)))
    lim = (c + terms * u) * mw + (off * (dy.double() * sz).abs()).sum(dims) if center else (c + terms * u) * mw
    assert bool(((dw.double().cpu() - rw).abs() <= lim + 2 * u * rw.abs()).all()), "dw"
    return y, dx, dz, dw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 32), (5, 3, 64), (37, 6, 128), (2, 33, 5, 256), (1, 999, 1, 128),
                                   (700, 24, 32)])
def test_matches_oracle(dev, shape, dtype, center):
    for shared in (True, False):
        check(dev, *make(shape, dtype, shared), 1e-6, center)


def test_long_batch_and_repeatable(dev):
    """More rows than units: several turns per unit."""
    x, z, w, dy = make((3000, 8, 128), "bf16", True, 7)
    a = check(dev, x, z, w, dy, 1e-6, False)
    b = check(dev, x, z, w, dy, 1e-6, False)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_zero_rows_and_large_gates(dev):
    """A row of zeros (eps alone under the root) and gates far out on both sides."""
    x, z, w, dy = make((4, 2, 64), "f32", True, 9)
    x[0] = 0
    z[1], z[2] = 80.0, -80.0
    y, dx, dz, dw = check(dev, x, z, w, dy, 1e-5, False)
    for t in (y, dx, dz, dw):
        assert bool(torch.isfinite(t).all())


def test_side_stream(dev):
    x, z, w, dy = (t.to(dev) for t in make((64, 4, 128), "bf16", False, 3))
    want = gdn.gdn_gated_norm_bwd(x, z, w, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.gdn_gated_norm_bwd(x, z, w, dy, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
