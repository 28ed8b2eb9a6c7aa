"""The output norm and gate in fp64, gradients written out."""
from __future__ import annotations

import torch


def _parts(x, z, eps, center):
    x, z = x.detach().double().cpu(), z.detach().double().cpu()
    c = x - x.mean(-1, keepdim=True) if center else x
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    return c * r, r, z, torch.sigmoid(z)


def forward(x, z, w, eps=1e-6, center=False):
    h, _, z, sg = _parts(x, z, eps, center)
    return w.detach().double().cpu() * h * z * sg


def backward(x, z, w, dy, eps=1e-6, center=False):
    """(dx, dz, dw) and the sums of absolute terms behind dx and dw."""
    h, r, z, sg = _parts(x, z, eps, center)
    w, dy = w.detach().double().cpu(), dy.detach().double().cpu()
    e = dy * w * z * sg
    dx = e - h * (e * h).mean(-1, keepdim=True)
    mag = e.abs() + h.abs() * (e * h).abs().mean(-1, keepdim=True)
    if center:
        dx = dx - e.mean(-1, keepdim=True)
        mag = mag + e.abs().mean(-1, keepdim=True)
    dz = dy * w * h * sg * (1 + z * (1 - sg))
    t = dy * h * z * sg
    dims = tuple(range(t.dim() - (1 if w.dim() == 1 else 2)))
    return dx * r, dz, t.sum(dims), mag * r, t.abs().sum(dims)
