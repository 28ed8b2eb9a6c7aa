"""gdn_tree_attn where the products of its steps and CTAs pass 31 bits."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

pytestmark = pytest.mark.gpu


def test_longest_caches_on_all_ctas(dev):
    """One sequence of 1.9e9 positions, its pages shared by the table's entries: 14.8 million
    key tiles, cut over all SMs.  A page counts as often as the table names it, so the
    result is a softmax of 8 pages with multiplicities.  Bound: weights in bf16 (2^-8, and
    as much for the result), and fp32 sums over the 16-key pieces of a CTA's share, which
    may drop up to a step (2^-23) each."""
    L, page, pages, d = 1_900_000_000, 128, 8, 64
    width = -(-L // page)
    gen = torch.Generator().manual_seed(81)
    kc, vc = (torch.randn(pages, page, 1, d, generator=gen).bfloat16() for _ in range(2))
    vc = (vc.float() * 0.25 + 1).bfloat16()
    q, k, v = (torch.randn(1, 1, 1, d, generator=gen).bfloat16() for _ in range(3))
    table = torch.randint(0, pages, (1, width), generator=gen, dtype=torch.int32)
    o = torch.full((1, 1, 1, d), float("nan"), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(int(gdn.lib().gdn_tree_attn_workspace(1, 1, 1, 1, d, gdn.GDN_BF16, page, width)),
                     dtype=torch.uint8, device=dev)
    gdn.gdn_tree_attn(torch.full((1, 1), -1, dtype=torch.int32, device=dev), q.to(dev), k.to(dev), v.to(dev), kc.to(dev),
                      vc.to(dev), table.to(dev), torch.tensor([L], dtype=torch.int32, device=dev), scale=0.125, o=o,
                      workspace=ws)
    assert gdn.gdn_query_device_status(ws) == gdn.GDN_OK
    times = torch.bincount(table[0, :-1].long(), minlength=pages).double()[:, None].repeat(1, page)
    times[table[0, -1].long(), :L - (width - 1) * page] += 1
    s = 0.125 * (kc[:, :, 0].double() @ q[0, 0, 0].double())
    w = times * torch.exp(s - s.max())
    own = torch.exp(0.125 * (k[0, 0, 0].double() @ q[0, 0, 0].double()) - s.max())
    total = w.sum() + own
    ref = ((w[..., None] * vc[:, :, 0].double()).sum((0, 1)) + own * v[0, 0, 0].double()) / total
    mag = ((w[..., None] * vc[:, :, 0].double().abs()).sum((0, 1)) + own * v[0, 0, 0].double().abs()) / total
    c = 2.0 ** -8 + (width / 148 * 8) * 2.0 ** -23
    err = (o[0, 0, 0].double().cpu() - ref).abs()
    assert bool((err <= c * mag + 2.0 ** -8 * (ref.abs() + c * mag)).all()), float((err / mag).max())
