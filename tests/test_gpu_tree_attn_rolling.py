"""gdn_tree_attn over a rolling cache: pages that lie wholly before the window have been
given back, and their table entries name no page."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

from . import test_gpu_tree_attn as base

pytestmark = pytest.mark.gpu


def workspace(x, dev):
    N, M, Hq, d = x["q"].shape
    return torch.empty(int(gdn.lib().gdn_tree_attn_workspace(N, M, Hq, x["k"].shape[2], d, gdn.GDN_BF16, x["kc"].shape[1],
                                                             x["table"].shape[1])), dtype=torch.uint8, device=dev)


@pytest.mark.parametrize("gone", [-1, 10 ** 6])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 65, 128, 200, 500])
def test_pages_given_back_are_not_read(dev, window, page, gone):
    """Lengths around whole pages and tiles.  The pages themselves hold NaN."""
    x = base.poison(base.make([300, 64, 0, 131, 256, 257, 640], 9, 4, 2, 64, page, kind="kary", seed=91))
    want = base.run(x, dev, 0.125, window)
    y = {n: t.clone() for n, t in x.items()}
    left = 0
    for n, L in enumerate(y["lens"].tolist()):
        for i in range(-(-L // page)):
            if (i + 1) * page <= L - window + 1:
                y["kc"][x["table"][n, i].long()] = y["vc"][x["table"][n, i].long()] = float("nan")
                y["table"][n, i] = gone
                left += 1
    assert left
    ws = workspace(y, dev)
    got = base.run(y, dev, 0.125, window, workspace=ws)
    assert gdn.gdn_query_device_status(ws) == gdn.GDN_OK
    assert torch.equal(got, want)
    base.check(x, dev, 0.125, window, o=got)


def test_pages_in_sight_are_still_checked(dev):
    """The page that holds the window's first position, and the one after it."""
    x = base.make([300], 3, 2, 2, 64, 32, kind="chain", seed=92)
    window = 100  # positions 201 .. 299: pages 6 .. 9
    for i, code in ((5, gdn.GDN_OK), (6, gdn.GDN_ERR_INVALID_ARG), (7, gdn.GDN_ERR_INVALID_ARG), (9, gdn.GDN_ERR_INVALID_ARG)):
        y = {n: t.clone() for n, t in x.items()}
        y["table"][0, i] = -1
        ws = workspace(y, dev)
        base.run(y, dev, 0.125, window, workspace=ws)
        assert gdn.gdn_query_device_status(ws) == code, i
