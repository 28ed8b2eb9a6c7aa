"""gdn_tree_attn with a v that is not finite: the nodes that see it are NaN, in its channel at
least, and the others as without it, bit for bit."""
import pytest
import torch

from . import test_gpu_tree_attn as base

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


def sees(parent, j):
    """Whether each node of a tree has j on its path."""
    up = parent.tolist()
    out = []
    for i in range(len(up)):
        k = i
        while k > j:
            k = up[k]
        out.append(k == j)
    return torch.tensor(out)


def depths(parent):
    d = []
    for p in parent.tolist():
        d.append(d[p] + 1 if p >= 0 else 0)
    return torch.tensor(d)


def check(got, clean, n, rows, head, channel, group):
    """Rows of sequence n lost for the query heads of a key head; all else the same."""
    lost = torch.zeros(clean.shape[:3], dtype=torch.bool, device=clean.device)
    lost[n, rows.to(clean.device), head * group:(head + 1) * group] = True
    assert bool(got[lost][:, channel].isnan().all())
    assert torch.equal(got[~lost], clean[~lost])


# units with CTAs of their own; the steps cut evenly; several row tiles; short and empty caches
CASES = [([300, 140], 12, 4, 2, 64, 32), ([900, 10], 33, 8, 1, 128, 16), ([200 + 7 * n for n in range(40)], 7, 8, 4, 64, 64),
         ([0, 130], 64, 16, 2, 128, 128), ([2000, 3], 5, 6, 2, 128, 64)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("window", [0, 3, 200])
def test_nodes(dev, case, window):
    x = base.make(*case, kind="random", seed=141)
    N, M, Hq, Hkv = len(case[0]), *case[1:4]
    clean = base.run(x, dev, 0.125, window)
    for t, j in enumerate((0, M // 2, M - 1)):
        y = {n: a.clone() for n, a in x.items()}
        n, head, c = t % N, t % Hkv, (11 * t) % case[4]
        y["v"][n, j, head, c] = BAD[t]
        d = depths(x["parent"][n])
        rows = sees(x["parent"][n], j)
        if window:
            rows &= d - d[j] < window
        assert bool(rows.any())
        check(base.run(y, dev, 0.125, window), clean, n, rows, head, c, Hq // Hkv)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("window", [2, 5, 64, 131])
def test_cached_positions_at_the_window(dev, case, window):
    """Positions that the first nodes see and deeper ones do not, those just out of sight,
    and the last."""
    x = base.make(*case, kind="chain", seed=142)
    N, M, Hq, Hkv, d, page = len(case[0]), *case[1:]
    clean = base.run(x, dev, 0.125, window)
    depth = torch.arange(M)
    for n in {0, N - 1}:
        L = case[0][n]
        for t, p in enumerate((L - window, L - window + 1, L - window + 2, L - 1)):
            if not 0 <= p < L:
                continue
            y = {m: a.clone() for m, a in x.items()}
            head, c = t % Hkv, (13 * t) % d
            y["vc"][x["table"][n, p // page], p % page, head, c] = BAD[t % 3]
            check(base.run(y, dev, 0.125, window), clean, n, L + depth - p < window, head, c, Hq // Hkv)


def test_several(dev):
    """Nodes on different branches, and one under another."""
    x = base.make([150], 6, 2, 2, 64, 32, seed=143)
    x["parent"][0] = torch.tensor([-1, 0, 0, 1, 2, -1])
    clean = base.run(x, dev, 0.125)
    y = {n: a.clone() for n, a in x.items()}
    y["v"][0, 1, 0, 3] = y["v"][0, 3, 0, 9] = float("inf")
    y["v"][0, 5, 0, 60] = float("nan")
    got = base.run(y, dev, 0.125)
    assert torch.equal(got[:, [0, 2, 4]], clean[:, [0, 2, 4]]) and torch.equal(got[:, :, 1], clean[:, :, 1])
    assert bool(got[0, [1, 3], 0, 3].isnan().all()) and bool(got[0, 3, 0, 9].isnan()) and bool(got[0, 5, 0, 60].isnan())
