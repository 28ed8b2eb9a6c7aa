"""Numbers that a C int cannot hold: ctypes would drop their higher bits and run the call
with what is left."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

from . import test_gpu_tree_attn as tree_tests

BIG = 2 ** 32


class Shaped:
    """A tensor as the checks see it, of a shape that nobody allocates."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda:0")

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)


def test_sizes_of_the_first_tensors(monkeypatch):
    monkeypatch.setattr(gdn, "_need", lambda *a: None)
    for shape in ((1, BIG + 5, 1, 16), (1, 4, 1, BIG + 16), (BIG + 1, 4, 1, 16)):
        q = Shaped(shape, torch.bfloat16)
        for _ in range(2):  # the first call of a type, and the next
            with pytest.raises(ValueError, match="more than"):
                gdn._lead(q, "q", 4)
    assert gdn._lead(Shaped((1, 4, 2, 16), torch.bfloat16), "q", 4)[0] == gdn.GDN_BF16
    assert gdn._lead(Shaped((2 ** 31 - 1, 4, 2, 16), torch.bfloat16), "q", 4)[0] == gdn.GDN_BF16
    x = Shaped((2, BIG + 32), torch.bfloat16)
    with pytest.raises(ValueError, match="more than"):
        gdn._norm_inputs(x, x, x)


def test_sizes_of_the_others():
    assert gdn._int(2 ** 31 - 1, "nseq") == 2 ** 31 - 1
    for n in (2 ** 31, BIG + 5):
        with pytest.raises(ValueError):
            gdn._int(n, "nseq")


@pytest.mark.gpu
def test_windows(dev):
    """A window that no position is outside of is none; a negative one is refused."""
    x = tree_tests.make([300, 64, 0, 131], 12, 4, 2, 64, 32, kind="kary", seed=95)
    want = tree_tests.run(x, dev, 0.125, 0)
    assert not torch.equal(want, tree_tests.run(x, dev, 0.125, 5))
    for window in (2 ** 31 - 1, 2 ** 31, BIG, BIG + 5, 2 ** 63):
        assert torch.equal(tree_tests.run(x, dev, 0.125, window), want), window
    for window in (-1, -BIG, 5 - BIG):
        with pytest.raises(gdn.GdnError):
            tree_tests.run(x, dev, 0.125, window)
    with pytest.raises(Exception):
        tree_tests.run(x, dev, 0.125, 5.5)


@pytest.mark.gpu
def test_wide_table(dev):
    """A block table of 2^32 + 5 entries is refused, not read as one of 5."""
    x = {n: t.to(dev) for n, t in tree_tests.make([30], 2, 2, 2, 64, 16, seed=96).items()}
    wide = torch.empty(1, BIG + 5, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="more than"):
        gdn.gdn_tree_attn(x["parent"], x["q"], x["k"], x["v"], x["kc"], x["vc"], wide, x["lens"])
    with pytest.raises(ValueError, match="more than"):
        gdn.gdn_tree_append(x["parent"], x["lens"], x["k"], x["v"], x["kc"], x["vc"], wide, x["lens"])
