"""gdn_tree_attn / gdn_tree_append against the fp64 oracle.

Bound of o: a score is a dot product of d exact bf16 products in fp32, at most
e_s = (d + 8) 2^-24 sum|scale q k| off, and exp adds 2 steps; a weight is rounded to bf16
(half a step, 2^-8) for its product with v; the sums of weights and of products
are fp32 over L + M terms with at most log-many rescalings:
|o - ref| <= (2^-8 + 2 e_s + (L + M + 64) 2^-24) mag, mag = sum p |v|, and half a step
of bf16 of the result."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn
from oracle import tree_attn as oracle

pytestmark = pytest.mark.gpu


def parents(N, M, kind, gen):
    if kind == "chain":
        return (torch.arange(M) - 1).repeat(N, 1).int()
    if kind == "star":
        return torch.full((N, M), -1, dtype=torch.int32)
    if kind == "kary":
        return torch.div(torch.arange(M) - 1, 3, rounding_mode="floor").repeat(N, 1).int()
    return torch.stack([torch.tensor([int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(M)])
                        for _ in range(N)]).int()


def make(lens, M, Hq, Hkv, d, page, kind="random", seed=0, amp=1.5):
    gen = torch.Generator().manual_seed(seed * 77 + M + page)
    N = len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    used = [-(-(n + M) // page) for n in lens]
    width = max(used) + 1
    order = torch.randperm(sum(used) + 2, generator=gen).int()
    table, at = torch.full((N, width), -1, dtype=torch.int32), 0
    for n, u in enumerate(used):
        table[n, :u] = order[at:at + u]
        at += u
    kc, vc = (r(sum(used) + 2, page, Hkv, d).bfloat16() for _ in range(2))
    return dict(parent=parents(N, M, kind, gen), q=(amp * r(N, M, Hq, d)).bfloat16(), k=r(N, M, Hkv, d).bfloat16(),
                v=r(N, M, Hkv, d).bfloat16(), kc=kc, vc=vc, table=table, lens=torch.tensor(lens, dtype=torch.int32))


def poison(x):
    """NaN in every cached row that no sequence may see."""
    page = x["kc"].shape[1]
    seen = torch.zeros(x["kc"].shape[:2], dtype=torch.bool)
    for n, L in enumerate(x["lens"].tolist()):
        for p in range(L):
            seen[x["table"][n, p // page], p % page] = True
    for c in ("kc", "vc"):
        x[c][~seen] = float("nan")
    return x


def run(x, dev, scale, window=0, **kw):
    d = {n: t.to(dev) for n, t in x.items()}
    o = gdn.gdn_tree_attn(d["parent"], d["q"], d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"], scale=scale,
                          window=window, **kw)
    torch.cuda.synchronize()
    return o


def check(x, dev, scale, window=0, o=None):
    o = run(x, dev, scale, window) if o is None else o
    ref, mag = oracle.attend(x["parent"], x["q"], x["k"], x["v"], x["kc"], x["vc"], x["table"], x["lens"], scale, window)
    d, L = x["q"].shape[-1], int(x["lens"].max()) + x["q"].shape[1]
    norm = x["q"].double().norm(dim=-1).amax() * max(float(x[n].double().nan_to_num().norm(dim=-1).amax()) for n in ("k", "kc"))
    c = 2.0 ** -8 + 2 * (d + 8) * 2.0 ** -24 * abs(scale) * float(norm) + (L + 64) * 2.0 ** -24
    err = (o.double().cpu() - ref).abs()
    lim = c * mag + 2.0 ** -8 * (ref.abs() + c * mag)
    assert bool((err <= lim).all()), float((err / lim).max())


CASES = [([0], 1, 1, 1, 64, 16), ([1, 0, 5], 3, 2, 1, 128, 16), ([130, 127, 128], 5, 4, 2, 64, 32),
         ([33, 300], 16, 8, 2, 128, 64), ([257], 64, 4, 4, 128, 128), ([40, 129], 33, 6, 1, 64, 16),
         ([515, 3], 1, 16, 2, 128, 64), ([200], 64, 16, 2, 64, 128), ([1300, 900, 1111], 1, 5, 5, 64, 16),
         ([900, 10], 3, 3, 1, 128, 32), ([640], 50, 6, 2, 64, 64)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_matches_oracle(dev, case, kind):
    x = poison(make(*case, kind=kind, seed=1))
    check(x, dev, case[4] ** -0.5)


@pytest.mark.parametrize("window", [1, 2, 7, 64, 128, 129, 10 ** 6])
def test_sliding_window(dev, window):
    x = poison(make([300, 64, 0, 131], 12, 4, 2, 64, 32, kind="kary", seed=2))
    check(x, dev, 0.125, window)


@pytest.mark.parametrize("scale", [-0.125, 0.0])
def test_scales_that_are_not_positive(dev, scale):
    check(poison(make([300, 5], 9, 4, 2, 64, 32, seed=12)), dev, scale)


@pytest.mark.parametrize("N,M,Hq,Hkv", [(40, 3, 4, 4), (75, 1, 2, 1), (160, 2, 2, 2)])
def test_many_sequences(dev, N, M, Hq, Hkv):
    """Units for half the SMs and more: CTAs work on several, sequences of all lengths."""
    lens = [(37 * n) % 300 for n in range(N)]
    check(poison(make(lens, M, Hq, Hkv, 64, 32, kind="chain", seed=13)), dev, 0.125)


def test_large_scores(dev):
    """Scores of several hundred: nearly one-hot weights, the maximum changing
    from tile to tile."""
    x = poison(make([700, 400], 8, 4, 1, 128, 64, seed=3, amp=12.0))
    check(x, dev, 0.3)


def test_long_cache_is_split(dev):
    x = poison(make([2600, 1900], 4, 4, 2, 64, 64, kind="kary", seed=4))
    check(x, dev, 0.125)


def test_shared_pages_and_repeatable(dev):
    """Two sequences on the same cached pages; the same call twice."""
    x = make([200, 150], 6, 4, 2, 128, 64, seed=5)
    x["table"][1, :4] = x["table"][0, :4]
    check(x, dev, 0.1)
    assert torch.equal(run(x, dev, 0.1), run(x, dev, 0.1))


def test_device_data_is_checked(dev):
    x = make([100, 60], 4, 2, 2, 64, 16, seed=6)
    ws = torch.empty(int(gdn.lib().gdn_tree_attn_workspace(2, 4, 2, 2, 64, gdn.GDN_BF16, 16, x["table"].shape[1])),
                     dtype=torch.uint8, device=dev)
    good = run(x, dev, 0.125, workspace=ws)
    assert gdn.gdn_query_device_status(ws) == gdn.GDN_OK
    for name, at, value in (("parent", (0, 2), 3), ("lens", (0,), 10 ** 6), ("lens", (0,), -5), ("table", (0, 1), 10 ** 6),
                            ("table", (0, 1), -1)):
        y = {n: t.clone() for n, t in x.items()}
        y[name][at] = value
        o = run(y, dev, 0.125, workspace=ws)
        assert gdn.gdn_query_device_status(ws) == gdn.GDN_ERR_INVALID_ARG, (name, value)
        assert torch.equal(o[1], good[1])
        if name == "parent":
            y["parent"][0, 2] = -1
            check(y, dev, 0.125, o=o)
        elif name == "lens":
            y["lens"][0] = 0
            check(y, dev, 0.125, o=o)
        else:  # positions 16 .. 31 of sequence 0 are not seen
            z = {n: t[:1] if n not in ("kc", "vc") else t for n, t in x.items()}
            keep = [p for p in range(100) if not 16 <= p < 32]
            flat = lambda c: c[z["table"][0, :7].long()].flatten(0, 1)[keep]  # noqa: E731
            pad = lambda c: torch.cat([c, c[:12]]).reshape(6, 16, 2, 64)  # noqa: E731
            z = dict(z, kc=pad(flat(x["kc"])), vc=pad(flat(x["vc"])), table=torch.arange(6).int()[None],
                     lens=torch.tensor([84], dtype=torch.int32))
            check(z, dev, 0.125, o=o[:1])


@pytest.mark.parametrize("M,page,kind", [(1, 16, "star"), (7, 16, "chain"), (20, 32, "random"), (64, 128, "chain")])
def test_append_matches_oracle(dev, M, page, kind):
    x = make([0, 1, page - 1, page, 3 * page + 5], M, 2, 2, 64, page, kind=kind, seed=7)
    acc = torch.tensor([-1, M - 1, M - 1, M // 2, 0], dtype=torch.int32)
    d = {n: t.to(dev) for n, t in x.items()}
    new = gdn.gdn_tree_append(d["parent"], acc.to(dev), d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"])
    torch.cuda.synchronize()
    kc, vc, ref = oracle.append(x["parent"], acc, x["k"], x["v"], x["kc"], x["vc"], x["table"], x["lens"])
    assert torch.equal(new.cpu(), ref) and torch.equal(d["kc"].cpu(), kc) and torch.equal(d["vc"].cpu(), vc)
    assert torch.equal(d["lens"].cpu(), x["lens"])
    # the lengths in place
    gdn.gdn_tree_append(d["parent"], acc.to(dev), d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"],
                        new_len=d["lens"])
    assert torch.equal(d["lens"].cpu(), ref)


def test_append_leaves_bad_sequences(dev):
    x = make([30, 31, 20, 12], 4, 2, 2, 64, 16, kind="chain", seed=8)
    x["table"][0, 1] = 10 ** 6      # the path starts on this page
    x["lens"][1] = 16 * x["table"].shape[1] - 2   # no room
    x["lens"][2] = -1
    acc = torch.tensor([3, 3, 3, 9], dtype=torch.int32)
    d = {n: t.to(dev) for n, t in x.items()}
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = gdn.gdn_tree_append(d["parent"], acc.to(dev), d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"],
                              status=status)
    assert gdn.gdn_query_device_status(status) == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(new.cpu(), x["lens"])
    assert torch.equal(d["kc"].cpu(), x["kc"]) and torch.equal(d["vc"].cpu(), x["vc"])


def test_verify_append_verify(dev):
    """A drafted chain verified, appended, and the next draft verified over the
    longer cache: the same as attention over one sequence; captured in a graph."""
    x = make([45, 100], 5, 4, 2, 64, 16, kind="chain", seed=9)
    d = {n: t.to(dev) for n, t in x.items()}
    acc = torch.tensor([2, 4], dtype=torch.int32, device=dev)

    def step():
        o1 = gdn.gdn_tree_attn(d["parent"], d["q"], d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"], scale=0.125)
        n = gdn.gdn_tree_append(d["parent"], acc, d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"])
        o2 = gdn.gdn_tree_attn(d["parent"], d["q"], d["k"], d["v"], d["kc"], d["vc"], d["table"], n, scale=0.125)
        return o1, n, o2

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o1, n, o2 = step()
    for name in ("kc", "vc"):
        d[name].copy_(x[name])
    graph.replay()
    torch.cuda.synchronize()
    check(x, dev, 0.125, o=o1)
    kc, vc, new = oracle.append(x["parent"], acc.cpu(), x["k"], x["v"], x["kc"], x["vc"], x["table"], x["lens"])
    assert torch.equal(n.cpu(), new)
    check(dict(x, kc=kc, vc=vc, lens=new), dev, 0.125, o=o2)


def test_nan_reaches_who_sees_it(dev):
    """A NaN in a node's key: NaN for the node and its descendants, nothing for the others;
    one in a cached key within the length: NaN for all nodes of the sequence."""
    x = make([140, 200], 12, 4, 2, 64, 32, kind="random", seed=31)
    clean = run(x, dev, 0.125)
    y = {n: t.clone() for n, t in x.items()}
    y["k"][0, 3, 1, 5] = float("nan")
    o = run(y, dev, 0.125)
    sees = torch.zeros(12, dtype=torch.bool)
    for i in range(12):
        j = i
        while j >= 0:
            sees[i] |= j == 3
            j = int(x["parent"][0, j])
    for i in range(12):
        assert torch.equal(o[0, i, :2], clean[0, i, :2])
        assert bool(o[0, i, 2:].isnan().all()) if sees[i] else torch.equal(o[0, i, 2:], clean[0, i, 2:]), i
    assert torch.equal(o[1], clean[1])
    p = 100
    y = {n: t.clone() for n, t in x.items()}
    y["kc"][x["table"][1, p // 32], p % 32, 0, 0] = float("nan")
    o = run(y, dev, 0.125)
    assert bool(o[1, :, :2].isnan().all()) and torch.equal(o[1, :, 2:], clean[1, :, 2:]) and torch.equal(o[0], clean[0])
