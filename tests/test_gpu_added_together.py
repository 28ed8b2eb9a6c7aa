"""The decay recurrence, the output norm and gate, draft-tree attention and the cache's
append as a model calls them: one after the other, on shared workspaces, captured.

Every stage is held to its own bound (the test files of the operators derive them), with
the tensors that the stage was really given: what a stage before it rounded is an input
to the next, not an error of it."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn
from oracle import tree_attn as tree_oracle

from . import test_gpu_decay as decay_tests
from . import test_gpu_gated_norm as norm_tests
from . import test_gpu_tree_attn as tree_tests

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [None, [0, 70, 70, 199, 261]])
def test_layer_forward_backward(dev, dtype, cu):
    """o = decay(q, k, v, g), y = norm(o, z); then dy -> do, dz, dw -> dq, dk, dv, dg, dh0."""
    B, T, H = (2, 150, 4) if cu is None else (1, 261, 4)
    x = decay_tests.make(B, T, H, 2, 64, 128, dtype, seed=31, nstates=None if cu is None else len(cu) - 1)
    gen = torch.Generator().manual_seed(32)
    z = torch.randn(B, T, H, 128, generator=gen).to(x["v"].dtype)
    dy = torch.randn(B, T, H, 128, generator=gen).to(x["v"].dtype)
    w = 1 + 0.1 * torch.randn(H, 128, generator=gen)
    d = {n: t.to(dev) for n, t in x.items()}
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev)
    o, hT = gdn.gdn_decay_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], cu_seqlens=c, scale=0.5)
    _, do, _, _ = norm_tests.check(dev, o.cpu(), z, w, dy, 1e-5, False)
    r = gdn.gdn_decay_bwd(d["q"], d["k"], d["v"], d["g"], do, d["h0"], d["dhT"], cu_seqlens=c, scale=0.5)
    torch.cuda.synchronize()
    decay_tests.check(dict(o=o, hT=hT, **r), dict(x, dO=do.cpu()), cu=cu, scale=0.5)


def test_hybrid_decode_captured(dev):
    """A decode step of a linear layer and a softmax layer, captured once and replayed for
    every token, in place on the state, the cache and its lengths: the same as eager
    calls bit for bit, and every token within the bounds of its operators."""
    N, H, d, steps = 3, 4, 64, 20
    x = tree_tests.make([30, 0, 15], 1, H, 2, d, 16, kind="star", seed=21)
    x["table"] = torch.arange(N * 4, dtype=torch.int32).view(N, 4)
    gen = torch.Generator().manual_seed(22)
    kc, vc = (torch.randn(N * 4, 16, 2, d, generator=gen).bfloat16() for _ in range(2))
    q, z, kl = (torch.randn(steps, N, 1, H, d, generator=gen).bfloat16() for _ in range(3))
    k, v = (torch.randn(steps, N, 1, 2, d, generator=gen).bfloat16() for _ in range(2))
    g = -torch.rand(steps, N, H, generator=gen)
    S0, w = torch.randn(N, H, d, d, generator=gen), torch.ones(d)

    def start():
        return dict(kc=kc.to(dev), vc=vc.to(dev), n=x["lens"].to(dev), S=S0.to(dev), q=q[0].to(dev), k=k[0].to(dev),
                    v=v[0].to(dev), z=z[0].to(dev), kl=kl[0].to(dev), g=g[0].to(dev), w=w.to(dev), t=x["table"].to(dev),
                    p=x["parent"].to(dev), a=torch.zeros(N, dtype=torch.int32, device=dev))

    def step(s):
        lin = gdn.gdn_decay_step(s["q"][:, 0], s["kl"][:, 0], s["z"][:, 0], s["g"], s["S"], scale=0.125)
        y = gdn.gdn_gated_norm_fwd(lin, s["z"][:, 0], s["w"])
        o = gdn.gdn_tree_attn(s["p"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["t"], s["n"], scale=0.125)
        gdn.gdn_tree_append(s["p"], s["a"], s["k"], s["v"], s["kc"], s["vc"], s["t"], s["n"], new_len=s["n"])
        return lin, y, o

    def feed(s, t):
        for n, src in (("q", q), ("k", k), ("v", v), ("z", z), ("kl", kl), ("g", g)):
            s[n].copy_(src[t])

    eager, graphed = start(), start()
    want = []
    for t in range(steps):
        feed(eager, t)
        want.append([a.clone() for a in step(eager)])
    step(start())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(graphed)
    for n, t in start().items():
        graphed[n].copy_(t)
    for t in range(steps):
        feed(graphed, t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[t]):
            assert torch.equal(a, b), t
    for n in ("S", "kc", "vc", "n"):
        assert torch.equal(eager[n], graphed[n]), n
    assert eager["n"].tolist() == [50, 20, 35]
    # the linear layer's tokens are one prompt's
    y = dict(q=q[:, :, 0].transpose(0, 1), k=kl[:, :, 0].transpose(0, 1), v=z[:, :, 0].transpose(0, 1),
             g=g.transpose(0, 1), h0=S0)
    y = {n: t.contiguous() for n, t in y.items()}
    y.update(dO=torch.zeros_like(y["v"]), dhT=torch.zeros_like(S0))
    decay_tests.check(dict(o=torch.stack([a[0] for a in want], 1), hT=eager["S"]), y, scale=0.125)
    # the last token's attention sees the prompt and all tokens before it
    last = dict(x, q=q[-1], k=k[-1], v=v[-1], kc=eager["kc"].cpu(), vc=eager["vc"].cpu(), lens=eager["n"].cpu() - 1)
    tree_tests.check(last, dev, 0.125, o=want[-1][2])
    ref, new = (kc.clone(), vc.clone()), x["lens"]
    for t in range(steps):
        root = torch.zeros(N, dtype=torch.int32)
        *ref, new = tree_oracle.append(x["parent"], root, k[t], v[t], *ref, x["table"], new)
    assert torch.equal(eager["kc"].cpu(), ref[0]) and torch.equal(eager["vc"].cpu(), ref[1])


def test_graphs_share_workspaces(dev):
    """Two captured graphs on the same workspaces, replayed in turn on one stream."""
    xs = [decay_tests.make(1, 300, 4, 2, 128, 128, "bf16", seed=s) for s in (41, 42)]
    ts = [tree_tests.make([900, 40], 8, 8, 2, 128, 64, seed=s) for s in (43, 44)]
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev)
    tws = torch.empty(1 << 26, dtype=torch.uint8, device=dev)
    graphs, outs, plain, held = [], [], [], []  # a graph reads its inputs where they were
    for x, t in zip(xs, ts):
        d, e = ({n: a.to(dev) for n, a in y.items()} for y in (x, t))
        held.append((d, e))

        def call(d=d, e=e, **kw):
            r = gdn.gdn_decay_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["h0"], d["dhT"],
                                  **({"workspace": ws} if kw else {}))
            o = gdn.gdn_tree_attn(e["parent"], e["q"], e["k"], e["v"], e["kc"], e["vc"], e["table"], e["lens"],
                                  scale=0.09, **({"workspace": tws} if kw else {}))
            return dict(r, o=o)

        plain.append(call())
        call(shared=True)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(shared=True))
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, plain):
        for n in want:
            if want[n] is not None:
                assert torch.equal(out[n], want[n]), n


def test_two_streams_at_once(dev):
    """Calls on two streams with workspaces of their own do not disturb each other."""
    x = decay_tests.make(2, 700, 4, 4, 128, 128, "bf16", seed=51)
    t = tree_tests.make([1500, 700, 3], 16, 8, 2, 128, 64, seed=52)
    want, wo = decay_tests.run(x, dev), tree_tests.run(t, dev, 0.1)
    d, e = ({n: a.to(dev) for n, a in y.items()} for y in (x, t))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            r = gdn.gdn_decay_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["h0"], d["dhT"])
        with torch.cuda.stream(s2):
            o = gdn.gdn_tree_attn(e["parent"], e["q"], e["k"], e["v"], e["kc"], e["vc"], e["table"], e["lens"],
                                  scale=0.1)
        outs.append((r, o))
    torch.cuda.synchronize()
    for r, o in outs:
        assert torch.equal(o, wo)
        for n in r:
            assert torch.equal(r[n], want[n]), n
