"""Cases for the operators around the gated delta-rule layer: linear attention
with a decay per head (prompt, training step, single token), attention of a
draft tree over a paged cache with the append of the accepted path, and the
gated output norm.

Each case is a dict of plain values; ``op`` names the operator:

* ``prompt``  gdn_decay_fwd: o and the final state;
* ``train``   gdn_decay_fwd followed by gdn_decay_bwd: outputs and gradients;
* ``step``    gdn_decay_step: one token for every sequence, state in place;
* ``verify``  gdn_tree_attn: every node of a draft tree over a paged cache;
* ``append``  gdn_tree_append: the accepted path's keys and values into the pages;
* ``norm``    gdn_gated_norm_fwd (and gdn_gated_norm_bwd where ``grad``).
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # one prompt of the long-context workload (16 heads, 8192 tokens), continued from a state
        dict(name="prompt long", op="prompt", B=1, T=8192, H=16, Hk=16, dk=128, dv=128, dtype="bf16",
             nseq=0, shift=-3.0, state=True),
        # requests of different lengths packed in one row, key heads shared, single precision
        dict(name="prompt packed f32", op="prompt", B=1, T=2051, H=6, Hk=2, dk=64, dv=64, dtype="f32",
             nseq=7, shift=-1.0, state=False),
        # the training step of the 350M-scale layer
        dict(name="train 350m", op="train", B=8, T=2048, H=8, Hk=8, dk=128, dv=128, dtype="bf16",
             nseq=0, shift=2.0, state=False),
        # ragged documents packed for training, four value heads to a key head, slow decay
        dict(name="train packed", op="train", B=1, T=3001, H=8, Hk=2, dk=128, dv=64, dtype="bf16",
             nseq=9, shift=-4.0, state=True),
        # the decode workload: 256 sequences of 16 heads
        dict(name="step 256", op="step", N=256, H=16, Hk=16, dk=128, dv=128, dtype="bf16", shift=0.0),
        # a few streams, where latency counts
        dict(name="step 3", op="step", N=3, H=4, Hk=2, dk=64, dv=128, dtype="f32", shift=-2.0),
        # 32 sequences, a 32-node draft tree each, caches of up to 8192 tokens
        dict(name="verify 32", op="verify", N=32, M=32, Hq=16, Hkv=4, d=128, ctx=8192, page=64, window=0,
             tree="kary"),
        # plain decoding of three short requests: one node, sliding window
        dict(name="verify single", op="verify", N=3, M=1, Hq=8, Hkv=8, d=64, ctx=777, page=16, window=512,
             tree="chain"),
        # commit of the accepted paths of a full batch
        dict(name="append 256", op="append", N=256, M=32, Hkv=4, d=128, page=64, tree="random"),
        # commit of a drafted chain
        dict(name="append 5", op="append", N=5, M=7, Hkv=2, d=64, page=16, tree="chain"),
        # the layer's output norm and gate in a training step of the 350M-scale layer
        dict(name="norm 350m", op="norm", B=8, T=2048, H=8, d=128, dtype="bf16", center=False, shared=True,
             grad=True),
        # the same epilogue for a few decoded tokens, group norm, single precision
        dict(name="norm decode", op="norm", B=37, T=1, H=6, d=64, dtype="f32", center=True, shared=False,
             grad=False),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "step", "verify", "append", "norm"])
    if op in ("prompt", "train"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        if dtype == "f32":
            dk, dv = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 1, 2, 4])
        nseq = rng.choice([0, 0, rng.randint(1, 12)])
        B = 1 if nseq else _log(rng, 1, 8)
        most = 131072 if dtype == "bf16" else 24576
        T = _log(rng, 1, max(1, min(8192, most // (B * H))))
        return dict(op=op, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, nseq=nseq,
                    shift=round(rng.uniform(-4.0, 2.0), 2), state=rng.random() < 0.5)
    if op == "step":
        Hk = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log(rng, 1, 256), H=Hk * rng.choice([1, 2]), Hk=Hk,
                    dk=rng.choice([16, 32, 64, 128]), dv=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "f32"]), shift=round(rng.uniform(-4.0, 2.0), 2))
    if op == "verify":
        Hkv, M = rng.choice([1, 2, 4, 8]), rng.randint(1, 64)
        ctx = _log(rng, 1, 8192)
        N = _log(rng, 1, max(1, min(64, (32 * 8192 * 4) // (ctx * Hkv))))
        G = rng.choice([1, 2, 4, 8])
        if N * M * G > 4096:
            M = max(1, 4096 // (N * G))
        return dict(op=op, N=N, M=M, Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), ctx=ctx,
                    page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    tree=rng.choice(["kary", "random", "chain"]))
    if op == "append":
        return dict(op=op, N=_log(rng, 1, 256), M=rng.randint(1, 64), Hkv=rng.choice([1, 2, 4]),
                    d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    tree=rng.choice(["kary", "random", "chain"]))
    B, H = _log(rng, 1, 16), rng.randint(1, 16)
    return dict(op=op, B=B, T=_log(rng, 1, max(1, 131072 // (B * H))), H=H, d=rng.choice([32, 64, 128]),
                dtype=rng.choice(["bf16", "f32"]), center=rng.random() < 0.5, shared=rng.random() < 0.5,
                grad=rng.random() < 0.7)


# ---- inputs ------------------------------------------------------------------
def _lens(case):
    """Lengths of the packed sequences (one of them empty when there are three or more)."""
    r = random.Random(case["T"] * 31 + case["nseq"])
    n, T = case["nseq"], case["T"]
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    if n >= 3:
        cuts[1] = cuts[0]
    cuts = [0] + sorted(cuts) + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _ctx(case):
    """Cached tokens of each sequence: between a third of ctx and ctx, one of them the full length."""
    r = random.Random(case["ctx"] * 17 + case["N"])
    return [case["ctx"]] + [r.randint(case["ctx"] // 3, case["ctx"]) for _ in range(case["N"] - 1)]


def _parents(case, gen):
    N, M = case["N"], case["M"]
    i = torch.arange(M, device="cuda")
    if case["tree"] == "chain":
        p = i - 1
    elif case["tree"] == "kary":
        p = torch.div(i - 1, 4, rounding_mode="floor")
    else:
        u = torch.rand(N, M, generator=gen, device="cuda")
        return (torch.floor(u * (i + 1)).long().clamp(max=M - 1).minimum(i) - 1).to(torch.int32)
    return p.to(torch.int32).expand(N, M).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = _DT[case.get("dtype", "bf16")]

    def rn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def unit(*shape):
        x = rn(*shape)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)).to(dt)

    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op in ("prompt", "train"):
        B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
        s.update(q=unit(B, T, Hk, dk), k=unit(B, T, Hk, dk), v=rn(B, T, H, dv).to(dt),
                 g=-torch.nn.functional.softplus(rn(B, T, H) + case["shift"]), scale=dk ** -0.5,
                 cu=None, lmax=T)
        ns = B
        if case["nseq"]:
            lens = _lens(case)
            ns = len(lens)
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(ns + 1)], dtype=torch.int32, device="cuda")
            s["lmax"] = max(lens)
        s["h0"] = rn(ns, H, dv, dk) * 0.1 if case["state"] else None
        if op == "train":
            s["dO"] = rn(B, T, H, dv).to(dt)
            s["dhT"] = rn(ns, H, dv, dk) * 0.3 if case["state"] else None
    elif op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        s.update(q=unit(N, Hk, dk), k=unit(N, Hk, dk), v=rn(N, H, dv).to(dt),
                 g=-torch.nn.functional.softplus(rn(N, H) + case["shift"]), scale=dk ** -0.5,
                 S=rn(N, H, dv, dk) * 0.3)
    elif op in ("verify", "append"):
        N, M, Hkv, d, page = (case[n] for n in ("N", "M", "Hkv", "d", "page"))
        s["parent"] = _parents(case, gen)
        s["k"], s["v"] = rn(N, M, Hkv, d).to(dt), rn(N, M, Hkv, d).to(dt)
        if op == "verify":
            lens = _ctx(case)
            s["q"] = (rn(N, M, case["Hq"], d) * 1.5).to(dt)
        else:
            r = random.Random(N)
            lens = [r.randint(0, 2 * page) for _ in range(N)]
            s["accepted"] = (torch.floor(torch.rand(N, generator=gen, device="cuda") * (M + 1)).int() - 1).clamp(max=M - 1)
        most = max(lens) + M
        width = -(-most // page)
        used = [-(-(n + M) // page) for n in lens]
        pages = torch.randperm(sum(used) + 3, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((N, width), -1, dtype=torch.int32)
        host, at = pages.cpu(), 0
        for n, u in enumerate(used):
            table[n, :u] = host[at:at + u]
            at += u
        s["table"] = table.cuda()
        s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["kc"] = rn(sum(used) + 3, page, Hkv, d).to(dt)
        s["vc"] = rn(sum(used) + 3, page, Hkv, d).to(dt)
        s["scale"], s["most"] = d ** -0.5, max(lens)
    else:
        B, T, H, d = (case[n] for n in ("B", "T", "H", "d"))
        s.update(x=(rn(B, T, H, d) * 2 + 0.3).to(dt), z=rn(B, T, H, d).to(dt),
                 w=1 + 0.2 * (rn(d) if case["shared"] else rn(H, d)), eps=1e-6)
        if case["grad"]:
            s["dy"] = rn(B, T, H, d).to(dt)
    return s


# ---- the framework's calls -----------------------------------------------------
def _run_own(s):
    import gated_delta_rule_153_b200 as gdn
    op = s["op"]
    if op == "prompt":
        return list(gdn.gdn_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], cu_seqlens=s["cu"],
                                      scale=s["scale"]))
    if op == "train":
        o, hT = gdn.gdn_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], cu_seqlens=s["cu"],
                                  scale=s["scale"])
        r = gdn.gdn_decay_bwd(s["q"], s["k"], s["v"], s["g"], s["dO"], s["h0"], s["dhT"],
                              cu_seqlens=s["cu"], scale=s["scale"])
        return [o, hT, r["dq"], r["dk"], r["dv"], r["dg"], r["dh0"]]
    if op == "step":
        o = gdn.gdn_decay_step(s["q"], s["k"], s["v"], s["g"], s["S"], scale=s["scale"])
        return [o, s["S"]]
    if op == "verify":
        return gdn.gdn_tree_attn(s["parent"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["len"],
                                 scale=s["scale"], window=s["case"]["window"])
    if op == "append":
        n = gdn.gdn_tree_append(s["parent"], s["accepted"], s["k"], s["v"], s["kc"], s["vc"], s["table"],
                                s["len"])
        return [n, s["kc"], s["vc"]]
    c = s["case"]["center"]
    y = gdn.gdn_gated_norm_fwd(s["x"], s["z"], s["w"], eps=s["eps"], center=c)
    if "dy" not in s:
        return y
    return [y, *gdn.gdn_gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], eps=s["eps"], center=c)]


# ---- plain forms ---------------------------------------------------------------
_C = 64  # tokens per chunk of the plain form


def _rows(s):
    """Token index [sequences, longest] of a packed row, and which of them exist."""
    at = s["cu"][:-1, None].long() + torch.arange(s["lmax"], device="cuda")
    ok = at < s["cu"][1:, None]
    return at.clamp(max=max(s["q"].shape[1] - 1, 0)), ok


def _chunked(x, n):
    """[B, T, H, d] -> [B, H, chunks, C, d] in fp32, zero past T."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * _C - x.shape[1]))
    return x.reshape(x.shape[0], n, _C, *x.shape[2:]).permute(0, 3, 1, 2, 4)


def _decay(s, grad):
    q, k, v, g = s["q"], s["k"], s["v"], s["g"]
    dO = s["dO"] if grad else None
    if s["cu"] is not None:
        at, ok = _rows(s)

        def pick(x):
            return x[0][at] * ok.reshape(*ok.shape, *([1] * (x.dim() - 2)))

        q, k, v, g = pick(q), pick(k), pick(v), pick(g)
        dO = pick(dO) if grad else None
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    n = max(1, -(-T // _C))
    rep = H // Hk
    scale = s["scale"]
    Q, K = _chunked(q, n).repeat_interleave(rep, 1), _chunked(k, n).repeat_interleave(rep, 1)
    V = _chunked(v, n)
    G = _chunked64(g, n).cumsum(-1)                                    # [B, H, n, C]
    last = G[..., -1:]
    keep = torch.ones(_C, _C, dtype=torch.bool, device="cuda").tril()
    D = torch.where(keep, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    P = scale * (Q @ K.transpose(-1, -2)) * D
    up, down = (last - G).float().exp()[..., None], G.float().exp()[..., None]
    # states: entering chunk c = sum over earlier chunks of their own sums, decayed
    N = V.transpose(-1, -2) @ (K * up)                                 # [B, H, n, dv, dk]
    E = torch.nn.functional.pad(last[..., 0].cumsum(-1), (1, 0))       # [B, H, n + 1]
    before = torch.ones(n + 1, n, dtype=torch.bool, device="cuda").tril(-1)
    W = torch.where(before, E[..., :, None] - E[..., None, 1:], -math.inf).float().exp()
    S = (W @ N.flatten(-2)).reshape(B, H, n + 1, dv, dk)
    if s["h0"] is not None:
        S = S + E.float().exp()[..., None, None] * s["h0"][:, :, None]
    S0, hT = S[:, :, :-1], S[:, :, -1]
    o = P @ V + scale * down * (Q @ S0.transpose(-1, -2))

    def back(x, like):                                                 # [B, H, n, C, d] -> like's rows
        x = x.permute(0, 2, 3, 1, 4).reshape(B, n * _C, x.shape[1], -1)[:, :T]
        if s["cu"] is not None:
            x = x[ok][None]
        return x.to(like.dtype)

    out = [back(o, s["v"]), hT]
    if not grad:
        return out
    Y = _chunked(dO, n)
    YV = Y @ V.transpose(-1, -2)
    A = scale * YV * D
    R = Y.transpose(-1, -2) @ (Q * (scale * down))
    after = torch.ones(n + 1, n, dtype=torch.bool, device="cuda").triu()
    W = torch.where(after, E[..., None, :-1] - E[..., :, None], -math.inf).float().exp()
    dS = (W @ R.flatten(-2)).reshape(B, H, n + 1, dv, dk)
    if s["dhT"] is not None:
        dS = dS + (E[..., -1:] - E).float().exp()[..., None, None] * s["dhT"][:, :, None]
    dh0, dS = dS[:, :, 0], dS[:, :, 1:]
    dq_s, dk_s = scale * down * (Y @ S0), up * (V @ dS)
    dq, dkk = A @ K + dq_s, A.transpose(-1, -2) @ Q + dk_s
    dvv = P.transpose(-1, -2) @ Y + up * (K @ dS.transpose(-1, -2))
    M = (P * YV).double().tril(-1)
    x = M.sum(-1) - M.sum(-2) + (Q * dq_s).double().sum(-1)
    b = (K * dk_s).double().sum(-1)
    cross = last[..., 0].exp() * (S0 * dS).double().sum((-1, -2))
    dg = x.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + cross[..., None]

    def shared(x):                                                     # gradients of shared key heads
        return x.reshape(B, Hk, rep, *x.shape[2:]).sum(2)

    dg = back(dg[..., None], s["g"])[..., 0]
    return out + [back(shared(dq), s["q"]), back(shared(dkk), s["k"]), back(dvv, s["v"]), dg,
                  dh0 if s["h0"] is not None else None]


def _chunked64(g, n):
    g = torch.nn.functional.pad(g.double(), (0, 0, 0, n * _C - g.shape[1]))
    return g.reshape(g.shape[0], n, _C, -1).permute(0, 3, 1, 2)


def _step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    S = s["S"]
    S.mul_(s["g"].exp()[..., None, None]).add_(s["v"].float()[..., :, None] * k[..., None, :])
    o = (S * (s["scale"] * q)[..., None, :]).sum(-1)
    return [o.to(s["q"].dtype), S]


def _ancestors(parent):
    """[N, M, M]: whether j is i or an ancestor of i; and the depth of each node."""
    N, M = parent.shape
    j = torch.arange(M, device="cuda")
    A = ((parent[..., None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, M - 1).bit_length()):
        A = ((A @ A) > 0).float()
    return A > 0, A.sum(-1).long() - 1


def _verify(s):
    q, M = s["q"].float(), s["q"].shape[1]
    rep = q.shape[2] // s["k"].shape[2]
    L = s["most"]
    table = s["table"].long().clamp(min=0)
    anc, depth = _ancestors(s["parent"])
    win = s["case"]["window"] or (1 << 30)

    def keys(cache, nodes):                                            # [N, Hkv, L + M, d]
        x = cache[table].flatten(1, 2)[:, :L]
        return torch.cat([x, nodes], 1).float().permute(0, 2, 1, 3)

    K, V = keys(s["kc"], s["k"]), keys(s["vc"], s["v"])
    n = s["len"].long()[:, None, None]
    p = torch.arange(L, device="cuda")
    back = n + depth[:, :, None] - p
    seen = torch.cat([(p < n) & (back < win), anc & (depth[:, :, None] - depth[:, None, :] < win)], -1)
    Q = q.unflatten(2, (-1, rep)).permute(0, 2, 3, 1, 4)               # [N, Hkv, rep, M, d]
    x = s["scale"] * (Q.flatten(2, 3) @ K.transpose(-1, -2)).unflatten(2, (rep, M))
    x = torch.where(seen[:, None, None], x, -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    o = (x.flatten(2, 3) @ V).unflatten(2, (rep, M)) / x.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype)


def _append(s):
    page, M = s["kc"].shape[1], s["k"].shape[1]
    anc, depth = _ancestors(s["parent"])
    acc = s["accepted"].long()
    row = anc[torch.arange(len(acc), device="cuda"), acc.clamp(min=0)] & (acc >= 0)[:, None]   # nodes on the path
    n, i = row.nonzero(as_tuple=True)
    at = s["len"].long()[n] + depth[n, i]
    where = s["table"].long()[n, at // page]
    s["kc"][where, at % page] = s["k"][n, i]
    s["vc"][where, at % page] = s["v"][n, i]
    return [s["len"] + row.sum(-1).int(), s["kc"], s["vc"]]


def _norm(s):
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    xc = x - x.mean(-1, keepdim=True) if s["case"]["center"] else x
    r = (xc * xc).mean(-1, keepdim=True).add(s["eps"]).rsqrt()
    h, sg = xc * r, 1 / (1 + (-z).exp())
    act = z * sg
    y = (w * h * act).to(s["x"].dtype)
    if "dy" not in s:
        return y
    dy = s["dy"].float()
    dh = dy * w * act
    dx = dh - h * (dh * h).mean(-1, keepdim=True)
    if s["case"]["center"]:
        dx = dx - dh.mean(-1, keepdim=True)
    dx = dx * r
    dz = dy * w * h * sg * (1 + z * (1 - sg))
    dw = (dy * h * act).double().sum((0, 1, 2) if w.dim() == 1 else (0, 1)).float()
    return [y, dx.to(s["x"].dtype), dz.to(s["z"].dtype), dw]


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "prompt":
        return _decay(state, False)
    if op == "train":
        return _decay(state, True)
    return {"step": _step, "verify": _verify, "append": _append, "norm": _norm}[op](state)


# ---- what a pass cannot do without -----------------------------------------------
def work(case):
    op = case["op"]
    e = 4 if case.get("dtype", "bf16") == "f32" else 2
    if op in ("prompt", "train"):
        B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
        tok, ns = B * T, (case["nseq"] or B)
        qk, v, g, st = tok * Hk * dk * e, tok * H * dv * e, tok * H * 4, ns * H * dk * dv * 4
        h0 = st if case["state"] else 0
        fwd = 2 * qk + 2 * v + g + st + h0
        pairs = tok * H * dk * dv
        if op == "prompt":
            return {"bytes": fwd, "flops": 4 * pairs}
        bwd = 4 * qk + 3 * v + 2 * g + 3 * h0
        return {"bytes": fwd + bwd, "flops": 14 * pairs}
    if op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        return {"bytes": N * (8 * H * dk * dv + 2 * Hk * dk * e + 2 * H * dv * e + 4 * H),
                "flops": 5 * N * H * dk * dv}
    if op == "verify":
        N, M, Hq, Hkv, d = (case[n] for n in ("N", "M", "Hq", "Hkv", "d"))
        win = case["window"] or (1 << 30)
        seen = sum(min(n, win) for n in _ctx(case))
        return {"bytes": 4 * d * (Hkv * (seen + N * M) + Hq * N * M) + 4 * N * (M + 1 + -(-case["ctx"] // case["page"])),
                "flops": 4 * d * Hq * M * (seen + N * M / 2)}
    if op == "append":
        N, M, Hkv, d = (case[n] for n in ("N", "M", "Hkv", "d"))
        depth = (M + 1) / 2 if case["tree"] == "chain" else math.log(M + 1, 4) if case["tree"] == "kary" else math.log(M + 1) + 0.5
        return {"bytes": N * depth * M / (M + 1) * Hkv * d * 8 + 4 * N * (M + 3), "flops": 0}
    n = case["B"] * case["T"] * case["H"] * case["d"]
    return {"bytes": n * e * (8 if case["grad"] else 3), "flops": n * (30 if case["grad"] else 10)}


# ---- 64-bit values, from the definitions -------------------------------------------
def _exact_decay(case, s):
    """Token pair by token pair, one sequence and head at a time; gradients by autograd."""
    B, T, H, Hk, dk, dv = (case[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
    grad = case["op"] == "train"
    spans = [(b, 0, T) for b in range(B)]
    if s["cu"] is not None:
        cu = s["cu"].tolist()
        spans = [(0, a, b) for a, b in zip(cu, cu[1:])]
    f = lambda x: None if x is None else x.double()  # noqa: E731
    q, k, v, g, h0 = (f(s[n]) for n in ("q", "k", "v", "g", "h0"))
    o, hT = torch.zeros_like(v), torch.zeros(len(spans), H, dv, dk, dtype=torch.float64, device="cuda")
    gr = {n: torch.zeros_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("g", g), ("h", h0)) if x is not None}
    for i, (b, lo, hi) in enumerate(spans):
        for h in range(H):
            kh = h // (H // Hk)
            leaf = [q[b, lo:hi, kh].clone(), k[b, lo:hi, kh].clone(), v[b, lo:hi, h].clone(), g[b, lo:hi, h].clone(),
                    h0[i, h].clone() if h0 is not None else torch.zeros(dv, dk, dtype=torch.float64, device="cuda")]
            if grad:
                for x in leaf:
                    x.requires_grad_(True)
            Q, K, V, gg, S = leaf
            total = torch.cumsum(gg, 0)
            decay = (total[:, None] - total[None, :]).masked_fill(
                ~torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").tril(), -math.inf).exp()
            oh = s["scale"] * (((Q @ K.T) * decay) @ V + total.exp()[:, None] * (Q @ S.T))
            if hi > lo:
                end = total[-1].exp() * S + V.T @ ((total[-1] - total).exp()[:, None] * K)
            else:
                end = S * 1.0
            o[b, lo:hi, h], hT[i, h] = oh.detach(), end.detach()
            if grad:
                loss = (oh * s["dO"][b, lo:hi, h].double()).sum()
                if s["dhT"] is not None:
                    loss = loss + (end * s["dhT"][i, h].double()).sum()
                d = torch.autograd.grad(loss, leaf, allow_unused=True)
                for n, x, at in (("q", d[0], (b, slice(lo, hi), kh)), ("k", d[1], (b, slice(lo, hi), kh)),
                                 ("v", d[2], (b, slice(lo, hi), h)), ("g", d[3], (b, slice(lo, hi), h)), ("h", d[4], (i, h))):
                    if x is not None and n in gr:
                        gr[n][at] += x
    out = [o, hT]
    return out + [gr["q"], gr["k"], gr["v"], gr["g"], gr.get("h")] if grad else out


def _exact_verify(case, s):
    N, M, Hq, Hkv, d, page = (case[n] for n in ("N", "M", "Hq", "Hkv", "d", "page"))
    rep, win = Hq // Hkv, case["window"] or (1 << 30)
    out = torch.zeros(N, M, Hq, d, dtype=torch.float64, device="cuda")
    parents, lens, table = s["parent"].tolist(), s["len"].tolist(), s["table"].long()
    for n in range(N):
        L = lens[n]
        rows = [[] for _ in range(M)]
        for i in range(M):
            up = parents[n][i]
            rows[i] = (rows[up] if up >= 0 else []) + [i]
        pg = table[n, :-(-L // page)]
        K = torch.cat([s["kc"][pg].flatten(0, 1)[:L], s["k"][n]]).double()
        V = torch.cat([s["vc"][pg].flatten(0, 1)[:L], s["v"][n]]).double()
        bias = torch.full((M, L + M), -math.inf, dtype=torch.float64)
        for i, path in enumerate(rows):
            at = L + len(path) - 1
            bias[i, max(0, at - win + 1):L] = 0
            bias[i, [L + j for j in path[-win:]]] = 0
        bias = bias.cuda()
        for h in range(Hq):
            x = s["q"][n, :, h].double() @ K[:, h // rep].T * s["scale"] + bias
            out[n, :, h] = torch.softmax(x, -1) @ V[:, h // rep]
    return out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("prompt", "train"):
        return _exact_decay(case, s)
    if op == "step":
        rep = case["H"] // case["Hk"]
        head = [h // rep for h in range(case["H"])]
        a = torch.exp(s["g"].double())
        S = torch.einsum("nh,nhvk->nhvk", a, s["S"].double()) + torch.einsum(
            "nhv,nhk->nhvk", s["v"].double(), s["k"].double()[:, head])
        return [torch.einsum("nhvk,nhk->nhv", S, s["q"].double()[:, head]) * s["scale"], S]
    if op == "verify":
        return _exact_verify(case, s)
    if op == "append":
        kc, vc, lens, page = s["kc"].double(), s["vc"].double(), s["len"].tolist(), case["page"]
        for n in range(case["N"]):
            path, j = [], int(s["accepted"][n])
            par, tab = s["parent"][n].tolist(), s["table"][n].tolist()
            while j >= 0:
                path.insert(0, j)
                j = par[j]
            for t, j in enumerate(path):
                p = lens[n] + t
                kc[tab[p // page], p % page] = s["k"][n, j].double()
                vc[tab[p // page], p % page] = s["v"][n, j].double()
            lens[n] += len(path)
        return [torch.tensor(lens, dtype=torch.int32, device="cuda"), kc, vc]
    x, z, w = (s[n].double().requires_grad_(True) for n in ("x", "z", "w"))
    c = x - x.mean(-1, keepdim=True) if case["center"] else x
    y = w * (c / torch.sqrt(c.pow(2).mean(-1, keepdim=True) + s["eps"])) * torch.nn.functional.silu(z)
    if not case["grad"]:
        return y.detach()
    return [y.detach(), *torch.autograd.grad(y, (x, z, w), s["dy"].double())]
