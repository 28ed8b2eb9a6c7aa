"""Draft-tree attention over a paged cache and the append of an accepted path,
row by row in fp64 / by plain indexing."""
from __future__ import annotations

import torch


def path_of(parent, i):
    """Root path of node i, root first (parent: a list)."""
    path = []
    while i >= 0:
        path.insert(0, i)
        i = parent[i]
    return path


def attend(parent, q, k, v, k_cache, v_cache, table, lens, scale=1.0, window=0):
    """(o, the softmax-weighted sum of |v|) for q [N,M,Hq,d]."""
    N, M, Hq, d = q.shape
    Hkv, page = k.shape[2], k_cache.shape[1]
    o = torch.zeros(N, M, Hq, d, dtype=torch.float64)
    mag = torch.zeros_like(o)
    for n in range(N):
        par, L = parent[n].tolist(), int(lens[n])
        at = [(int(table[n, p // page]), p % page) for p in range(L)]
        for i in range(M):
            path = path_of(par, i)
            pos = L + len(path) - 1
            lo = max(0, pos - window + 1) if window else 0
            rows_k = [k_cache[g, r] for g, r in at[lo:]] + [k[n, j] for t, j in enumerate(path) if L + t >= lo]
            rows_v = [v_cache[g, r] for g, r in at[lo:]] + [v[n, j] for t, j in enumerate(path) if L + t >= lo]
            K, V = torch.stack(rows_k).double(), torch.stack(rows_v).double()   # [keys, Hkv, d]
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                s = scale * (K[:, kh] @ q[n, i, h].double())
                p = torch.exp(s - s.max())
                p = p / p.sum()
                o[n, i, h] = p @ V[:, kh]
                mag[n, i, h] = p @ V[:, kh].abs()
    return o, mag


def append(parent, accepted, k, v, k_cache, v_cache, table, lens):
    """New caches and lengths."""
    kc, vc, new, page = k_cache.clone(), v_cache.clone(), lens.clone(), k_cache.shape[1]
    for n in range(k.shape[0]):
        path = path_of(parent[n].tolist(), int(accepted[n]))
        for t, j in enumerate(path):
            p = int(lens[n]) + t
            kc[int(table[n, p // page]), p % page] = k[n, j]
            vc[int(table[n, p // page]), p % page] = v[n, j]
        new[n] += len(path)
    return kc, vc, new
