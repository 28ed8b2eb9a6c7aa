"""Refusals of gdn_decay_*, gdn_tree_attn / gdn_tree_append and gdn_gated_norm_*:
everything wrong that the host can see is refused before any launch (CPU only)."""
import ctypes

import pytest
import torch

import gated_delta_rule_153_b200 as gdn

INV, UNS, WSP = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32
BIG = 1 << 40


def at(i):
    """Addresses 4 GiB apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) << 32)


def dims(**kw):
    return gdn.gdn_decay_dims(**{**dict(B=1, T=64, H=4, Hk=2, dk=128, dv=128, dtype=BF, scale=1.0), **kw})


def fwd(d, cu=None, nseq=0, ws_bytes=BIG, **kw):
    p = dict(q=at(0), k=at(1), v=at(2), g=at(3), h0=None, o=at(4), hT=None, ws=at(5), **{}) | kw
    return gdn.lib().gdn_decay_fwd(ctypes.byref(d) if d else None, cu, nseq, p["q"], p["k"], p["v"], p["g"], p["h0"],
                                   p["o"], p["hT"], p["ws"], ws_bytes, None)


def bwd(d, cu=None, nseq=0, ws_bytes=BIG, **kw):
    p = dict(q=at(0), k=at(1), v=at(2), g=at(3), h0=None, dO=at(4), dhT=None, dq=at(6), dk=at(7), dv=at(8), dg=at(9),
             dh0=None, ws=at(5)) | kw
    return gdn.lib().gdn_decay_bwd(ctypes.byref(d), cu, nseq, p["q"], p["k"], p["v"], p["g"], p["h0"], p["dO"], p["dhT"],
                                   p["dq"], p["dk"], p["dv"], p["dg"], p["dh0"], p["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INV), (dict(T=0), INV), (dict(H=0), INV), (dict(Hk=0), INV), (dict(Hk=3), INV), (dict(Hk=8), INV),
    (dict(dtype=5), INV), (dict(scale=float("inf")), INV), (dict(B=1 << 16, T=1 << 16), INV),
    (dict(dk=96), UNS), (dict(dv=256), UNS), (dict(dk=0), UNS)])
def test_decay_dims(kw, code):
    d = dims(**kw)
    assert fwd(d) == code and bwd(d) == code
    assert gdn.gdn_decay_fwd_workspace(d) == 0 and gdn.gdn_decay_bwd_workspace(d) == 0


def test_decay_pointers():
    d = dims()
    assert fwd(None) == INV
    for n in ("q", "k", "v", "g", "o"):
        assert fwd(d, **{n: None}) == INV
        assert fwd(d, **{n: ctypes.c_void_p((7 << 32) + 8)}) == INV
    for n in ("q", "k", "v", "g", "dO", "dq", "dk", "dv", "dg"):
        assert bwd(d, **{n: None}) == INV
        assert bwd(d, **{n: ctypes.c_void_p((11 << 32) + 8)}) == INV
    assert bwd(d, h0=at(10)) == INV and bwd(d, dh0=at(10)) == INV
    # outputs over inputs, partly
    inside = ctypes.c_void_p(at(2).value + 256)
    assert fwd(d, o=inside) == INV and fwd(d, hT=at(3)) == INV and fwd(d, h0=at(10), hT=at(10)) == INV
    assert fwd(d, ws=ctypes.c_void_p(at(4).value + 256)) == INV
    assert bwd(d, dq=at(7)) == INV and bwd(d, dv=at(4)) == INV and bwd(d, h0=at(10), dh0=at(10)) == INV
    need = gdn.gdn_decay_bwd_workspace(d)
    assert need > 0
    assert bwd(d, ws_bytes=need - 1) == WSP and bwd(d, ws=None) == WSP
    assert bwd(d, ws=ctypes.c_void_p(at(5).value + 16)) == WSP
    assert fwd(d, ws=None) == WSP and fwd(d, ws_bytes=gdn.gdn_decay_fwd_workspace(d) - 1) == WSP


def test_decay_offsets():
    d = dims()
    assert fwd(d, cu=at(12)) == INV                      # offsets without a count
    assert fwd(d, nseq=2) == INV and fwd(d, nseq=-1) == INV
    assert fwd(dims(B=2), cu=at(12), nseq=2) == INV
    assert fwd(d, cu=ctypes.c_void_p(at(12).value + 2), nseq=2) == INV
    assert gdn.gdn_decay_bwd_workspace(d, 9) > gdn.gdn_decay_bwd_workspace(d, 1) > 0


def test_decay_step():
    def step(N=2, H=4, Hk=2, dk=128, dv=64, dtype=BF, scale=1.0, **kw):
        p = dict(q=at(0), k=at(1), v=at(2), g=at(3), s=at(4), o=at(5)) | kw
        return gdn.lib().gdn_decay_step(N, H, Hk, dk, dv, dtype, scale, p["q"], p["k"], p["v"], p["g"], p["s"], p["o"], None)
    assert step(N=0) == INV and step(Hk=3) == INV and step(dtype=9) == INV and step(scale=float("nan")) == INV
    assert step(dk=48) == UNS and step(dv=7) == UNS
    for n in ("q", "k", "v", "g", "s", "o"):
        assert step(**{n: None}) == INV
    assert step(s=ctypes.c_void_p(at(4).value + 4)) == INV and step(o=at(2)) == INV


def attn(N=2, M=4, Hq=4, Hkv=2, d=64, dtype=BF, scale=1.0, window=0, pages=9, page=16, width=4, ws_bytes=BIG, **kw):
    p = dict(parent=at(0), q=at(1), k=at(2), v=at(3), kc=at(4), vc=at(5), table=at(6), lens=at(7), o=at(8), ws=at(9)) | kw
    return gdn.lib().gdn_tree_attn(N, M, Hq, Hkv, d, dtype, scale, window, p["parent"], p["q"], p["k"], p["v"], pages, page,
                                   width, p["kc"], p["vc"], p["table"], p["lens"], p["o"], p["ws"], ws_bytes, None)


def append(N=2, M=4, Hkv=2, d=64, dtype=BF, pages=9, page=16, width=4, **kw):
    p = dict(parent=at(0), acc=at(1), k=at(2), v=at(3), kc=at(4), vc=at(5), table=at(6), lens=at(7), new=at(8), st=None) | kw
    return gdn.lib().gdn_tree_append(N, M, Hkv, d, dtype, p["parent"], p["acc"], p["k"], p["v"], pages, page, width,
                                     p["kc"], p["vc"], p["table"], p["lens"], p["new"], p["st"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), INV), (dict(M=0), INV), (dict(Hkv=0), INV), (dict(pages=0), INV), (dict(width=0), INV),
    (dict(dtype=4), INV), (dict(pages=1 << 30, page=128), INV), (dict(width=1 << 30, page=128), INV),
    (dict(width=(1 << 24) - 1, page=128), INV),
    (dict(M=65), UNS), (dict(d=96), UNS), (dict(d=256), UNS), (dict(dtype=F32), UNS), (dict(page=48), UNS),
    (dict(page=256), UNS)])
def test_tree_dims(kw, code):
    assert attn(**kw) == code and append(**kw) == code


def test_tree_arguments():
    assert attn(Hq=3) == INV and attn(window=-1) == INV and attn(scale=float("nan")) == INV
    for n in ("parent", "q", "k", "v", "kc", "vc", "table", "lens", "o"):
        assert attn(**{n: None}) == INV
    assert attn(q=ctypes.c_void_p(at(1).value + 8)) == INV and attn(lens=ctypes.c_void_p(at(7).value + 2)) == INV
    assert attn(o=at(1)) == INV and attn(o=ctypes.c_void_p(at(4).value + 64)) == INV
    assert attn(ws=None) == WSP and attn(ws=ctypes.c_void_p(at(9).value + 16)) == WSP and attn(ws_bytes=0) == WSP
    for n in ("parent", "acc", "k", "v", "kc", "vc", "table", "lens", "new"):
        assert append(**{n: None}) == INV
    assert append(kc=ctypes.c_void_p(at(4).value + 8)) == INV and append(kc=at(2)) == INV and append(vc=at(4)) == INV
    assert append(new=ctypes.c_void_p(at(7).value + 4)) == INV


def test_norm_arguments():
    def f(rows=12, H=3, d=64, wh=1, dtype=BF, eps=1e-6, **kw):
        p = dict(x=at(0), z=at(1), w=at(2), y=at(3)) | kw
        return gdn.lib().gdn_gated_norm_fwd(rows, H, d, wh, dtype, 0, eps, p["x"], p["z"], p["w"], p["y"], None)

    def b(rows=12, H=3, d=64, wh=1, dtype=BF, eps=1e-6, ws_bytes=BIG, **kw):
        p = dict(x=at(0), z=at(1), w=at(2), dy=at(3), dx=at(4), dz=at(5), dw=at(6), ws=at(7)) | kw
        return gdn.lib().gdn_gated_norm_bwd(rows, H, d, wh, dtype, 0, eps, p["x"], p["z"], p["w"], p["dy"], p["dx"], p["dz"],
                                            p["dw"], p["ws"], ws_bytes, None)
    for fn in (f, b):
        assert fn(rows=0) == INV and fn(rows=13) == INV and fn(H=0) == INV and fn(wh=2) == INV and fn(dtype=3) == INV
        assert fn(eps=-1.0) == INV and fn(eps=float("nan")) == INV and fn(d=96) == UNS and fn(d=512) == UNS
        assert fn(x=None) == INV and fn(w=None) == INV and fn(z=ctypes.c_void_p(at(1).value + 4)) == INV
    assert f(y=at(0)) == INV and f(y=ctypes.c_void_p(at(1).value + 16)) == INV
    assert b(dx=at(3)) == INV and b(dz=at(4)) == INV and b(dw=at(2)) == INV
    need = gdn.lib().gdn_gated_norm_bwd_workspace(12, 3, 64, BF)
    assert need > 0 and b(ws_bytes=need - 1) == WSP and b(ws=None) == WSP


def test_bindings_refuse_host_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(TypeError):
        gdn.gdn_decay_fwd(x, x, x, g)
    with pytest.raises(TypeError):
        gdn.gdn_decay_bwd(x, x, x, g, x)
    with pytest.raises(TypeError):
        gdn.gdn_decay_step(x[0], x[0], x[0], g[0], torch.zeros(4, 2, 64, 64))
    with pytest.raises(TypeError):
        gdn.gdn_gated_norm_fwd(x, x, torch.ones(64))
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        gdn.gdn_tree_attn(i, x, x, x, x, x, i, i[0, :1])
    with pytest.raises(TypeError):
        gdn.gdn_tree_append(i, i[0, :1], x, x, x, x, i, i[0, :1])
