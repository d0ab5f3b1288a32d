"""Host-side refusals of the feature stage (no GPU: every call here returns
before it enqueues anything) and its workspace sizes."""
import pytest

from sparse_output_layer_amd import haste as H

INV, UNS, WS = H.HASTE_ERR_INVALID, H.HASTE_ERR_UNSUPPORTED, H.HASTE_ERR_WORKSPACE
A, B_, C, D_, E, F_, G, H_, I_ = (i << 28 for i in range(1, 10))    # far apart


@pytest.fixture(scope="module")
def L():
    return H.lib()


def emb(**kw):
    d = dict(B=4, n=9, V=50, D=8, e_dtype=1, y_dtype=0, g_dtype=0, scale=1.0)
    d.update(kw)
    return H.EmbedDesc(**d)


def test_embed_refusals(L):
    def fwd(d=emb(), rp=A, t=B_, w=C, e=D_, y=E, ws=None, n=0):
        return L.haste_embed_fwd(d, rp, t, w, e, y, ws, n, None)
    assert fwd(None) == INV
    bad = (dict(B=0), dict(n=-1), dict(V=0), dict(D=0), dict(D=-3), dict(e_dtype=2), dict(y_dtype=-1), dict(g_dtype=7))
    for kw in bad:
        assert fwd(emb(**kw)) == INV, kw
        assert L.haste_embed_fwd_workspace_bytes(emb(**kw), 1) == 0 and L.haste_embed_bwd_workspace_bytes(emb(**kw)) == 0
    assert fwd(emb(D=(1 << 20) + 1)) == UNS
    assert fwd(rp=None) == INV                      # a token a row needs n = B
    assert fwd(t=None) == INV and fwd(e=None) == INV and fwd(y=None) == INV
    assert fwd(rp=A + 2) == INV and fwd(t=B_ + 1) == INV and fwd(w=C + 3) == INV and fwd(e=D_ + 1) == INV and fwd(y=E + 2) == INV
    assert fwd(y=D_ + 16) == INV and fwd(y=A) == INV and fwd(y=B_ + 32) == INV and fwd(y=C) == INV
    big = emb(n=5000)
    need = L.haste_embed_fwd_workspace_bytes(big, 1)
    assert need > 0 and L.haste_embed_fwd_workspace_bytes(big, 0) == 0 and L.haste_embed_fwd_workspace_bytes(emb(), 1) == 0
    assert fwd(big) == WS and fwd(big, ws=F_, n=need - 1) == WS and fwd(big, ws=F_ + 64, n=need) == WS
    assert fwd(big, ws=D_ - 256, n=need) == INV     # over the table

    def bwd(d=emb(), rp=A, t=B_, w=C, e=D_, dy=E, de=F_, acc=0, dw=None, ws=G, n=1 << 27):
        return L.haste_embed_bwd(d, rp, t, w, e, dy, de, acc, dw, ws, n, None)
    assert bwd(None) == INV and bwd(de=None) == INV and bwd(dy=None) == INV and bwd(de=F_ + 2) == INV
    assert bwd(e=None, dw=F_ + 65536) == INV and bwd(dw=F_ + 65537) == INV
    assert bwd(de=E) == INV and bwd(de=D_, dw=F_) == INV and bwd(dw=F_ + 16) == INV and bwd(dw=C) == INV
    assert bwd(ws=None) == WS and bwd(n=16) == WS and bwd(ws=G + 32) == WS and bwd(ws=E & ~255) == INV
    assert bwd(emb(D=1 << 21)) == UNS
    assert L.haste_embed_bwd_workspace_bytes(emb(n=0)) == 0 < L.haste_embed_bwd_workspace_bytes(emb())


def test_embed_entry_limit(L):
    """More entries than one launch has threads for, in bags and for dE."""
    d = emb(n=(1 << 28) + 1)
    assert L.haste_embed_fwd(d, A, 1 << 40, None, 1 << 41, 1 << 42, 1 << 43, 1 << 40, None) == UNS
    assert L.haste_embed_bwd(d, A, 1 << 40, None, 1 << 41, 1 << 42, 1 << 43, 0, None, 1 << 44, 1 << 40, None) == UNS
    # many rows take the way with a workspace, however few the entries
    assert L.haste_embed_fwd_workspace_bytes(emb(B=1 << 20, n=9), 1) == 0 < L.haste_embed_fwd_workspace_bytes(emb(B=(1 << 20) + 1, n=9), 1)


def adn(**kw):
    d = dict(B=4, D=8, o_dtype=1, r_dtype=0, y_dtype=0, w_dtype=0, flags=0, eps=1e-5, alpha=1.0, reserved0=0)
    d.update(kw)
    return H.AddNormDesc(**d)


def test_addnorm_refusals(L):
    W = H.AddNormPointers

    def fwd(d=adn(), o=A, r=B_, w=None, dr=None, ro=C, y=D_, st=E):
        return L.haste_addnorm_fwd(d, o, r, w, dr, ro, y, st, None)
    assert fwd(None) == INV
    bad = (dict(B=0), dict(D=0), dict(o_dtype=2), dict(r_dtype=-1), dict(y_dtype=5), dict(w_dtype=3), dict(flags=4), dict(eps=-1.0),
           dict(eps=float("nan")), dict(reserved0=1))
    for kw in bad:
        assert fwd(adn(**kw)) == INV, kw
        assert L.haste_addnorm_bwd_workspace_bytes(adn(**kw)) == 0
    assert fwd(o=None) == INV and fwd(r=None) == INV and fwd(ro=None) == INV
    assert fwd(o=A + 1) == INV and fwd(r=B_ + 2) == INV and fwd(ro=C + 2) == INV and fwd(y=D_ + 1) == INV and fwd(st=E + 2) == INV
    assert fwd(ro=A) == INV and fwd(ro=B_ + 4) == INV and fwd(y=C + 64) == INV and fwd(y=B_) == INV and fwd(st=D_ + 16) == INV
    assert fwd(w=W(None, F_, None, None, None)) == INV                  # post weights without the flag
    assert fwd(y=None, w=W(None, None, None, F_, None)) == INV          # weights of a norm that is not there
    assert fwd(adn(flags=2)) == INV                                     # no gate's rows
    assert fwd(w=W(F_ + 1, None, None, None, None)) == INV and fwd(w=W(C, None, None, None, None)) == INV
    assert fwd(dr=H.DropoutStruct(2.0, 0, 0, 0)) == INV

    def bwd(d=adn(), o=A, ro=B_, w=None, st=C, dy=D_, dro=E, drp=None, dr=F_, do=G, g=None, ws=None, n=0):
        return L.haste_addnorm_bwd(d, o, ro, w, st, dy, dro, drp, dr, do, g, 0, ws, n, None)
    assert bwd(dy=None, dro=None) == INV and bwd(ro=None) == INV and bwd(st=None) == INV and bwd(adn(flags=1), dy=None, st=None) == INV
    assert bwd(o=None) == INV and bwd(dr=None) == INV and bwd(do=None) == INV and bwd(dr=A) == INV and bwd(do=E) == INV and bwd(dr=E + 4) == INV
    assert bwd(g=W(None, H_, None, None, None)) == INV and bwd(dy=None, g=W(None, None, None, H_, None)) == INV
    assert bwd(g=W(H_ + 1, None, None, None, None)) == INV and bwd(g=W(D_, None, None, None, None), ws=I_, n=1 << 20) == INV
    need = L.haste_addnorm_bwd_workspace_bytes(adn())
    gr = W(None, None, None, H_, H_ + 64)
    assert need >= 4 * 8 * 4 and bwd(g=gr) == WS and bwd(g=gr, ws=I_, n=need - 1) == WS and bwd(g=gr, ws=I_ + 8, n=need) == WS
    assert bwd(g=gr, ws=G, n=need) == INV and bwd(g=W(None, None, None, H_, H_ + 16), ws=I_, n=need) == INV


def lin(**kw):
    d = dict(M=40, K=64, N=32, x_dtype=1, y_dtype=0, b_dtype=0, act=2, reserved0=0, ld_x=0, ld_dx=0)
    d.update(kw)
    return H.LinearDesc(**d)


def test_linear_refusals(L):
    def fwd(d=lin(), x=A, W=B_, b=C, r=D_, y=E, z=F_, ws=None, n=0):
        return L.haste_linear_fwd(d, x, W, b, r, y, z, ws, n, None)
    assert fwd(None) == INV
    for kw in (dict(M=0), dict(K=0), dict(N=0), dict(x_dtype=2), dict(y_dtype=-1), dict(b_dtype=3), dict(act=4), dict(act=-1),
               dict(reserved0=1), dict(ld_x=63), dict(ld_dx=63)):
        assert fwd(lin(**kw)) == INV, kw
        assert L.haste_linear_fwd_workspace_bytes(lin(**kw), A, B_) == 0 == L.haste_linear_bwd_workspace_bytes(lin(**kw), A, B_, C)
    for kw in (dict(K=(1 << 22) + 1), dict(N=(1 << 22) + 1), dict(ld_x=(1 << 22) + 1), dict(x_dtype=0, y_dtype=1)):
        assert fwd(lin(**kw)) == UNS, kw
    assert fwd(x=None) == INV and fwd(W=None) == INV and fwd(y=None) == INV
    assert fwd(x=A + 1) == INV and fwd(W=B_ + 1) == INV and fwd(b=C + 2) == INV and fwd(r=D_ + 2) == INV and fwd(y=E + 1) == INV and fwd(z=F_ + 2) == INV
    assert fwd(lin(act=0)) == INV                                   # z without an activation
    assert fwd(y=A) == INV and fwd(y=B_ + 64) == INV and fwd(y=C) == INV and fwd(r=E + 16) == INV and fwd(z=E + 64) == INV and fwd(z=D_) == INV
    q = L.haste_linear_fwd_workspace_bytes
    assert q(lin(), A, B_) == 0 and q(lin(M=8, K=65), A, B_) == 0   # few rows are read where they lie
    n = q(lin(K=65), A, B_)
    assert n >= (40 + 32) * 72 * 2 and q(lin(), A + 2, B_) >= 40 * 128 and q(lin(ld_x=65), A, B_) == q(lin(), A + 2, B_)
    assert fwd(lin(K=65)) == WS and fwd(lin(K=65), ws=G, n=n - 1) == WS and fwd(lin(K=65), ws=G + 16, n=n) == WS
    assert fwd(lin(K=65), ws=F_, n=n) == INV                        # over z

    def bwd(d=lin(), x=A, W=B_, dy=C, z=D_, add=None, dx=E, dW=F_, db=G, ws=H_, n=1 << 27):
        return L.haste_linear_bwd(d, x, W, dy, z, add, dx, dW, db, 0, ws, n, None)
    assert bwd(dx=None, dW=None, db=None) == INV and bwd(x=None) == INV and bwd(W=None) == INV and bwd(dy=None) == INV and bwd(z=None) == INV
    assert bwd(dx=None, add=I_) == INV and bwd(add=I_ + 1) == INV and bwd(dW=F_ + 1) == INV and bwd(db=G + 2) == INV
    assert bwd(dx=A) == INV and bwd(dW=B_) == INV and bwd(db=C) == INV and bwd(dW=E + 64) == INV and bwd(add=E + 16) == INV
    assert bwd(lin(ld_dx=80), add=E) == INV                         # dx_add over a strided dx
    assert bwd(ws=None) == WS and bwd(n=64) == WS and bwd(ws=H_ + 1) == WS and bwd(ws=C & ~255) == INV
    need = L.haste_linear_bwd_workspace_bytes(lin(), A, B_, C)
    assert need >= 40 * 32 * 2 and bwd(dx=None, dW=None, n=256) == WS
