"""Host-side refusals of the feature stage (no GPU: every call here returns
before it enqueues anything) and its workspace sizes."""
import pytest

from sparse_output_layer_amd import haste as H

INV, UNS, WS = H.HASTE_ERR_INVALID, H.HASTE_ERR_UNSUPPORTED, H.HASTE_ERR_WORKSPACE
A, B_, C, D_, E, F_, G = (i << 28 for i in range(1, 8))    # far apart


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
