"""Host-side refusals of the operators around the layer (no GPU: every call
here returns before it enqueues anything) and their workspace sizes."""
import ctypes

import pytest

from sparse_output_layer_amd import haste as H

OK, INV, UNS, WS = H.HASTE_OK, H.HASTE_ERR_INVALID, H.HASTE_ERR_UNSUPPORTED, H.HASTE_ERR_WORKSPACE
A, B_, C, D_, E = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000    # far apart


@pytest.fixture(scope="module")
def L():
    return H.lib()


def test_dropout_refusals(L):
    def go(B=4, D=8, xt=0, yt=0, x=A, d=H.DropoutStruct(0.5, 0, 1, 2), y=B_):
        return L.haste_dropout_apply(B, D, xt, yt, x, d, y, None)
    assert go(B=0) == INV and go(D=0) == INV and go(B=-1) == INV
    assert go(xt=2) == INV and go(yt=-1) == INV
    assert go(x=None) == INV and go(y=None) == INV and go(d=None) == INV
    assert go(x=A + 2) == INV and go(y=B_ + 1) == INV and go(xt=1, x=A + 1) == INV
    for p in (-0.1, 1.01, float("nan"), float("inf")):
        assert go(d=H.DropoutStruct(p, 0, 1, 2)) == INV
    assert go(d=H.DropoutStruct(0.5, 1, 1, 2)) == INV            # reserved
    assert go(y=A + 64) == INV and go(y=A, yt=1) == INV          # overlap; in place needs one type
    assert b"overlaps" in L.haste_last_error()


def norm(**kw):
    d = dict(B=4, D=8, x_dtype=1, y_dtype=0, w_dtype=0, eps=1e-5, ld_x=0, ld_dx=0)
    d.update(kw)
    return H.NormDesc(**d)


def test_norm_refusals(L):
    def fwd(d=norm(), x=A, g=B_, b=B_ + 64, dr=None, y=C, m=D_, r=D_ + 64):
        return L.haste_norm_fwd(d, x, g, b, dr, y, m, r, None)
    assert L.haste_norm_fwd(None, A, None, None, None, C, None, None, None) == INV
    for kw in (dict(B=0), dict(D=0), dict(x_dtype=3), dict(y_dtype=9), dict(w_dtype=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(ld_x=7), dict(ld_x=1 << 41)):
        assert fwd(norm(**kw)) == INV, kw
    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(m=None) == INV and fwd(r=None) == INV
    assert fwd(x=A + 1) == INV and fwd(y=C + 2) == INV and fwd(g=B_ + 1) == INV
    assert fwd(y=A) == INV and fwd(y=A + 60) == INV and fwd(m=C + 16) == INV and fwd(r=D_ + 8) == INV
    assert fwd(dr=H.DropoutStruct(2.0, 0, 0, 0)) == INV

    def bwd(d=norm(), x=A, g=B_, m=D_, r=D_ + 64, dy=C, dr=None, dx=E, dg=None, db=None, ws=None, n=0):
        return L.haste_norm_bwd(d, x, g, m, r, dy, dr, dx, dg, db, 0, ws, n, None)
    assert bwd(norm(ld_dx=7)) == INV and bwd(m=None) == INV and bwd(r=None) == INV
    assert bwd(dy=None) == INV and bwd(dx=None) == INV and bwd(dx=A) == INV and bwd(dx=C + 4) == INV
    assert bwd(dg=B_ + 4096) == WS                                # a weight gradient needs the workspace
    assert bwd(dg=B_ + 4096, ws=0x60000000, n=16) == WS
    need = L.haste_norm_bwd_workspace_bytes(norm())
    assert need >= 2 * 8 * 4 and bwd(dg=B_ + 4096, ws=0x60000080, n=need) == WS     # alignment
    assert bwd(dg=B_ + 4096, ws=E & ~0xFF, n=need) == INV         # over dx
    assert L.haste_norm_bwd_workspace_bytes(norm(B=0)) == 0
    assert L.haste_norm_bwd_workspace_bytes(norm(B=1 << 30, D=1 << 20)) > 0


def lpd(**kw):
    d = dict(B=4, dtype=1, H=64, L=1000, ld_h=0, ld_z=0)
    d.update(kw)
    return H.LogprobDesc(**d)


def test_logprob_refusals(L):
    big = 1 << 30

    def bce(**kw):
        d = dict(row_ptr=C, labels=C + 4096, nnz=5, grad_scale=1.0)
        d.update(kw)
        return H.BceStruct(**d)

    def fwd(d=lpd(), zh=A, z=B_, g=None, lp=None, lse=D_, ent=None, ws=E, n=big):
        return L.haste_logprob_fwd(d, zh, z, g, lp, lse, ent, ws, n, None)
    for kw in (dict(B=0), dict(dtype=4), dict(H=-1), dict(H=0, L=0), dict(L=2 ** 31 - 64), dict(H=2 ** 40), dict(ld_h=63),
               dict(ld_z=999), dict(ld_z=1 << 41)):
        assert fwd(lpd(**kw)) == INV, kw
        if not any(k.startswith("ld") for k in kw):
            assert L.haste_logprob_workspace_bytes(lpd(**kw), None) == 0
    assert fwd(zh=None) == INV and fwd(z=None) == INV and fwd(lse=None) == INV and fwd(zh=A + 1) == INV
    assert fwd(lp=D_ + 4096) == INV                               # logp without labels
    assert fwd(ws=None) == WS and fwd(n=4) == WS and fwd(ws=E + 16) == WS
    assert fwd(g=bce(nnz=-1)) == INV and fwd(g=bce(labels=None)) == INV and fwd(g=bce(row_ptr=None)) == INV
    assert fwd(g=bce(row_ptr=C + 2)) == INV and fwd(g=bce(label_offset=-1)) == INV
    assert fwd(g=bce(topk=9)) == INV and fwd(g=bce(topk=3)) == INV
    t = dict(topk=3, topk_val=D_ + 4096, topk_idx=D_ + 8192)
    assert fwd(g=bce(topk_kprime=2, topk_buckets=4, **t)) == UNS
    assert fwd(g=bce(label_offset=2 ** 31 - 100, **t)) == UNS     # ids are int32
    assert fwd(lse=A + 16) == INV and fwd(ent=D_ + 8) == INV and fwd(ws=B_ & ~0xFF) == INV
    n0 = L.haste_logprob_workspace_bytes(lpd(), None)
    assert 0 < n0 <= L.haste_logprob_workspace_bytes(lpd(), bce(**t))

    def bwd(d=lpd(), zh=A, z=B_, g=bce(), lse=D_, ent=D_ + 4096, dl=None, de=None, dzh=E, dz=E + 4096):
        return L.haste_logprob_bwd(d, zh, z, g, lse, ent, dl, de, dzh, dz, None)
    assert bwd(zh=None) == INV and bwd(dz=None) == INV and bwd(dzh=None) == INV and bwd(lse=None) == INV
    assert bwd(g=None) == INV                                     # nothing to differentiate
    assert bwd(g=None, dl=C, de=C) == INV                         # dlogp without labels
    assert bwd(de=C + 8192, ent=None) == INV
    assert bwd(dzh=A) == INV and bwd(dz=B_) == INV and bwd(dz=E + 64) == INV and bwd(dz=E + 4097) == INV


def test_i8_refusals(L):
    def q(rows=4, D=70, dt=0, ld=0, x=A, o=B_, s=C):
        return L.haste_quantize_rows(rows, D, dt, ld, x, o, s, None)
    assert q(rows=0) == INV and q(D=0) == INV and q(dt=5) == INV and q(ld=69) == INV and q(ld=1 << 41) == INV
    assert q(D=131073) == UNS
    assert q(x=None) == INV and q(x=A + 2) == INV and q(o=B_ + 8) == INV and q(s=C + 1) == INV and q(s=None) == INV
    assert q(o=A) == INV and q(s=B_ + 128) == INV

    def g(d=H.HeadDesc(4, 70, 9, 0), x=A, xs=B_, w=C, wsc=D_, z=E):
        return L.haste_head_fwd_i8(d, x, xs, w, wsc, z, None)
    assert g(None) == INV
    for kw in ((0, 70, 9, 0), (4, 0, 9, 0), (4, 70, 0, 0), (4, 70, 9, 7)):
        assert g(H.HeadDesc(*kw)) == INV, kw
    assert g(H.HeadDesc(4, 131073, 9, 0)) == UNS
    assert g(x=A + 8) == INV and g(w=None) == INV and g(xs=None) == INV and g(wsc=D_ + 2) == INV and g(z=E + 2) == INV
    assert g(z=C + 64) == INV and g(z=B_) == INV
