"""Host-side checks of the operators around the layer at the ends of their
ranges (no GPU)."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_output_layer_amd", "csrc")


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    """cut_rows of csrc/lp_cut.h, compiled for the host: (nc, per, nb, covered)."""
    d = tmp_path_factory.mktemp("cut")
    (d / "cut.cpp").write_text("""
#include "lp_cut.h"
extern "C" void cut(int B, int64_t H, int64_t L, int bf, int64_t *o) {
    const haste::Cut c = haste::cut_rows(B, H, L, bf != 0);
    const int64_t v[] = {c.nc[0], c.nc[1], c.per[0], c.per[1], c.nb, c.items, c.covered()};
    for (int i = 0; i < 7; ++i) o[i] = v[i];
}
""")
    so = d / "cut.so"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "cut.cpp"), "-o", str(so)])
    f = ctypes.CDLL(str(so)).cut
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]

    def go(B, Hn, L, bf):
        o = (ctypes.c_int64 * 7)()
        f(B, Hn, L, int(bf), o)
        return list(o)
    return go


def test_every_logit_is_in_a_chunk_that_its_kernel_covers(cut):
    """Both parts, either alone, numbers of rows and widths on both sides of
    every change of the rule, wherever in a vector a row starts: the chunks
    reach the row's end, none is empty, and none is longer than the batches of
    the kernel that is launched for it (256 threads of four vectors a batch)."""
    for bf in (False, True):
        V = 8 if bf else 4
        widths = {1, 2, V, V + 1, 1000, 5_000_000, 2 ** 31 - 2}
        for vec in (1, 1024, 2048, 4096, 8192, 16384, 32768):
            for d in (-1, 0, 1, 2, V):
                widths.add(max(1, vec * V - 2 * V + 2 + d))
                widths.add(vec * V + d)
        widths.update(range(4096 * V, 8400 * V, 1999))
        for n in sorted(widths):
            for other in (0, 1, 8191, 4097 * V):
                if n + other > 2 ** 31 - 1:
                    continue
                for B in (1, 2, 63, 64, 255, 256, 257, 511, 512, 513, 1024, 4096):
                    for parts in ((n, other), (other, n)):
                        c = cut(B, *parts, bf)
                        at = (B, parts, bf, c)
                        nb, items, ok = c[4:]
                        assert ok == 1 and nb in (1, 2, 4, 8) and items == B * (c[0] + c[1]), at
                        for p in (0, 1):
                            nc, per = c[p], c[2 + p]
                            if parts[p] == 0:
                                assert nc == 0, at
                                continue
                            vecs = -(-(parts[p] + V - 1) // V)     # a row that starts at a vector's last element
                            assert nc * per >= vecs and per <= nb * 4 * 256 and nc >= 1, at
                            # alone and short enough: one launch
                            if other == 0 and vecs <= 4 * 4 * 256 and nc > 1:
                                raise AssertionError(at)


def test_rows_in_each_others_gaps():
    """Rows of x and dx with one stride that share bytes are refused at every
    offset that makes them (rows that do not are tested on the device)."""
    from sparse_output_layer_amd import haste as H
    B, D, ld = 4, 8, 24
    A = 0x10000000
    d = H.NormDesc(B, D, H.HASTE_F32, H.HASTE_F32, H.HASTE_F32, 0.0, ld, ld)
    rows = {A + 4 * (r * ld + c) for r in range(B) for c in range(D)}
    seen = 0
    for off in range(-4 * ld * B, 4 * ld * B + 1, 4):
        dx = {a + off for a in rows}
        if rows & dx:
            seen += 1
            assert H.lib().haste_norm_bwd(d, A, None, A + 0x10000, A + 0x20000, A + 0x30000, None, A + off, None, None, 0, None,
                                          0, None) == H.HASTE_ERR_INVALID, off
    assert seen == (2 * B - 1) * (2 * D - 1)
