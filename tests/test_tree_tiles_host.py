"""The tree attention's key tiles and pages (csrc/tree_tiles.cuh), compiled as
host C++, against whole numbers without a size: for lengths up to 2^31 - 1 no
table entry outside a sequence's pages is named (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_scaled_dot_fwd_b200", "csrc")

WRAPPER = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include "tree_tiles.cuh"
extern "C" {
int tiles(int n) { return attn::tr::key_tiles(n); }
int page(int jt, int i, int np, int ps, int L) {
  return attn::tr::tile_page(jt, i, np, 128 / ps, ps, L);
}
// in 32 bits that wrap, without asking first whether the tile is a cached one
int rounded_tiles(int n) { return (int)((unsigned)n + 127u) / 128; }
int product_page(int jt, int i, int ps, int L) {
  const unsigned pg = (unsigned)jt * (128 / ps) + i;
  return i < 128 / ps && (int)(pg * ps) < L ? (int)pg : -1;
}
}
"""

TOP = 2 ** 31 - 1
LENGTHS = [0, 1, 7, 127, 128, 129, 255, 256, 1000, 4096, 10 ** 6 + 3] + \
    [TOP - x for x in (0, 1, 7, 8, 15, 63, 64, 126, 127, 128, 255, 256)]


@pytest.fixture(scope="module")
def P(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("tree_tiles")
    src = d / "wrapper.cpp"
    src.write_text(WRAPPER)
    so = d / "libtiles.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-fPIC", "-shared", "-I", CSRC, str(src),
                    "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
def test_tiles_and_pages(P, ps):
    for L in LENGTHS:
        np = P.tiles(L)
        assert np == -(-L // 128)
        # the last cached tiles, and the drafted ones behind them
        for jt in range(max(0, np - 3), np + 9):
            for i in range(32):
                key = jt * 128 + i * ps
                want = jt * (128 // ps) + i if i < 128 // ps and key < L and jt < np else -1
                assert P.page(jt, i, np, ps, L) == want, (L, jt, i)
                assert want < -(-L // ps)


def test_rounding_up_first_names_entries_that_are_not_there(P):
    assert P.rounded_tiles(TOP - 7) < 0
    L, ps = TOP - 127, 128
    assert P.product_page(L // ps + 1, 0, ps, L) > -(-L // ps)
