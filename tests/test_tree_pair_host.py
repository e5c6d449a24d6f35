"""The pair of softmax warps of the tree attention's narrow form
(csrc/tree_pair.cuh), compiled as host C++: whatever waits give up in either
warp, both make the same steps at their common barrier (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_scaled_dot_fwd_b200", "csrc")

# A unit of n tiles as the kernel goes through it.  Each warp runs up to its
# next use of the barrier, where it names the step it is at; both must be at
# the same one.  Per tile and warp two waits (before the vote, and under an
# exchange) come through or not, whatever came before, and a rescale may be
# asked for: `bits` holds them all.
WRAPPER = r"""
#define __device__
#define __forceinline__ inline
#include "tree_pair.cuh"

// leaving on what only this warp knows
struct Private : attn::tr::PairExit {
  bool more(int j, int n) const { return ok() && j < n; }
};

enum Step { VOTE, EXCHANGE, WEIGHTS, END };

template <class Exit>
struct Warp {
  Exit exit;
  int j = 0, at = 0;      // tile, place in it
  bool asked = false;     // what this warp brings to a vote
  Step step;
  // runs to the next step; `vote` and `partner_ok` are the last one's outcome
  void run(int n, int who, unsigned bits, bool vote, bool partner_ok) {
    for (;;) {
      const unsigned b = bits >> (5 * j);
      switch (at) {
        case 0:
          if (!exit.more(j, n)) { step = END; return; }
          exit.waited(!((b >> who) & 1));
          asked = ((b >> 4) & 1) || j == 0 || !exit.ok();
          step = VOTE; at = 1;
          return;
        case 1:
          if (!vote) { ++j; at = 0; break; }
          step = EXCHANGE; at = 2;
          return;
        case 2:
          if (!exit.meet(partner_ok)) { ++j; at = 0; break; }
          if (j > 0) exit.waited(!((b >> (2 + who)) & 1));
          step = WEIGHTS; at = 3;
          return;
        default:
          ++j; at = 0;
      }
    }
  }
};

template <class Exit>
bool together(int n, unsigned bits) {
  Warp<Exit> w[2];
  bool vote = false, ok[2] = {true, true};
  for (;;) {
    for (int i = 0; i < 2; ++i) w[i].run(n, i, bits, vote, ok[i ^ 1]);
    if (w[0].step != w[1].step) return false;
    if (w[0].step == END) return true;
    vote = w[0].asked || w[1].asked;
    for (int i = 0; i < 2; ++i) ok[i] = w[i].exit.ok();
  }
}

// how many of all outcomes part the warps
extern "C" long parted(int n, int own) {
  long bad = 0;
  for (unsigned bits = 0; bits < 1u << (5 * n); ++bits)
    bad += own ? !together<Private>(n, bits) : !together<attn::tr::PairExit>(n, bits);
  return bad;
}
"""


@pytest.fixture(scope="module")
def P(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("tree_pair")
    src = d / "wrapper.cpp"
    src.write_text(WRAPPER)
    so = d / "libpair.so"
    subprocess.run([gxx, "-std=c++17", "-O2", "-fPIC", "-shared", "-I", CSRC, str(src), "-o", str(so)],
                   check=True)
    L = ctypes.CDLL(str(so))
    L.parted.restype = ctypes.c_long
    return L


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_both_warps_make_the_same_steps(P, n):
    assert P.parted(n, 0) == 0


def test_leaving_on_private_knowledge_parts_them(P):
    # (from three tiles on: a wait after the second tile's vote, then another tile)
    assert P.parted(3, 1) > 0
