// tree_pair.cuh -- how the two softmax warps that share a quarter of the TMEM
// lanes go through a unit's key tiles and, when a wait gives up, leave
// together.
#pragma once

namespace attn {
namespace tr {

// On every tile the pair meets at a vote; where one of them asks (a rescale, the
// first tile, a wait that gave up) it also exchanges maxima and states, and
// meets once more after the tile's weights.  Both use one named barrier, so
// they must make the same steps: a wait that gives up in one warp only marks
// its state, and both leave on the next exchange, where each sees the other's.
// What gives up after the last exchange of a unit's tiles is seen by the vote of
// all softmax warps at its end.
struct PairExit {
  int state = 0;       // 1: a wait of this warp gave up, 2: both warps have left

  __device__ __forceinline__ bool ok() const { return state == 0; }
  __device__ __forceinline__ void waited(bool through) {
    if (!through && state == 0) state = 1;
  }
  // whether tile j of n is taken (the same in both warps)
  __device__ __forceinline__ bool more(int j, int n) const { return state < 2 && j < n; }
  // at an exchange, with the partner's ok(): whether the tile goes on
  __device__ __forceinline__ bool meet(bool partner_ok) {
    if (state != 0 || !partner_ok) state = 2;
    return state == 0;
  }
};

}  // namespace tr
}  // namespace attn
