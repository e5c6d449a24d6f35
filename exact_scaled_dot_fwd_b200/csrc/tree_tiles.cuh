// tree_tiles.cuh -- the key tiles of the tree attention and the pages in them.
// Lengths reach 2^31 - 1: what rounds one up does so without a sign.
#pragma once

namespace attn {
namespace tr {

constexpr int kTile = 128;        // keys per tile, rows per slot

// Tiles of n keys.
__host__ __device__ __forceinline__ int key_tiles(int n) {
  return (int)(((unsigned)n + (kTile - 1)) / kTile);
}

// Block-table entry of page i of tile jt of L cached keys (np = key_tiles(L),
// npg pages of page_size keys a tile); -1 if there is no cached key in it.
__host__ __device__ __forceinline__ int tile_page(int jt, int i, int np, int npg, int page_size,
                                                  int L) {
  return jt < np && i < npg && jt * kTile + i * page_size < L ? jt * npg + i : -1;
}

}  // namespace tr
}  // namespace attn
