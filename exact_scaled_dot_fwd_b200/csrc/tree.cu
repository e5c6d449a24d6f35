// tree.cu -- attention for a tree of drafted tokens over a cache: node i of a
// sequence sees every cached key, itself and its ancestors.
//
// The rows of one kv head of one sequence -- its live nodes times the query
// heads that share the kv head, packed without the padding nodes -- are cut
// into row groups of up to 256.  A unit is one (sequence, kv head, row
// group); its keys come in tiles of 128: the cached ones (ceil(L / 128) tiles,
// whole pages each), then the drafted ones, so only the last cached tile
// needs a length mask and only the drafted tiles the tree.
//
// Work split: all units' tiles are laid end to end with a cost each (Split)
// and cut evenly over one persistent CTA per SM.  A CTA so gets a run of
// segments (unit, tiles [j0, j0 + n)).  A unit that lies in one CTA is
// finished there; one that crosses a cut leaves an fp32 partial result with
// its log-sum-exp per CTA (at most two a CTA, its first and last segment),
// and a second kernel joins them.
//
// Warp roles:
//   0-7   softmax, two warpgroups (a thread owns a TMEM lane)
//   8     tcgen05.mma issuer, TMEM allocator
//   9     cuts the segments, loads K tiles by TMA
//   10    loads Q rows (by TMA; where nodes are missing, gathered by cp.async),
//         clears the dead output rows
//   11    loads V tiles by TMA (a box costs a warp some 100 cycles, and 16-token
//         pages make 16 boxes of a tile's K and V: at d = 64 out of L2 a tile took
//         1.13 us with one warp for both, 0.70 with two).  With row pairs, where
//         the products bound the tile, warp 10 does (1% faster than a 12th warp).
//
// Two forms, chosen by the rows of a kv head (its query heads times Nq):
//   up to 128: one row tile, TMEM S0 S1 S2 O; both warpgroups take every key
//     tile, and the fewer the rows the more copies of them the lanes hold (see
//     the softmax); S is three tiles ahead of P V.
//   more ("wide"): TMEM S0 S1 O0 O1, a slot for each warpgroup, taken in turn.
//     A row group above 128 rows is a pair: slot t holds its rows 128 t .. and
//     each key tile is taken by both slots.  A smaller one (the last of a kv
//     head) is in both slots, which take every other key tile; their (max,
//     sum, O) are joined when the segment ends.
// The rows are the M side of the MMAs.  With few rows most of M is padding or
// copies, but a tile's products take about 1000 cycles at d = 128 against the
// 2700 that its 64 KB need from HBM, so it costs nothing until two row tiles are
// full.
//
// Measured: 16 sequences of 1k to 16k keys, 36 to 64 rows on 8 kv heads, d =
// 128, 16-token pages: 109 us cool, 125 after 0.6 s of load; the main kernel reads
// 5.7 TB/s from HBM.  8 of 8k to 32k, 256 rows: 203 us cool (0.91 PFLOP/s), 244
// after load.  Row pairs take 1.9 to 2.2 us a tile and 25 to 30 us beside their
// tiles; a tile's products are 1.5 us and its exponentials 1.0, so neither pipe is
// full: what bounds them is the chain of a slot (two passes over S, the hand-off,
// P V, the next S), as in the prefill kernel.
//
// P goes back to TMEM as bf16 over its S and is the A operand of P V: a
// weight is off by at most 2^-8, as for every kernel of this library; sums,
// maxima and O stay in fp32.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tile_plan.cuh"
#include "tree_pair.cuh"
#include "tree_tiles.cuh"

namespace attn {
namespace tr {

constexpr int threads(bool wide) { return wide ? 352 : 384; }
constexpr int kMaxB = 2048;
constexpr int kSegSlots = 4;      // depth of the ring of segments
constexpr int seg_readers(bool wide) { return wide ? 10 : 11; }   // warps: MMA, Q, V, 8 softmax
constexpr float kRescaleLog2 = 8.0f;

// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division takes
// some hundred cycles)
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0
             ? (long long)((unsigned)a / (unsigned)b)
             : a / b;
}

// Costs of the work split, in fifths of a tile's HBM time: a tile of up to 128
// rows, one of a pair, and what one more unit costs a CTA (its epilogue, the
// next unit's first tiles): measured as the time by which CTAs with two
// segments end later than those with one, 3.5 to 4.6 us up to 64 rows, 9 above.
constexpr int kCostTile = 5, kCostPair = 8;
__host__ __device__ constexpr int unit_cost(int rp) { return rp > 128 ? 32 : (rp > 64 ? 28 : 16); }

template <int D>
struct Smem {
  static constexpr int kBox = kTile * 128;       // 64-column half of a tile
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int NS = D == 128 ? 5 : 10;   // ring of K and V tiles
  static constexpr int kQ = 0;                   // Q tiles [2]
  static constexpr int kKV = 2 * kTileBytes;
  static constexpr int kMl = kKV + NS * kTileBytes;   // float2 [2][128]: (max, sum) of a slot's rows
  static constexpr int kBar = kMl + 2 * kTile * 8;
  enum {
    FULL = 0,
    EMPTY = FULL + NS,
    Q_FULL = EMPTY + NS,      // [2], 2 arrivals
    Q_EMPTY = Q_FULL + 2,     // [2]
    S_FULL = Q_EMPTY + 2,     // [3]
    P_FULL = S_FULL + 3,      // [3], 128 or 256 arrivals
    O_FULL = P_FULL + 3,      // [2]
    SEG_FULL = O_FULL + 2,    // [kSegSlots]
    SEG_EMPTY = SEG_FULL + kSegSlots,   // [kSegSlots], seg_readers arrivals
    MMA_DONE = SEG_EMPTY + kSegSlots,
    NUM_BARS = MMA_DONE + 1
  };
  static constexpr int kSeg = kBar + NUM_BARS * 8;   // int [kSegSlots][kSegInts]
  static constexpr int kSegInts = 8;
  static constexpr int kTmemSlot = kSeg + kSegSlots * kSegInts * 4;
  static constexpr int kAbort = kTmemSlot + 8;
  // int [NS + 2]: the position each stage, the tile each Q buffer was last filled for
  static constexpr int kArmed = kAbort + 8;
  static constexpr int kTotal = kArmed + (NS + 2) * 4;   // (the base is 1024-byte aligned)
  static_assert(kTotal <= 232448, "shared memory over the 227 KB per-CTA limit");
};

struct Args {
  TreeArgs t;
  float* part_o;      // [2 * ranges][RP][D]
  float* part_lse;    // [2 * ranges][RP], log2 units
  struct Record* records;   // [ranges]
  int G, RP, grid, ranges, oob_row;
  int cost_unit;
};

// What a range leaves for the join: the unit it starts and does not finish.
struct Record {
  int last;           // range that holds the unit's last tile; -1: no such unit
  int slot;           // its partial slot here; it is 2 * range in those after
  int b, h, rg, rows, nb;   // the unit and its rows
  int w, nt, pad;     // its tiles and their cost
  long long p0;       // where it starts
  long long T;        // total cost
  long long pad2;
};
static_assert(sizeof(Record) == 64, "copied in 16-byte pieces");

// A segment as its readers see it.
struct Seg {
  int b, h, rg;       // unit
  int j0, n;          // key tiles [j0, j0 + n); n = 0 ends the stream
  int L, nb;          // cached keys, live nodes
  int flags;          // 1: the CTA's first segment, 2: the whole unit
  __device__ __forceinline__ int np() const { return key_tiles(L); }
};

__device__ __forceinline__ int cached_len(const TreeArgs& t, int b) {
  return clamp_len(t.key_lens ? t.key_lens[b] : t.Nk, t.Nk);
}
__device__ __forceinline__ int live_nodes(const TreeArgs& t, int b) {
  return clamp_len(t.new_lens ? t.new_lens[b] : t.Nq, t.Nq);
}

// The units of one sequence and their costs.
struct Split {
  int nt;              // tiles of a unit (0: no live node, no unit)
  int nrg;             // row groups of a kv head
  int cu;              // what a unit costs beside its tiles
  int w_last;          // tile cost of the last row group (the others are pairs)
  long long head;      // cost of a kv head
  __device__ __forceinline__ Split(int L, int nb, int G, int cost_unit) : cu(cost_unit) {
    const int rows = G * nb;
    nt = nb > 0 ? key_tiles(L) + key_tiles(nb) : 0;
    nrg = (rows + 2 * kTile - 1) / (2 * kTile);
    w_last = rows - (nrg - 1) * 2 * kTile > kTile ? kCostPair : kCostTile;
    head = nb > 0 ? (long long)(nrg - 1) * unit(kCostPair) + unit(w_last) : 0;
  }
  __device__ __forceinline__ int weight(int rg) const { return rg < nrg - 1 ? kCostPair : w_last; }
  __device__ __forceinline__ long long unit(int w) const { return cu + (long long)nt * w; }
};

// Where tile j of a unit starts (the unit's own cost belongs to tile 0), and how
// many of its nt tiles start before x.
__device__ __forceinline__ long long tile_at(int j, int w, int cu) {
  return j == 0 ? 0 : cu + (long long)j * w;
}
__device__ __forceinline__ int tiles_before(long long x, int w, int nt, int cu) {
  if (x <= 0) return 0;
  x -= cu;
  if (x <= 0) return 1;
  const long long j = div_pos(x + w - 1, w);
  return j > nt ? nt : (int)j;
}

// The cuts: range i is [at(i), at(i + 1)) of the total cost.
struct Cuts {
  long long T;
  int n;
  __device__ __forceinline__ Cuts(long long total, const Args& a) : T(total), n(a.ranges) {}
  __device__ __forceinline__ long long at(int i) const { return div_pos(T * i, n); }
  // the range that holds x
  __device__ __forceinline__ int of(long long x) const {
    int c = (int)div_pos(x * n, T);
    while (c + 1 < n && at(c + 1) <= x) ++c;
    while (c > 0 && at(c) > x) --c;
    return c;
  }
};

// Eight consecutive TMEM columns (see tc::st16).
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 4D tiled load (no multicast): one page of a paged cache, d = 128.
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Node and ancestors of up to 32 nodes as bits, lane i holding the parent of node
// i (-1: none): each round takes in the set of the ancestor reached so far and
// doubles the distance to it.  A parent that does not come before its node is
// reported and taken as none.
__device__ __forceinline__ uint32_t ancestors32(int parent, int lane) {
  if (parent < -1 || parent >= lane) {
    atomicExch(&g_device_status, (int)ATTN_ERANGE);
    parent = -1;
  }
  uint32_t set = 1u << lane;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int from = parent < 0 ? lane : parent;
    set |= __shfl_sync(0xffffffffu, set, from);
    const int up = __shfl_sync(0xffffffffu, parent, from);
    parent = parent < 0 ? -1 : up;
  }
  return set;
}

}  // namespace tr

template <int D, bool kPaged, int kKeys>
__global__ void __launch_bounds__(tr::threads(kKeys == 0), 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ CUtensorMap tkn, const __grid_constant__ CUtensorMap tvn,
                   tr::Args a) {
  using namespace tr;
  using L = Smem<D>;
  constexpr bool kWide = kKeys == 0;
  constexpr int kCopies = kWide ? 1 : 64 / kKeys;   // of the rows in a row tile
  constexpr int NS = L::NS;
  constexpr uint32_t kIdescS = tc::idesc_bf16(kTile, kTile, false, false);
  constexpr uint32_t kIdescPV = tc::idesc_bf16(kTile, D, false, true);
  // no room for aligning by hand: the swizzled tiles rely on the declaration
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  volatile int* segs = reinterpret_cast<volatile int*>(smem + L::kSeg);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  volatile int* armed = reinterpret_cast<volatile int*>(smem + L::kArmed);
  const TreeArgs& t = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the join may launch now; it waits for this grid before it reads anything
  asm volatile("griddepcontrol.launch_dependents;");
  if ((smem_u32(smem) & 1023u) != 0) {   // (never seen; nothing below would be in place)
    atomicExch(&g_device_status, (int)ATTN_ECUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NUM_BARS; ++i) {
      uint32_t c = 1;
      if (i >= L::P_FULL && i < L::O_FULL) c = kWide ? 128 : 256;
      if (i == L::Q_FULL || i == L::Q_FULL + 1) c = 2;
      if (!kWide && (i == L::Q_EMPTY || i == L::Q_EMPTY + 1)) c = 8;
      if (i >= L::SEG_EMPTY && i < L::SEG_EMPTY + kSegSlots) c = seg_readers(kWide);
      mbar_init(&bars[i], c);
    }
    *abort_flag = 0;
    for (int i = 0; i < NS + 2; ++i) armed[i] = -1;
    fence_mbar_init();
  }
  if (warp == 8) {
    tc::alloc(tmem_slot, 512);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  // Launched as a programmatic dependent of the previous kernel in the
  // stream: nothing in global memory is touched before it has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // next segment from the ring; every lane of a reading warp takes part
  auto next_seg = [&](int& k, Seg& s) -> bool {
    const int slot = k % kSegSlots;
    if (!mbar_wait_warp(&bars[L::SEG_FULL + slot], (k / kSegSlots) & 1, abort_flag)) return false;
    volatile int* p = segs + slot * L::kSegInts;
    s.b = p[0]; s.h = p[1]; s.rg = p[2]; s.j0 = p[3];
    s.n = p[4]; s.L = p[5]; s.nb = p[6]; s.flags = p[7];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[L::SEG_EMPTY + slot]);
    ++k;
    return s.n > 0;
  };
  auto group_rows = [&](const Seg& s) -> int {   // live rows of the segment's row group
    const int r = a.G * s.nb - s.rg * 2 * kTile;
    return r < 2 * kTile ? r : 2 * kTile;
  };
  // Ring positions of a segment of n tiles that starts at g.  Pair: K0 V0 K1
  // V1 ..; else the first kAhead K, then V0 and the next K, V1 and the next
  // K, ..: the order in which the MMAs use them.
  constexpr int kAhead = kWide ? 2 : 3;
  auto k_pos = [](int g, int j, bool pair) {
    return pair ? g + 2 * j : (j < kAhead ? g + j : g + 2 * j - kAhead + 1);
  };
  auto v_pos = [](int g, int j, int n, bool pair) {
    return pair ? g + 2 * j + 1 : (j <= n - kAhead ? g + kAhead + 2 * j : g + n + j);
  };

  // The K or the V tiles of a segment into their ring positions, by one warp.
  auto load_tiles = [&](const Seg& s, int g, bool is_v) -> bool {
    const int n = s.n, np = s.np();
    const bool pair = kWide && group_rows(s) > kTile;
    const int bh = s.b * t.Hkv + s.h;
    const int npg = kPaged ? kTile / t.page_size : 0;
    const int32_t* table = kPaged ? t.block_table + (size_t)s.b * t.max_pages : nullptr;
    const CUtensorMap* map = is_v ? &tv : &tk;
    const CUtensorMap* map_new = is_v ? &tvn : &tkn;
    // this lane's entry of the block table for tile j (-1: a page past the
    // cached keys), looked up two tiles before it is needed
    auto entry = [&](int j) -> int {
      const int pg = j < n ? tile_page(s.j0 + j, lane, np, npg, t.page_size, s.L) : -1;
      return pg >= 0 ? table[pg] : -1;
    };
    int e0 = kPaged ? entry(0) : 0, e1 = kPaged ? entry(1) : 0;
    for (int j = 0; j < n; ++j) {
      const int e2 = kPaged ? entry(j + 2) : 0;
      const int jt = s.j0 + j, pos = is_v ? v_pos(g, j, n, pair) : k_pos(g, j, pair);
      const int st = pos % NS;
      uint64_t* full = &bars[L::FULL + st];
      bool w_ok = true;
      if (lane == 0) {
        w_ok = mbar_wait(&bars[L::EMPTY + st], ((pos / NS) & 1) ^ 1, abort_flag);
        if (w_ok) {
          mbar_arrive_expect_tx(full, L::kTileBytes);
          armed[st] = pos;
        }
      }
      if (!__shfl_sync(0xffffffffu, w_ok, 0)) return false;
      uint8_t* dst = smem + L::kKV + st * L::kTileBytes;
      if (jt >= np) {
        if (lane < D / 64)
          tma_load_3d(dst + lane * L::kBox, map_new, lane * 64, (jt - np) * kTile, bh, full);
      } else if constexpr (kPaged) {
        if (lane < npg) {
          // (pages past the cached keys: the row past the cache, zeros)
          const int row = tile_page(jt, lane, np, npg, t.page_size, s.L) >= 0
                              ? paged_cache_row(e0, t.num_pages, t.Hkv, s.h, t.page_size, a.oob_row)
                              : a.oob_row;
          if constexpr (D == 128) tma_load_4d(dst + lane * t.page_size * 256, map, row >> 3, full);
          else tma_load_2d(dst + lane * t.page_size * 128, map, 0, row, full);
        }
      } else {
        if (lane < D / 64) tma_load_3d(dst + lane * L::kBox, map, lane * 64, jt * kTile, bh, full);
      }
      e0 = e1;
      e1 = e2;
    }
    return true;
  };

  // The Q rows of a segment, `part` of `parts` of them, by one warp: row r of the
  // unit is node r % nb of head r / nb.  Where no node is missing the rows lie
  // together and come by TMA, a box for each copy.  Else a lane copies one
  // 16-byte chunk of every (32 / chunks)-th row, to each of the row's copies.
  auto load_q = [&](const Seg& s, int qt, int part, int parts) -> bool {
    constexpr int kChunks = D / 8, kStep = 32 / kChunks, span = kTile / kCopies;
    const int c = lane % kChunks, rows = group_rows(s);
    const int nq = kWide && rows > kTile ? 2 : 1;
    if (s.nb == t.Nq) {
      for (int sl = 0; part == 0 && sl < nq; ++sl) {
        const int buf = (qt + sl) & 1;
        uint64_t* full = &bars[L::Q_FULL + buf];
        if (!mbar_wait_warp(&bars[L::Q_EMPTY + buf], (((qt + sl) >> 1) & 1) ^ 1, abort_flag))
          return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, L::kTileBytes);
          armed[NS + buf] = qt + sl;
          for (int cp = 0; cp < kCopies; ++cp)
            for (int hb = 0; hb < D / 64; ++hb)
              tma_load_3d(smem + L::kQ + buf * L::kTileBytes + hb * L::kBox + cp * span * 128, &tq,
                          hb * 64, s.rg * 2 * kTile + sl * kTile, s.b * t.Hkv + s.h, full);
          mbar_arrive(full);
        }
        __syncwarp();
      }
      return true;
    }
    const int dg = kStep / s.nb, di = kStep % s.nb;
    const __nv_bfloat16* qb = t.q + ((size_t)s.b * t.Hq + (size_t)s.h * a.G) * t.Nq * D + c * 8;
    for (int sl = 0; sl < nq; ++sl) {
      const int buf = (qt + sl) & 1;
      if (!mbar_wait_warp(&bars[L::Q_EMPTY + buf], (((qt + sl) >> 1) & 1) ^ 1, abort_flag))
        return false;
      const uint32_t dst = smem_u32(smem + L::kQ + buf * L::kTileBytes) +
                           (uint32_t)(c >> 3) * L::kBox;
      const int r0 = s.rg * 2 * kTile + sl * kTile, some = span / parts;
      int r_end = rows - sl * kTile < span ? rows - sl * kTile : span;
      if (r_end > (part + 1) * some) r_end = (part + 1) * some;
      int r = part * some + lane / kChunks, gh = (r0 + r) / s.nb, i = (r0 + r) % s.nb;
#pragma unroll 4
      for (; r < r_end; r += kStep) {
        const __nv_bfloat16* src = qb + ((size_t)gh * t.Nq + i) * D;
#pragma unroll
        for (int cp = 0; cp < kCopies; ++cp)
          cp_async_16(dst + sw128_offset(r + cp * span, c & 7), src);
        gh += dg;
        i += di;
        if (i >= s.nb) { i -= s.nb; ++gh; }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int sl = 0; sl < nq; ++sl) {   // (the second tile's rows are on their way too)
      if (sl + 1 < nq) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (part == 0) armed[NS + ((qt + sl) & 1)] = qt + sl;
        for (int x = parts; x < 3; ++x) mbar_arrive(&bars[L::Q_FULL + ((qt + sl) & 1)]);
      }
    }
    return true;
  };

  if (warp == 9) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      tma_prefetch_desc(&tkn);
      tma_prefetch_desc(&tvn);
    }
    int k = 0, g = 0;        // segments and ring positions so far
    bool ok = true;
    int b = 0, h = 0, rg = 0, j0 = 0, Lb = 0, nb = 0;
    long long p0 = 0;        // where the current unit starts
    Split sp(0, 0, 1, a.cost_unit);
    // total cost, and the sequence in which this CTA's share starts: a lane
    // sums `per` sequences, the warp the lanes' sums
    auto seq_cost = [&](int i) -> long long {
      return (long long)t.Hkv * Split(cached_len(t, i), live_nodes(t, i), a.G, a.cost_unit).head;
    };
    const int per = (t.B + 31) >> 5;
    long long mine = 0;
#pragma unroll 4
    for (int i = lane * per; i < (lane + 1) * per; ++i)
      if (i < t.B) mine += seq_cost(i);
    long long at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    const long long T = __shfl_sync(0xffffffffu, at, 31);
    at -= mine;
    const Cuts cuts(T, a);
    const long long start = cuts.at(blockIdx.x), end = cuts.at(blockIdx.x + 1);
    bool more = start < end;
    if (more) {
      const int src = __ffs(__ballot_sync(0xffffffffu, at <= start && start < at + mine)) - 1;
      b = lane * per;
      if (lane == src && per > 1)
        for (long long c; at + (c = seq_cost(b)) <= start; at += c) ++b;
      b = __shfl_sync(0xffffffffu, b, src);
      at = __shfl_sync(0xffffffffu, at, src);
    }
    Record rec;
    rec.last = -1;
    rec.T = T;
    int ahead = -1, ahead_L = 0, ahead_n = 0;
    // first unit with live nodes at or after (b, 0, 0)
    auto load_seq = [&]() {
      for (; b < t.B; ++b) {
        Lb = b == ahead ? clamp_len(ahead_L, t.Nk) : cached_len(t, b);
        nb = b == ahead ? clamp_len(ahead_n, t.Nq) : live_nodes(t, b);
        sp = Split(Lb, nb, a.G, a.cost_unit);
        // the next sequence's lengths, asked for now and looked at when it comes
        ahead = b + 1;
        if (ahead < t.B) {
          ahead_L = t.key_lens ? t.key_lens[ahead] : t.Nk;
          ahead_n = t.new_lens ? t.new_lens[ahead] : t.Nq;
        }
        if (sp.nt > 0) return;
      }
    };
    auto next_unit = [&]() {
      p0 += sp.unit(sp.weight(rg));
      j0 = 0;
      if (++rg == sp.nrg) {
        rg = 0;
        if (++h == t.Hkv) {
          h = 0;
          ++b;
          load_seq();
        }
      }
    };
    if (more) {
      load_seq();
      long long rel = start - at;
      h = (int)div_pos(rel, sp.head);
      rel -= h * sp.head;
      rg = (int)div_pos(rel, sp.unit(kCostPair));
      if (rg > sp.nrg - 1) rg = sp.nrg - 1;
      rel -= rg * sp.unit(kCostPair);
      p0 = start - rel;
      j0 = rel == 0 ? 0 : tiles_before(rel, sp.weight(rg), sp.nt, a.cost_unit);
      if (j0 == sp.nt) next_unit();
    }
    while (ok) {
      const int w = sp.weight(rg);
      int n = 0;
      if (more && b < t.B && p0 + tile_at(j0, w, a.cost_unit) < end) n = tiles_before(end - p0, w, sp.nt, a.cost_unit) - j0;
      const int slot = k % kSegSlots;
      if (!mbar_wait_warp(&bars[L::SEG_EMPTY + slot], ((k / kSegSlots) & 1) ^ 1, abort_flag)) break;
      const bool whole = j0 == 0 && n == sp.nt;
      if (lane == 0) {
        volatile int* p = segs + slot * L::kSegInts;
        p[0] = b; p[1] = h; p[2] = rg; p[3] = j0;
        p[4] = n; p[5] = Lb; p[6] = nb; p[7] = (k == 0 ? 1 : 0) | (whole ? 2 : 0);
        mbar_arrive(&bars[L::SEG_FULL + slot]);
      }
      if (n == 0) break;
      if (j0 == 0 && n < sp.nt) {   // this CTA starts a unit that others finish
        const int rows = a.G * nb - rg * 2 * kTile;
        rec.last = cuts.of(p0 + tile_at(sp.nt - 1, w, a.cost_unit));
        rec.slot = 2 * blockIdx.x + (k == 0 ? 0 : 1);
        rec.b = b; rec.h = h; rec.rg = rg;
        rec.rows = rows < 2 * kTile ? rows : 2 * kTile;
        rec.nb = nb; rec.w = w; rec.nt = sp.nt; rec.p0 = p0;
      }
      ++k;

      Seg sg;
      sg.b = b; sg.h = h; sg.rg = rg; sg.j0 = j0; sg.n = n; sg.L = Lb; sg.nb = nb;
      ok = load_tiles(sg, g, false);
      g += 2 * n;
      j0 += n - 1;   // (only its being the unit's last tile matters below)
      if (j0 == sp.nt - 1) next_unit(); else more = false;
    }
    if (lane == 0) {
      a.records[blockIdx.x] = rec;
    }
  } else if (!kWide && warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    // One slot: S of tile u (counted over the segments) in buffer u % 3, three
    // tiles ahead of P V, O behind them.
    const uint32_t q_base = smem_u32(smem + L::kQ), kv_base = smem_u32(smem + L::kKV);
    auto commit = [&](int bar) {
      if (elect_one()) tc::commit(&bars[bar]);
      __syncwarp();
    };
    int k = 0, g = 0, qt = 0, u0 = 0;
    bool ok = true;
    Seg s;
    while (ok && next_seg(k, s)) {
      const int n = s.n, np = s.np();
      auto grouped = [&](int j) { return kPaged && D == 128 && s.j0 + j < np; };
      auto do_s = [&](int j) -> bool {
        const int pos = k_pos(g, j, false), buf = (u0 + j) % 3;
        if (!mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag)) return false;
        tc::fence_after();
        const uint32_t half = grouped(j) ? 1024u : (uint32_t)L::kBox;
        const uint64_t dq = tc::smem_desc_sw128(q_base + (qt & 1) * L::kTileBytes, 16, 1024);
        const uint64_t dk = tc::smem_desc_sw128(kv_base + (pos % NS) * L::kTileBytes, 16,
                                                grouped(j) ? 2048 : 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ss(tmem + 128u * buf, dq + (uint64_t)(((kk >> 2) * L::kBox + (kk & 3) * 32) >> 4),
                       dk + (uint64_t)(((kk >> 2) * half + (kk & 3) * 32) >> 4), kIdescS,
                       kk > 0 ? 1u : 0u);
          tc::commit(&bars[L::S_FULL + buf]);
          tc::commit(&bars[L::EMPTY + pos % NS]);
        }
        __syncwarp();
        return true;
      };
      if (!mbar_wait_warp(&bars[L::Q_FULL + (qt & 1)], (qt >> 1) & 1, abort_flag)) break;
      for (int j = 0; ok && j < kAhead && j < n; ++j) ok = do_s(j);
      for (int j = 0; ok && j < n; ++j) {
        const int u = u0 + j, pos = v_pos(g, j, n, false);
        if (!mbar_wait_warp(&bars[L::P_FULL + u % 3], (u / 3) & 1, abort_flag)) { ok = false; break; }
        if (!mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag)) { ok = false; break; }
        tc::fence_after();
        const uint32_t half = grouped(j) ? 1024u : (uint32_t)L::kBox;
        const uint32_t grp = grouped(j) ? 2048u : 1024u;
        const uint64_t dv = tc::smem_desc_sw128(kv_base + (pos % NS) * L::kTileBytes, half, grp);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc::mma_ts(tmem + 384u, tmem + 128u * (u % 3) + kk * 8,
                       dv + (uint64_t)((kk * 2 * grp) >> 4), kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
          tc::commit(&bars[L::O_FULL + (u & 1)]);
          tc::commit(&bars[L::EMPTY + pos % NS]);
        }
        __syncwarp();
        if (j + kAhead < n) ok = do_s(j + kAhead);
      }
      g += 2 * n;
      u0 += n;
      ++qt;
    }
    // every MMA of this CTA must be complete before TMEM is released
    commit(L::MMA_DONE);
    mbar_wait_warp(&bars[L::MMA_DONE], 0, nullptr);
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t q_base = smem_u32(smem + L::kQ), kv_base = smem_u32(smem + L::kKV);
    auto commit = [&](int bar) {
      if (elect_one()) tc::commit(&bars[bar]);
      __syncwarp();
    };
    int k = 0, g = 0, qt = 0, pw0 = 0, pw1 = 0;
    bool ok = true;
    Seg s;
    while (ok && next_seg(k, s)) {
      const bool pair = group_rows(s) > kTile;
      const int n = s.n, ns = pair ? 2 * n : n, np = s.np();
      // strides of a tile: a page of d = 128 lands as 8-row groups of [half 0
      // | half 1], everything else as 64-column halves
      auto grouped = [&](int j) { return kPaged && D == 128 && s.j0 + j < np; };
      auto do_s = [&](int st) -> bool {
        const int sl = st & 1, j = pair ? st >> 1 : st;
        const int pos = k_pos(g, j, pair), q = pair ? qt + sl : qt;
        if (pair ? st < 2 : st == 0) {
          if (!mbar_wait_warp(&bars[L::Q_FULL + (q & 1)], (q >> 1) & 1, abort_flag)) return false;
        }
        if (!pair || sl == 0) {
          if (!mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag)) return false;
        }
        tc::fence_after();
        const uint32_t half = grouped(j) ? 1024u : (uint32_t)L::kBox;
        const uint64_t dq = tc::smem_desc_sw128(q_base + (q & 1) * L::kTileBytes, 16, 1024);
        const uint64_t dk = tc::smem_desc_sw128(kv_base + (pos % NS) * L::kTileBytes, 16,
                                                grouped(j) ? 2048 : 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ss(tmem + 128u * sl, dq + (uint64_t)(((kk >> 2) * L::kBox + (kk & 3) * 32) >> 4),
                       dk + (uint64_t)(((kk >> 2) * half + (kk & 3) * 32) >> 4), kIdescS,
                       kk > 0 ? 1u : 0u);
        }
        __syncwarp();
        commit(L::S_FULL + sl);
        if (!pair || sl == 1) commit(L::EMPTY + pos % NS);
        if (pair ? st >= ns - 2 : st == ns - 1) commit(L::Q_EMPTY + (q & 1));
        return true;
      };
      for (int st = 0; ok && st < 2 && st < ns; ++st) ok = do_s(st);
      for (int st = 0; ok && st < ns; ++st) {
        const int sl = st & 1, j = pair ? st >> 1 : st;
        const int pos = v_pos(g, j, n, pair);
        int& pw = sl ? pw1 : pw0;
        if (!mbar_wait_warp(&bars[L::P_FULL + sl], pw & 1, abort_flag)) { ok = false; break; }
        ++pw;
        if (!pair || sl == 0) {
          if (!mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag)) { ok = false; break; }
        }
        tc::fence_after();
        const uint32_t half = grouped(j) ? 1024u : (uint32_t)L::kBox;
        const uint32_t grp = grouped(j) ? 2048u : 1024u;
        const uint64_t dv = tc::smem_desc_sw128(kv_base + (pos % NS) * L::kTileBytes, half, grp);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc::mma_ts(tmem + 256u + (uint32_t)D * sl, tmem + 128u * sl + kk * 8,
                       dv + (uint64_t)((kk * 2 * grp) >> 4), kIdescPV, (st >= 2 || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
        if (!pair || sl == 1) commit(L::EMPTY + pos % NS);
        if (st >= ns - 2) commit(L::O_FULL + sl);
        if (st + 2 < ns) ok = do_s(st + 2);
      }
      g += 2 * n;
      qt += pair ? 2 : 1;
    }
    // every MMA of this CTA must be complete before TMEM is released
    commit(L::MMA_DONE);
    mbar_wait_warp(&bars[L::MMA_DONE], 0, nullptr);
  } else if (!kWide && warp == 11) {
    // ------------------------------------------------------------ V tiles
    int k = 0, g = 0;
    Seg s;
    while (next_seg(k, s)) {
      if (k == 1 && !load_q(s, 0, 1, 2)) break;   // half of the first segment's Q
      if (!load_tiles(s, g, true)) break;
      g += 2 * s.n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 10) {
    // ------------------------------------------------------------ Q rows
    int k = 0, qt = 0;
    Seg s;
    int g = 0;
    while (next_seg(k, s)) {
      if (!load_q(s, qt, 0, !kWide && k == 1 ? 2 : 1)) break;
      qt += kWide && group_rows(s) > kTile ? 2 : 1;
      if (kWide && !load_tiles(s, g, true)) break;
      g += 2 * s.n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // rows of the nodes a sequence does not have
    if (t.new_lens) {
      for (long long x = blockIdx.x; x < (long long)t.B * t.Hq; x += a.grid) {
        const int nb = live_nodes(t, (int)(x / t.Hq));
        uint4* o = reinterpret_cast<uint4*>(t.o + (x * t.Nq + nb) * D);
        for (int e = lane; e < (t.Nq - nb) * (D / 8); e += 32) o[e] = make_uint4(0, 0, 0, 0);
        if (t.lse)
          for (int e = nb + lane; e < t.Nq; e += 32) t.lse[x * t.Nq + e] = -INFINITY;
      }
    }
  } else if (!kWide) {
    // ------------------------------------------------------------ softmax
    // Both warpgroups take every tile: warps q and q + 4 share the lanes of
    // quarter q, the one the first 64 keys, the other the last.  With 64 rows or
    // fewer the lanes hold 2 copies of the rows, with 32 or fewer 4, and copy c
    // takes the c-th part of either 64 keys: its P is zero elsewhere, its O
    // row is the sum over its keys, and the copies' maxima and sums are joined
    // when the segment ends.  So all 8 warps work on any number of rows, 64,
    // 32 or 16 keys a thread: a tile of 25 rows at d = 64 took 1.13 us with one
    // warp of each warpgroup on whole rows of every other tile.
    const int hf = warp >> 2, qr = warp & 3;
    const int r = qr * 32 + lane;             // TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(qr * 32) << 16);
    const float sl2 = t.scale_log2;
    const bool o_32B = (reinterpret_cast<uintptr_t>(t.o) & 31) == 0;
    float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
    int k = 0, g = 0, u0 = 0, qt = 0;
    PairExit pair;
    Seg s;
    bool live = next_seg(k, s);
    while (!bar_vote_or(1, 256, !live)) {
      const int rows = group_rows(s), n = s.n, np = s.np();
      constexpr int copies = kCopies, per_copy = 4 / copies;   // warps
      const int copy = qr / per_copy;
      const int lr = (qr - copy * per_copy) * 32 + lane;   // row of the unit
      const bool idle = lr - lane >= rows;                 // no live row in this warp
      const bool dead = lr >= rows;                        // computes on anything, is not stored
      const int rr = lr < rows ? lr : rows - 1;
      const int head = rr / s.nb, node = rr - head * s.nb;
      float m_run = -INFINITY, l_run = 0.f;
      // a small tree's parents, asked for here and looked at on its tile
      const bool small = s.nb <= 32;
      int parent = -1;
      if (small && s.j0 + n > np && lane < s.nb) parent = t.parents[(size_t)s.b * t.Nq + lane];

      // one tile, NC keys of this thread from key k0 of the tile on
      auto tile = [&](auto mask, int j, int jt, int valid) {
        constexpr int NC = kWide ? 64 : kKeys;
        constexpr bool masked = decltype(mask)::value;
        const int u = u0 + j;
        const int k0 = 64 * hf + copy * NC;
        const uint32_t sc = lanes + 128u * (u % 3);
        unsigned long long seen = ~0ull;                   // bit e: key k0 + e is visible
        if (masked) {
          if (jt < np) {
            const int e = valid - k0;
            seen = e >= 64 ? ~0ull : (e <= 0 ? 0ull : (1ull << e) - 1ull);
          } else if (small) {
            const uint32_t set = __shfl_sync(0xffffffffu, ancestors32(parent, lane), node);
            seen = k0 < 32 ? set >> k0 : 0u;
          } else {
            // the node and its ancestors among drafts [first, first + NC)
            const int first = (jt - np) * kTile + k0;
            const int32_t* par = t.parents + (size_t)s.b * t.Nq;
            seen = 0ull;
            for (int v = node; v >= first;) {
              if (v - first < NC) seen |= 1ull << (v - first);
              const int p = par[v];
              if (p < -1 || p >= v) {
                atomicExch(&g_device_status, (int)ATTN_ERANGE);
                break;
              }
              v = p;
            }
          }
        }
        // A wait that gives up only marks the warp: it goes on to the next vote, where
        // it and its partner leave together.
        pair.waited(mbar_wait_warp(&bars[L::S_FULL + u % 3], (u / 3) & 1, abort_flag));
        // P V of tile u - 2 (each of its barrier's phases is waited for, in order)
        if (u >= 2)
          pair.waited(mbar_wait_warp(&bars[L::O_FULL + (u & 1)], ((u - 2) >> 1) & 1, abort_flag));
        tc::fence_after();
        if (masked && valid < kTile && hf == 0) {
          // values that do not exist: anything may be stored there
          const int pos = v_pos(g, j, n, false);
          pair.waited(mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag));
          if (r >= valid) {
            const bool grouped = kPaged && D == 128 && jt < np;
            uint8_t* vt = smem + L::kKV + (pos % NS) * L::kTileBytes +
                          (grouped ? (r >> 3) * 2048 + (r & 7) * 128 : r * 128);
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(vt + hb * (grouped ? 1024 : L::kBox) + c * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (idle) {
          tc::fence_before();
          mbar_arrive(&bars[L::P_FULL + u % 3]);
          return;
        }
        // P with the running maximum, which usually stands (O is rescaled only
        // when a score passes it by more than 8 in log2 units), and the tile's
        // maximum, from one read of S in chunks of up to 32 scores
        constexpr int CH = NC < 32 ? NC : 32;
        uint32_t pk[NC / 2];
        float rs = 0.f, m_tile = -INFINITY;
        auto scores = [&](auto want_max, auto want_p) {
          const float mu = m_run == -INFINITY ? 0.f : m_run;
          const float2 c_sl2 = make_float2(sl2, sl2), c_m = make_float2(-mu, -mu);
          float2 rs2 = make_float2(0.f, 0.f), rs3 = make_float2(0.f, 0.f);
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < NC / CH; ++c) {
            float sv[CH];
            if constexpr (CH == 16) tc::ld16f(sc + k0 + CH * c, sv); else tc::ld32f(sc + k0 + CH * c, sv);
            tc::wait_ld();
            if (masked) {
#pragma unroll
              for (int e = 0; e < CH; ++e) sv[e] = (seen >> (CH * c + e)) & 1ull ? sv[e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < CH / 2; ++e) {
              if (decltype(want_max)::value) m4[e & 3] = max3(m4[e & 3], sv[2 * e], sv[2 * e + 1]);
              if (decltype(want_p)::value) {
                const float2 y = __ffma2_rn(make_float2(sv[2 * e], sv[2 * e + 1]), c_sl2, c_m);
                const float2 p = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                if (e & 1) rs3 = __fadd2_rn(rs3, p); else rs2 = __fadd2_rn(rs2, p);
                pk[CH / 2 * c + e] = pack_bf16x2(p.x, p.y);
              }
            }
          }
          if (decltype(want_max)::value)
            m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
          rs2 = __fadd2_rn(rs2, rs3);
          rs = rs2.x + rs2.y;
        };
        if (j > 0) scores(std::true_type(), std::true_type());
        else scores(std::true_type(), std::false_type());
        // The two threads of a lane agree.  (The vote is also what lets the
        // second one write its P over scores that the first has read.)
        const bool need = !dead && m_tile > m_run + kRescaleLog2;
        if (bar_vote_or(3 + qr, 64, need || j == 0 || !pair.ok())) {
          ml[hf * kTile + r] = make_float2(m_tile, pair.ok() ? 1.f : 0.f);
          asm volatile("bar.sync %0, 64;" ::"r"(3 + qr) : "memory");
          const float2 other = ml[(hf ^ 1) * kTile + r];
          if (!pair.meet(__all_sync(0xffffffffu, other.y != 0.f))) return;
          const float m_row = fmaxf(m_tile, other.x);
          const float m_new = !dead && m_row > m_run + kRescaleLog2 ? m_row : m_run;
          if (j > 0) {
            pair.waited(mbar_wait_warp(&bars[L::O_FULL + ((u - 1) & 1)], ((u - 1) >> 1) & 1, abort_flag));
            tc::fence_after();
            const float f = (m_new > m_run && m_run != -INFINITY) ? exp2_approx(m_run - m_new) : 1.f;
            l_run *= f;
#pragma unroll 1
            for (int c = hf * (D / 64); c < (hf + 1) * (D / 64); ++c) {
              float o[32];
              tc::ld32f(lanes + 384u + 32 * c, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tc::st32f(lanes + 384u + 32 * c, o);
            }
          }
          m_run = m_new;
          scores(std::false_type(), std::true_type());
          asm volatile("bar.sync %0, 64;" ::"r"(3 + qr) : "memory");   // (as the vote)
        }
        l_run += rs;
        // keys [64 hf, 64 hf + 64) of P: this copy's, and zeros
        const uint32_t pc = sc + 32u * hf;
        if constexpr (NC == 64) {
          tc::st16(pc, pk);
          tc::st16(pc + 16, pk + 16);
        } else {
          constexpr int W = NC / 2;
#pragma unroll
          for (int c = 0; c < 64 / NC; ++c) {
            uint32_t x[W];
#pragma unroll
            for (int e = 0; e < W; ++e) x[e] = c == copy ? pk[e] : 0u;
            if constexpr (W == 16) tc::st16(pc + 16 * c, x); else st8(pc + 8 * c, x);
          }
        }
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&bars[L::P_FULL + u % 3]);
      };
      for (int j = 0; pair.more(j, n); ++j) {
        const int jt = s.j0 + j;                           // tile of the unit
        const int valid = jt < np ? s.L - jt * kTile : s.nb - (jt - np) * kTile;
        if (jt >= np || valid < kTile) tile(std::true_type(), j, jt, valid);
        else tile(std::false_type(), j, jt, valid);
      }
      // ---- segment end
      asm volatile("bar.sync %0, 64;" ::"r"(3 + qr) : "memory");   // (maxima of the last vote read)
      ml[hf * kTile + r] = make_float2(m_run, l_run);
      if (pair.ok()) {
        const int u = u0 + n - 1;
        pair.waited(mbar_wait_warp(&bars[L::O_FULL + (u & 1)], (u >> 1) & 1, abort_flag));
      }
      // (also orders the exchange; every softmax thread leaves on the same vote)
      if (bar_vote_or(2, 256, !pair.ok())) break;
      tc::fence_after();
      float m = -INFINITY, l = 0.f;
      for (int c = 0; c < copies; ++c) m = fmaxf(m, ml[c * per_copy * 32 + lr].x);
      for (int c = 0; c < copies; ++c) {
        const float2 x0 = ml[c * per_copy * 32 + lr], x1 = ml[kTile + c * per_copy * 32 + lr];
        const float lc = x0.y + x1.y;
        l += x0.x == -INFINITY ? 0.f * lc : lc * exp2_approx(x0.x - m);   // (a NaN stays one)
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float f = (m_run == -INFINITY ? 0.f : exp2_approx(m_run - m)) * inv;
      const bool direct = (s.flags & 2) != 0;
      const int slot = 2 * blockIdx.x + ((s.flags & 1) ? 0 : 1);
      const size_t orow = ((size_t)s.b * t.Hq + (size_t)s.h * a.G + head) * t.Nq + node;
      const size_t prow = (size_t)slot * a.RP + lr;
      // the copies are added up through this segment's Q tile, which its MMAs
      // have read: [half][copy of a pair][32 columns][lanes of a copy]
      float* ex = reinterpret_cast<float*>(smem + L::kQ + (qt & 1) * L::kTileBytes) +
                  hf * (L::kTileBytes / 8) + lr;
      constexpr int span = per_copy * 32;
#pragma unroll 1
      for (int c = hf * (D / 64); c < (hf + 1) * (D / 64); ++c) {   // half of the columns
        float o[32];
        if (!idle) {
          tc::ld32f(lanes + 384u + 32 * c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
        }
        for (int half = copies >> 1; half > 0; half >>= 1) {
          float* x = ex + (copy & (half - 1)) * 32 * span;
          if (copy >= half && copy < 2 * half) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e * span] = o[e];
          }
          asm volatile("bar.sync %0, 128;" ::"r"(7 + hf) : "memory");
          if (copy < half) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] += x[e * span];
          }
          asm volatile("bar.sync %0, 128;" ::"r"(7 + hf) : "memory");
        }
        const bool store = copy == 0 && !dead;
        if (store && direct) {
          __nv_bfloat16* dst = t.o + orow * D + 32 * c;
          uint4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q].x = pack_bf16x2(o[8 * q + 0], o[8 * q + 1]);
            v[q].y = pack_bf16x2(o[8 * q + 2], o[8 * q + 3]);
            v[q].z = pack_bf16x2(o[8 * q + 4], o[8 * q + 5]);
            v[q].w = pack_bf16x2(o[8 * q + 6], o[8 * q + 7]);
          }
          if (o_32B) {
            st_global_32B(dst, v[0], v[1]);
            st_global_32B(dst + 16, v[2], v[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(dst + 8 * q) = v[q];
          }
        } else if (store) {
          float* dst = a.part_o + prow * D + 32 * c;
          auto u4 = [&](int q) {
            return make_uint4(__float_as_uint(o[4 * q]), __float_as_uint(o[4 * q + 1]),
                              __float_as_uint(o[4 * q + 2]), __float_as_uint(o[4 * q + 3]));
          };
#pragma unroll
          for (int q = 0; q < 4; ++q) st_global_32B(dst + 8 * q, u4(2 * q), u4(2 * q + 1));
        }
        __syncwarp();
      }
      if (copy == 0 && !dead && hf == 0) {
        const float lse = l == 0.f ? -INFINITY : m + __log2f(l);
        if (!direct) a.part_lse[prow] = lse;
        else if (t.lse) t.lse[orow] = lse * kLn2;
      }
      tc::fence_before();
      // the exchange went through the Q tile, which TMA may fill next
      if constexpr (kCopies > 1) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::Q_EMPTY + (qt & 1)]);
      g += 2 * n;
      u0 += n;
      ++qt;
      live = next_seg(k, s);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int sl = warp >> 2;                 // slot
    const int r = (warp & 3) * 32 + lane;     // row of the slot = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_off + 128u * sl;
    const uint32_t ocol = tmem + lane_off + 256u + (uint32_t)D * sl;
    const float sl2 = t.scale_log2;
    const bool o_32B = (reinterpret_cast<uintptr_t>(t.o) & 31) == 0;
    float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
    int k = 0, g = 0, sw = 0, ow0 = 0, ow1 = 0;
    bool ok = true;
    Seg s;
    // a failed read of the ring is voted on below like any other failure
    bool live = next_seg(k, s);
    while (!bar_vote_or(1, 256, !live)) {
      const int rows = group_rows(s), n = s.n, np = s.np();
      const bool pair = rows > kTile;
      const int lr = pair ? sl * kTile + r : r;          // row within the group
      const int warp_row = lr - lane;
      const bool idle = warp_row >= rows;                // no live row in this warp
      const bool dead = lr >= rows;                      // computes on anything, is not stored
      float m_run = -INFINITY, l_run = 0.f;
      // a small tree's parents, asked for here and looked at on its tile
      const bool small = s.nb <= 32;
      int parent = -1;
      if (small && s.j0 + n > np && lane < s.nb) parent = t.parents[(size_t)s.b * t.Nq + lane];
      const int steps = pair ? n : (n + 1 - sl) / 2;
      auto rescale = [&](int x, bool need, float m_tile) {
        const float m_new = need ? m_tile : m_run;
        if (x > 0) {
          const float f = (need && m_run != -INFINITY) ? exp2_approx(m_run - m_new) : 1.f;
          l_run *= f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::ld32f(ocol + 32 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tc::st32f(ocol + 32 * c, o);
          }
        }
        m_run = m_new;
      };
      for (int x = 0; x < steps; ++x) {
        const int j = pair ? x : 2 * x + sl;
        const int jt = s.j0 + j;                         // tile of the unit
        // keys of the tile that exist; the rest are masked, and their values
        // cleared, as anything may be stored there
        const int valid = jt < np ? s.L - jt * kTile : s.nb - (jt - np) * kTile;
        uint32_t bits[4] = {0u, 0u, 0u, 0u};
        const bool masked = jt >= np || valid < kTile;
        if (masked && !idle) {
          if (jt < np) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int e = valid - 32 * c;
              bits[c] = e >= 32 ? 0xffffffffu : (e <= 0 ? 0u : (1u << e) - 1u);
            }
          } else if (small) {
            const int node = (s.rg * 2 * kTile + (dead ? rows - 1 : lr)) % s.nb;
            bits[0] = __shfl_sync(0xffffffffu, ancestors32(parent, lane), node);
          } else {
            // the node and its ancestors among drafts [base, base + 128)
            const int base = (jt - np) * kTile;
            const int32_t* par = t.parents + (size_t)s.b * t.Nq;
            int v = (s.rg * 2 * kTile + (dead ? rows - 1 : lr)) % s.nb;
            while (v >= base) {
              const int e = v - base;
              if (e < kTile) {
                const uint32_t bit = 1u << (e & 31);
#pragma unroll
                for (int c = 0; c < 4; ++c) bits[c] |= (e >> 5) == c ? bit : 0u;
              }
              const int p = par[v];
              if (p < -1 || p >= v) {
                atomicExch(&g_device_status, (int)ATTN_ERANGE);
                break;
              }
              v = p;
            }
          }
        }
        if (!mbar_wait_warp(&bars[L::S_FULL + sl], sw & 1, abort_flag)) { ok = false; break; }
        ++sw;
        tc::fence_after();
        if (valid < kTile && (!pair || sl == 0)) {
          // (a pair's second product on this tile is issued after the first,
          // which waits for this slot's P)
          const int pos = v_pos(g, j, n, pair);
          if (!mbar_wait_warp(&bars[L::FULL + pos % NS], (pos / NS) & 1, abort_flag)) { ok = false; break; }
          if (r >= valid) {
            const bool grouped = kPaged && D == 128 && jt < np;
            uint8_t* vt = smem + L::kKV + (pos % NS) * L::kTileBytes +
                          (grouped ? (r >> 3) * 2048 + (r & 7) * 128 : r * 128);
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(vt + hb * (grouped ? 1024 : L::kBox) + c * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (idle) {
          tc::fence_before();
          mbar_arrive(&bars[L::P_FULL + sl]);
          continue;
        }
        // An unmasked tile: two passes over S in halves, one for the tile's
        // maximum, one for P with the running maximum, which usually stands (O
        // is rescaled only when a live row of the warp passes it by more than 8
        // in log2 units).  Nothing of S is held across the passes: there are no
        // registers for it.  (The branch is on what the whole warp shares:
        // tcgen05 moves are warp-wide.)
        if (!masked) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float sv[64];
            tc::ld32f(scol + 64 * c, sv);
            tc::ld32f(scol + 64 * c + 32, sv + 32);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) m4[e & 3] = max3(m4[e & 3], sv[2 * e], sv[2 * e + 1]);
          }
          const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
          const bool need = !dead && m_tile > m_run + kRescaleLog2;
          if (__any_sync(0xffffffffu, need)) rescale(x, need, m_tile);
          const float mu = m_run == -INFINITY ? 0.f : m_run;
          const float2 c_sl2 = make_float2(sl2, sl2), c_m = make_float2(-mu, -mu);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float sv[64];
            uint32_t pk[32];
            tc::ld32f(scol + 64 * c, sv);
            tc::ld32f(scol + 64 * c + 32, sv + 32);
            tc::wait_ld();
            float2 rs2 = make_float2(0.f, 0.f), rs3 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 y = __ffma2_rn(make_float2(sv[2 * e], sv[2 * e + 1]), c_sl2, c_m);
              const float2 p = make_float2(exp2_approx(y.x), exp2_approx(y.y));
              if (e & 1) rs3 = __fadd2_rn(rs3, p); else rs2 = __fadd2_rn(rs2, p);
              pk[e] = pack_bf16x2(p.x, p.y);
            }
            rs2 = __fadd2_rn(rs2, rs3);
            l_run += rs2.x + rs2.y;
            tc::st16(scol + 32 * c, pk);
            tc::st16(scol + 32 * c + 16, pk + 16);
          }
          tc::wait_st();
          tc::fence_before();
          mbar_arrive(&bars[L::P_FULL + sl]);
          continue;
        }
        // A masked tile: two passes over S in chunks of 32 keys; a chunk that no
        // row of the warp sees is skipped.
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t w = c == 0 ? bits[0] : c == 1 ? bits[1] : c == 2 ? bits[2] : bits[3];
          if (!__any_sync(0xffffffffu, w != 0u)) continue;
          float sv[32];
          tc::ld32f(scol + 32 * c, sv);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, (w >> e) & 1u ? sv[e] : -INFINITY);
        }
        const float m_tile = mx * sl2;
        const bool need = !dead && m_tile > m_run + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) rescale(x, need, m_tile);
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        float rs = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t w = c == 0 ? bits[0] : c == 1 ? bits[1] : c == 2 ? bits[2] : bits[3];
          uint32_t pk[16];
          if (!__any_sync(0xffffffffu, w != 0u)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0u;
          } else {
            float sv[32];
            tc::ld32f(scol + 32 * c, sv);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float x0 = (w >> (2 * e)) & 1u ? sv[2 * e] : -INFINITY;
              const float x1 = (w >> (2 * e + 1)) & 1u ? sv[2 * e + 1] : -INFINITY;
              const float p0 = exp2_approx(fmaf(x0, sl2, -m_use));
              const float p1 = exp2_approx(fmaf(x1, sl2, -m_use));
              rs += p0 + p1;
              pk[e] = pack_bf16x2(p0, p1);
            }
          }
          tc::st16(scol + 16 * c, pk);
        }
        l_run += rs;
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&bars[L::P_FULL + sl]);
      }
      // ---- segment end
      if (!pair) ml[sl * kTile + r] = make_float2(m_run, l_run);
      // (also orders the exchange; every softmax thread leaves on the same vote)
      if (bar_vote_or(2, 256, !ok)) break;
      float f0 = 0.f, f1 = 0.f, m = m_run, l = l_run;
      const bool two = !pair && n > 1;                   // slot 1 took part as well
      if (!pair) {
        const float2 x0 = ml[r], x1 = ml[kTile + r];
        m = fmaxf(x0.x, x1.x);
        const float w0 = x0.x == -INFINITY ? 0.f : exp2_approx(x0.x - m);
        const float w1 = x1.x == -INFINITY ? 0.f : exp2_approx(x1.x - m);
        l = x0.y * w0 + x1.y * w1;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f0 = w0 * inv;
        f1 = w1 * inv;
      } else {
        f0 = l == 0.f ? 0.f : 1.f / l;   // (a NaN among the scores stays one)
      }
      if (!pair || sl == 0) {
        if (!mbar_wait_warp(&bars[L::O_FULL], ow0 & 1, abort_flag)) ok = false;
      }
      if (two || (pair && sl == 1)) {
        if (!mbar_wait_warp(&bars[L::O_FULL + 1], ow1 & 1, abort_flag)) ok = false;
      }
      ++ow0;
      if (two || pair) ++ow1;
      tc::fence_after();
      const bool direct = (s.flags & 2) != 0;
      const int slot = 2 * blockIdx.x + ((s.flags & 1) ? 0 : 1);
      const bool store = !dead;
      const int rr = s.rg * 2 * kTile + (dead ? rows - 1 : lr), head = rr / s.nb;
      const size_t orow =
          ((size_t)s.b * t.Hq + (size_t)s.h * a.G + head) * t.Nq + (rr - head * s.nb);
      const size_t prow = (size_t)slot * a.RP + lr;
      // pair: all columns of the own slot; else half of the columns of both
      const uint32_t oa = tmem + lane_off + 256u + (pair ? (uint32_t)D * sl : 0u);
      const int c_lo = pair ? 0 : sl * (D / 64), c_hi = pair ? D / 32 : (sl + 1) * (D / 64);
      if (!idle) {
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          float o[32];
          tc::ld32f(oa + 32 * c, o);
          if (two) {
            float o1[32];
            tc::ld32f(oa + D + 32 * c, o1);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
          } else {
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f0;
          }
          if (store && direct) {
            __nv_bfloat16* dst = t.o + orow * D + 32 * c;
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q].x = pack_bf16x2(o[8 * q + 0], o[8 * q + 1]);
              v[q].y = pack_bf16x2(o[8 * q + 2], o[8 * q + 3]);
              v[q].z = pack_bf16x2(o[8 * q + 4], o[8 * q + 5]);
              v[q].w = pack_bf16x2(o[8 * q + 6], o[8 * q + 7]);
            }
            if (o_32B) {
              st_global_32B(dst, v[0], v[1]);
              st_global_32B(dst + 16, v[2], v[3]);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(dst + 8 * q) = v[q];
            }
          } else if (store) {
            float* dst = a.part_o + prow * D + 32 * c;
            auto u4 = [&](int q) {
              return make_uint4(__float_as_uint(o[4 * q]), __float_as_uint(o[4 * q + 1]),
                                __float_as_uint(o[4 * q + 2]), __float_as_uint(o[4 * q + 3]));
            };
#pragma unroll
            for (int q = 0; q < 4; ++q) st_global_32B(dst + 8 * q, u4(2 * q), u4(2 * q + 1));
          }
        }
      }
      if (store && (pair || sl == 0)) {
        const float lse = l == 0.f ? -INFINITY : m + __log2f(l);
        if (!direct) a.part_lse[prow] = lse;
        else if (t.lse) t.lse[orow] = lse * kLn2;
      }
      tc::fence_before();
      g += 2 * n;
      // both slots' O have been read before either slot's next P is released
      // (the vote at the loop's head)
      live = ok && next_seg(k, s);
    }
  }

  tc::fence_before();
  __syncthreads();
  // every load must have landed before the CTA may exit (they all have, unless
  // a wait gave up)
  if (warp == 9 && lane < NS && armed[lane] >= 0)
    mbar_wait(&bars[L::FULL + lane], (armed[lane] / NS) & 1, nullptr);
  if (warp == 10 && lane < 2 && armed[NS + lane] >= 0)
    mbar_wait(&bars[L::Q_FULL + lane], (armed[NS + lane] >> 1) & 1, nullptr);
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// Joins the partial results of the units that cross a cut: blockIdx.x = the
// range in which the unit starts, blockIdx.y = a chunk of its rows, 4 rows a
// warp.  Four parts at a time, in the order of the keys: all their columns are
// asked for first, then a lane loads the log-sum-exp of one (part, row) and
// makes its weight under a running maximum.  Bound by latency (the record, then
// the partial results, then the store) and, with 256 rows, by how many partial
// results (up to 128 KB a part, out of L2) are on their way at once.
constexpr int kJoinWarps = 4, kJoinRows = 4, kJoinParts = 4;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) tree_join_kernel(tr::Args a) {
  using namespace tr;
  constexpr int E = D / 32;
  const TreeArgs& t = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x, r0 = (blockIdx.y * kJoinWarps + warp) * kJoinRows;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Record u = a.records[c0];
  if (u.last < 0 || r0 >= u.rows) return;
  const int nr = u.rows - r0 < kJoinRows ? u.rows - r0 : kJoinRows;
  const Cuts cuts(u.T, a);
  const int lp = lane / kJoinRows, lr = lane % kJoinRows;   // this lane's part and row of a batch
  float m = -INFINITY, sum = 0.f;      // of row lr, the same in every lane group
  float acc[kJoinRows][E];
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
  for (int base = c0; base <= u.last; base += 32) {
    // ranges that hold a tile of the unit (a short one may hold none)
    const int c = base + lane;
    bool has = c <= u.last;
    if (has && c > c0)
      has = tiles_before(cuts.at(c + 1) - u.p0, u.w, u.nt, a.cost_unit) > tiles_before(cuts.at(c) - u.p0, u.w, u.nt, a.cost_unit);
    unsigned bal = __ballot_sync(0xffffffffu, has);
    while (bal) {
      const int n = __popc(bal) < kJoinParts ? __popc(bal) : kJoinParts;
      float v[kJoinParts][kJoinRows][E];
      int ms = 0;
#pragma unroll
      for (int k = 0; k < kJoinParts; ++k) {
        const int ci = base + __ffs(bal) - 1;
        bal &= bal - 1;
        const int slot = ci == c0 ? u.slot : 2 * ci;
        ms = lp == k ? slot : ms;
        const float* src = a.part_o + ((size_t)slot * a.RP + r0) * D + lane * E;
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
          const bool ld = k < n && i < nr;
          if constexpr (E == 4)
            *reinterpret_cast<float4*>(v[k][i]) =
                ld ? *reinterpret_cast<const float4*>(src + i * D) : make_float4(0.f, 0.f, 0.f, 0.f);
          else
            *reinterpret_cast<float2*>(v[k][i]) =
                ld ? *reinterpret_cast<const float2*>(src + i * D) : make_float2(0.f, 0.f);
        }
      }
      const float ls = lp < n && lr < nr ? a.part_lse[(size_t)ms * a.RP + r0 + lr] : -INFINITY;
      float mx = fmaxf(m, ls);
#pragma unroll
      for (int o = kJoinRows; o < kJoinRows * kJoinParts; o <<= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float f = m == -INFINITY ? 0.f : exp2_approx(m - mx);
      const float w = ls == -INFINITY ? 0.f : exp2_approx(ls - mx);
      float ws = w;
#pragma unroll
      for (int o = kJoinRows; o < kJoinRows * kJoinParts; o <<= 1)
        ws += __shfl_xor_sync(0xffffffffu, ws, o);
      sum = sum * f + ws;
      m = mx;
#pragma unroll
      for (int i = 0; i < kJoinRows; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] *= fi;
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) {
          const float wi = __shfl_sync(0xffffffffu, w, k * kJoinRows + i);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[i][e] = fmaf(wi, v[k][i][e], acc[i][e]);
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int rr = u.rg * 2 * kTile + r0;
  int head = rr / u.nb, node = rr - head * u.nb;
  const size_t unit = (size_t)u.b * t.Hq + (size_t)u.h * a.G;
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) {
    const float fi = __shfl_sync(0xffffffffu, inv, i);
    if (i < nr) {
      const size_t row = (unit + head) * t.Nq + node;
      uint32_t* o = reinterpret_cast<uint32_t*>(t.o + row * D + lane * E);
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[i][0] * fi, acc[i][1] * fi),
                                                  pack_bf16x2(acc[i][2] * fi, acc[i][3] * fi));
      else
        *o = pack_bf16x2(acc[i][0] * fi, acc[i][1] * fi);
      if (t.lse && lane == i) t.lse[row] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
    }
    if (++node == u.nb) {
      node = 0;
      ++head;
    }
  }
}

// ------------------------------------------------------------------ host side

bool tree_supported(int B, int Nq, int d) {
  return (d == 64 || d == 128) && Nq <= 1024 && B <= tr::kMaxB;
}

namespace {
int rows_per_slot(int Hq, int Hkv, int Nq) {
  const long long rows = (long long)(Hq / Hkv) * Nq;
  return rows < 2 * tr::kTile ? (int)rows : 2 * tr::kTile;
}
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

template <int D, bool kPaged, int kKeys>
int launch_tree_k(const tr::Args& a, const CUtensorMap& tk, const CUtensorMap& tv,
                  const CUtensorMap& tkn, const CUtensorMap& tvn, cudaStream_t st) {
  auto kern = tree_tc_kernel<D, kPaged, kKeys>;
  constexpr int smem = tr::Smem<D>::kTotal;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return ATTN_ECUDA;
  // q as [B * Hkv, rows of a kv head, d], in boxes of one copy's rows
  CUtensorMap tq;
  if (make_tmap_3d_bf16(&tq, a.t.q, D, (uint64_t)a.G * a.t.Nq, (uint64_t)a.t.B * a.t.Hkv, 64,
                        kKeys == 0 ? tr::kTile : 2 * kKeys) != ATTN_OK)
    return ATTN_ECUDA;
  const int rc = launch_programmatic(kern, dim3(a.grid), dim3(tr::threads(kKeys == 0)), smem, st, tq, tk, tv, tkn,
                                     tvn, a);
  if (rc != ATTN_OK) return rc;
  constexpr int HB = kJoinWarps * kJoinRows;
  return launch_programmatic(tree_join_kernel<D>, dim3(a.ranges, (a.RP + HB - 1) / HB),
                             dim3(kJoinWarps * 32), 0, st, a);
}

template <int D, bool kPaged>
int launch_tree_t(const tr::Args& a, const CUtensorMap& tk, const CUtensorMap& tv,
                  const CUtensorMap& tkn, const CUtensorMap& tvn, cudaStream_t st) {
  // how many keys of a tile's half a thread takes: the fewer rows, the more
  // copies of them the 128 lanes hold
  if (a.RP > 128) return launch_tree_k<D, kPaged, 0>(a, tk, tv, tkn, tvn, st);
  if (a.RP > 64) return launch_tree_k<D, kPaged, 64>(a, tk, tv, tkn, tvn, st);
  if (a.RP > 32) return launch_tree_k<D, kPaged, 32>(a, tk, tv, tkn, tvn, st);
  return launch_tree_k<D, kPaged, 16>(a, tk, tv, tkn, tvn, st);
}
}  // namespace

size_t tree_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int num_sms) {
  (void)B;
  const size_t rp = (size_t)rows_per_slot(Hq, Hkv, Nq), slots = 2 * (size_t)num_sms;
  return round256(slots * rp * d * sizeof(float)) + round256(slots * rp * sizeof(float)) +
         round256((size_t)num_sms * sizeof(tr::Record));
}

int launch_tree(const TreeArgs& t, int d, void* workspace, int num_sms, cudaStream_t st) {
  tr::Args a;
  a.t = t;
  a.G = t.Hq / t.Hkv;
  a.RP = rows_per_slot(t.Hq, t.Hkv, t.Nq);
  a.grid = num_sms;
  const size_t slots = 2 * (size_t)num_sms;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(w);
  w += round256(slots * a.RP * d * sizeof(float));
  a.part_lse = reinterpret_cast<float*>(w);
  w += round256(slots * a.RP * sizeof(float));
  a.records = reinterpret_cast<tr::Record*>(w);
  a.ranges = num_sms;
  a.cost_unit = tr::unit_cost(a.RP);
  // the drafts [B * Hkv, Nq, d] and a contiguous cache [B * Hkv, Nk, d] in
  // boxes of 128 rows x 64 columns; a paged cache page by page
  CUtensorMap tk, tv, tkn, tvn;
  const uint64_t mats = (uint64_t)t.B * t.Hkv;
  if (make_tmap_3d_bf16(&tkn, t.kn, d, t.Nq, mats, 64, tr::kTile) != ATTN_OK) return ATTN_ECUDA;
  if (make_tmap_3d_bf16(&tvn, t.vn, d, t.Nq, mats, 64, tr::kTile) != ATTN_OK) return ATTN_ECUDA;
  a.oob_row = 0;
  if (!t.block_table) {
    if (make_tmap_3d_bf16(&tk, t.kc, d, t.Nk, mats, 64, tr::kTile) != ATTN_OK) return ATTN_ECUDA;
    if (make_tmap_3d_bf16(&tv, t.vc, d, t.Nk, mats, 64, tr::kTile) != ATTN_OK) return ATTN_ECUDA;
    return d == 128 ? launch_tree_t<128, false>(a, tk, tv, tkn, tvn, st)
                    : launch_tree_t<64, false>(a, tk, tv, tkn, tvn, st);
  }
  const uint64_t rows = (uint64_t)t.num_pages * t.Hkv * t.page_size;
  a.oob_row = (int)rows;
  if (d == 128) {
    const uint32_t groups = (uint32_t)t.page_size / 8;
    if (make_tmap_grouped_bf16(&tk, t.kc, rows, groups) != ATTN_OK) return ATTN_ECUDA;
    if (make_tmap_grouped_bf16(&tv, t.vc, rows, groups) != ATTN_OK) return ATTN_ECUDA;
    return launch_tree_t<128, true>(a, tk, tv, tkn, tvn, st);
  }
  const uint32_t ps = (uint32_t)t.page_size;
  if (make_tmap_2d_bf16(&tk, t.kc, d, rows, 64, ps) != ATTN_OK) return ATTN_ECUDA;
  if (make_tmap_2d_bf16(&tv, t.vc, d, rows, 64, ps) != ATTN_OK) return ATTN_ECUDA;
  return launch_tree_t<64, true>(a, tk, tv, tkn, tvn, st);
}

}  // namespace attn
