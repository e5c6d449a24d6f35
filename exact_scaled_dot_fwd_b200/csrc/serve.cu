// serve.cu -- the passes around attention over a paged cache: the page plan
// of a step (block tables and slot maps from request lengths) and the append
// of new keys and values, rotated at their own positions.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope_math.cuh"
#include "tile_plan.cuh"

namespace attn {

// ------------------------------------------------------------------ page plan
//
// With h(x) = ceil(x / page_size), sequence b takes a_b = max(0, h(new) -
// h(old)) pages and gives back the r_b pages among its table entries [h(new),
// h(old)): an entry outside [0, num_pages) -- one that got no page in a
// shortage -- is none.  Its pages are the queue's entries A_b .. A_b + a_b - 1
// with A_b = sum_{c < b} a_c (r likewise at the tail), so every entry and slot
// has a closed form once the two prefix sums are known, and nothing has to be
// exchanged between CTAs: each one sums the lengths below its own sequences
// again (8 bytes per sequence, out of L2) instead of waiting for a scan kernel.
// Only the CTAs whose own sequences shrink, and the one that writes the state,
// also look through the entries that the sequences below give back.
//
// Bound by launch latency: the whole step is a few KB to a few MB (256 decode
// steps 5.5 us, 32 prompts of 8192 tokens 6.6 us).  Where very many pages come
// back at once, by the one CTA that looks through all of them (683 of 2048
// requests finished, 1.0 M pages: 121 us).

namespace {
constexpr int kPlanAhead = 2;      // sequences of a thread whose lengths are on their way together
constexpr int kPlanMaxS = 64;      // sequences per CTA
constexpr int kPlanItems = 1024;   // slots per CTA, about
}  // namespace

struct PlanArgs {
  const int32_t* old_lens;
  const int32_t* new_lens;
  int32_t* table;
  int32_t* ring;
  const int32_t* state_in;
  int32_t* state_out;
  const int32_t* index;
  int32_t* slots;
  int B, N, max_pages, page_size, num_pages;
  int S;        // sequences per CTA
  int chunks;   // CTAs per sequence group (S == 1 when above 1)
};

struct PlanSeq {
  int o, n;      // old and new length
  int ho, hn;    // pages held before and after
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int b) {
  PlanSeq s;
  const int cap = a.max_pages * a.page_size;
  s.o = clamp_len(a.old_lens[b], cap);
  s.n = clamp_len(a.new_lens[b], cap);
  // (both terms are below 2^31)
  s.ho = (int)(((unsigned)s.o + (unsigned)a.page_size - 1u) / (unsigned)a.page_size);
  s.hn = (int)(((unsigned)s.n + (unsigned)a.page_size - 1u) / (unsigned)a.page_size);
  return s;
}

// How many of the table entries [lo, hi) of a row are pages: the share of lane
// `i` of `n` (at least 4), in 16-byte loads between the row's odd ends.
__device__ __forceinline__ int pages_among(const int32_t* row, int lo, int hi, int i, int n,
                                           int num_pages) {
  const int32_t* p = row + lo;
  const int len = hi > lo ? hi - lo : 0;
  int head = (int)((0u - (unsigned)(reinterpret_cast<uintptr_t>(p) >> 2)) & 3u);
  if (head > len) head = len;
  const int whole = (len - head) >> 2, tail = head + 4 * whole;
  auto is_page = [&](int e) { return (unsigned)e < (unsigned)num_pages ? 1 : 0; };
  int c = 0;
  if (i < head) c += is_page(p[i]);
  if (i < len - tail) c += is_page(p[tail + i]);
  const int4* q = reinterpret_cast<const int4*>(p + head);
#pragma unroll 4
  for (int j = i; j < whole; j += n) {
    const int4 e = q[j];
    c += is_page(e.x) + is_page(e.y) + is_page(e.z) + is_page(e.w);
  }
  return c;
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs a) {
  constexpr int kPlanWarps = kPlanThreads / 32;
  __shared__ long long s_red[2][kPlanWarps];
  __shared__ PlanSeq s_seq[kPlanMaxS];
  __shared__ long long s_take[kPlanMaxS], s_give[kPlanMaxS];
  __shared__ int s_pages[kPlanMaxS];   // pages that a unit gives back
  __shared__ long long s_all[2];       // taken and given back up to and with this CTA's sequences
  __shared__ int s_list[3][kPlanThreads * kPlanAhead], s_listed;   // sequences that shrink
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = blockIdx.x / a.chunks, chunk = blockIdx.x - grp * a.chunks;
  const int b0 = grp * a.S;
  const int S = a.B - b0 < a.S ? a.B - b0 : a.S;
  const bool last = b0 + S == a.B && chunk == 0;   // this CTA also writes the queue's new state
  const int P = a.num_pages;

  PlanSeq below[kPlanAhead];
  auto load_below = [&](unsigned base) {   // (unsigned: B may be just below 2^31)
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i) {
      const unsigned b = base + i * kPlanThreads + tid;
      below[i] = {0, 0, 0, 0};
      if (b < (unsigned)b0) below[i] = plan_seq(a, (int)b);
    }
  };
  load_below(0);
  bool shrinks = false;
  if (tid < S) {
    const PlanSeq s = plan_seq(a, b0 + tid);
    s_seq[tid] = s;
    shrinks = s.ho > s.hn;
  }
  if (tid == 0) s_listed = 0;
  // (a group's first chunk gives back for all of them)
  const bool gives = __syncthreads_or(shrinks) && chunk == 0;

  // pages taken and given back by the sequences below b0: those that shrink
  // are listed and looked through by 8 lanes each
  long long tk = 0, gv = 0;
  for (unsigned base = 0; base < (unsigned)b0;) {
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i) {
      const PlanSeq s = below[i];
      if (s.hn > s.ho) tk += s.hn - s.ho;
      if ((gives || last) && s.ho > s.hn) {
        const int at = atomicAdd(&s_listed, 1);
        s_list[0][at] = (int)(base + i * kPlanThreads + tid);
        s_list[1][at] = s.hn;
        s_list[2][at] = s.ho;
      }
    }
    base += kPlanThreads * kPlanAhead;
    if (base < (unsigned)b0) load_below(base);
    if (gives || last) {
      __syncthreads();
      const int n = s_listed;
      for (int i = tid >> 3; i < n; i += kPlanThreads / 8)
        gv += pages_among(a.table + (size_t)s_list[0][i] * a.max_pages, s_list[1][i], s_list[2][i],
                          lane & 7, 8, P);
      __syncthreads();
      if (tid == 0) s_listed = 0;
      __syncthreads();
    }
  }
  tk = warp_sum(tk); gv = warp_sum(gv);
  if (lane == 0) { s_red[0][warp] = tk; s_red[1][warp] = gv; }

  // What this CTA's own sequences give back, in units of a sequence (of a part
  // of one for every warp where a CTA has a single sequence), a warp each.
  const int parts = a.S > 1 ? 1 : kPlanWarps;
  const int units = S * parts;
  auto unit_lo = [&](const PlanSeq& q, int k) -> int {   // first entry of its k-th part
    return q.hn + (int)((long long)(q.ho - q.hn) * k / parts);
  };
  for (int u = warp; u < units; u += kPlanWarps) {
    const int s = a.S > 1 ? u : 0, k = u - s * parts;
    const PlanSeq q = s_seq[s];
    int c = 0;
    if (gives && q.ho > q.hn)
      c = __reduce_add_sync(0xffffffffu,
                            pages_among(a.table + (size_t)(b0 + s) * a.max_pages, unit_lo(q, k),
                                        unit_lo(q, k + 1), lane, 32, P));
    if (lane == 0) s_pages[u] = c;
  }
  __syncthreads();
  if (warp == 0) {
    long long t0 = 0, g0 = 0;
    for (int w = 0; w < kPlanWarps; ++w) { t0 += s_red[0][w]; g0 += s_red[1][w]; }
    // exclusive scans over this CTA's sequences and units, 32 at a time
    for (int base = 0; base < units; base += 32) {
      const int i = base + lane;
      long long t = 0, g = i < units ? s_pages[i] : 0;
      if (i < S && s_seq[i].hn > s_seq[i].ho) t = s_seq[i].hn - s_seq[i].ho;
      long long xt = t, xg = g;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, xt, o);
        const long long yg = __shfl_up_sync(0xffffffffu, xg, o);
        if (lane >= o) { xt += yt; xg += yg; }
      }
      if (i < S) s_take[i] = t0 + xt - t;
      if (i < units) s_give[i] = g0 + xg - g;
      t0 += __shfl_sync(0xffffffffu, xt, 31);
      g0 += __shfl_sync(0xffffffffu, xg, 31);
    }
    if (lane == 0) { s_all[0] = t0; s_all[1] = g0; }
  }
  __syncthreads();

  // the queue; a state from elsewhere cannot lead outside the ring
  int head = a.state_in[0] % P;
  if (head < 0) head += P;
  const int count = clamp_len(a.state_in[1], P);
  bool bad = false;
  // m-th page taken, or -1
  auto taken = [&](long long m) -> int {
    if (m >= count) return -1;
    return a.ring[(int)((head + m) % P)];
  };

  if (last && tid == 0) {
    const long long t = s_all[0], g = s_all[1];
    const long long served = t < count ? t : count;
    const long long room = P - count;
    const long long back = g < room ? g : room;
    a.state_out[0] = (int)((head + served) % P);
    a.state_out[1] = (int)(count - served + back);
    if (t > count || g > room) bad = true;
  }

  // table entries taken: a warp per sequence (all warps and chunks on the one
  // sequence of a long row)
  const int w0 = a.S > 1 ? warp : 0, wn = a.S > 1 ? kPlanWarps : 1;
  const int l0 = a.S > 1 ? lane : chunk * kPlanThreads + tid;
  const int ln = a.S > 1 ? 32 : a.chunks * kPlanThreads;
  for (int s = w0; s < S; s += wn) {
    const PlanSeq q = s_seq[s];
    int32_t* row = a.table + (size_t)(b0 + s) * a.max_pages;
    // (unsigned: a row may end just below 2^31)
    for (unsigned j = (unsigned)q.ho + l0; j < (unsigned)q.hn; j += ln)
      row[j] = taken(s_take[s] + (j - (unsigned)q.ho));
  }
  // pages given back, in the order of their entries, 128 at a time
  for (int u = gives ? warp : units; u < units; u += kPlanWarps) {
    const int s = a.S > 1 ? u : 0, k = u - s * parts;
    const PlanSeq q = s_seq[s];
    if (q.ho <= q.hn) continue;
    const int32_t* row = a.table + (size_t)(b0 + s) * a.max_pages;
    const int hi = unit_lo(q, k + 1);
    long long m = s_give[u];
    for (long long j = unit_lo(q, k); j < hi; j += 128) {
      int page[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) page[i] = j + 32 * i + lane < hi ? row[j + 32 * i + lane] : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = (unsigned)page[i] < (unsigned)P;
        const unsigned bal = __ballot_sync(0xffffffffu, ok);
        const long long at = m + __popc(bal & ((1u << lane) - 1));
        if (ok && at < P - count) a.ring[(int)(((long long)head + count + at) % P)] = page[i];
        m += __popc(bal);
      }
    }
  }

  // slots
  const int i0 = a.S > 1 ? 0 : chunk * kPlanItems;
  int per = a.N - i0;
  if (a.S == 1 && per > kPlanItems) per = kPlanItems;
  for (int it = tid; it < S * per; it += kPlanThreads) {
    const int s = it / per, i = i0 + (it - s * per);
    const PlanSeq q = s_seq[s];
    const size_t at = (size_t)(b0 + s) * a.N + i;
    const int t = a.index ? a.index[at] : i;
    int slot = -1;
    if (t >= 0 && t < q.n - q.o) {
      const int p = q.o + t;
      const int j = p / a.page_size;
      const int page = j < q.ho ? a.table[(size_t)(b0 + s) * a.max_pages + j]
                                : taken(s_take[s] + (j - q.ho));
      if ((unsigned)page < (unsigned)P) slot = page * a.page_size + (p - j * a.page_size);
      else bad = true;
    }
    a.slots[at] = slot;
  }
  if (bad) atomicExch(&g_device_status, (int)ATTN_ERANGE);
}

int launch_paged_plan(const int32_t* old_lens, const int32_t* new_lens, int32_t* block_table,
                      int32_t* free_pages, const int32_t* state_in, int32_t* state_out,
                      const int32_t* index, int32_t* slots, int B, int N, int max_pages,
                      int page_size, int num_pages, cudaStream_t st) {
  PlanArgs a;
  a.old_lens = old_lens; a.new_lens = new_lens; a.table = block_table; a.ring = free_pages;
  a.state_in = state_in; a.state_out = state_out; a.index = index; a.slots = slots;
  a.B = B; a.N = N; a.max_pages = max_pages; a.page_size = page_size; a.num_pages = num_pages;
  a.S = kPlanItems / N;
  if (a.S < 1) a.S = 1;
  if (a.S > kPlanMaxS) a.S = kPlanMaxS;
  a.chunks = a.S > 1 ? 1 : (N + kPlanItems - 1) / kPlanItems;
  const long long grid = (long long)((B + a.S - 1) / a.S) * a.chunks;
  // Many sequences in few CTAs: more threads for the sums over those below a
  // CTA's own (1000 sequences, one in ten finished: 8.0 us against 12.7 with 256;
  // 256 that decode: 5.6 against 5.9).  Not for a few sequences (8 that decode:
  // 4.5 us against 3.7), nor for more CTAs than SMs: with 1024 threads of 64
  // registers an SM holds one (600 prompts of 300 tokens: 9.4 us against 6.5).
  return B > 32 && grid <= 148
             ? launch_programmatic(paged_plan_kernel<1024>, dim3((unsigned)grid), dim3(1024), 0,
                                   st, a)
             : launch_programmatic(paged_plan_kernel<256>, dim3((unsigned)grid), dim3(256), 0, st,
                                   a);
}

// ------------------------------------------------------------------ append
//
// A CTA owns a tile of tokens for a slab of the head rows [q heads | k heads |
// v heads].  It builds the (cos, sin) of its tokens in shared memory (the
// frequency of a thread's pairs is raised once, the angle is formed and
// reduced in 64 bits as in rope_apply, so the results are the same bits) and
// a list of the tokens that have a slot, then streams the rows: a thread
// takes 32 bytes of a row -- the two 16-byte chunks that hold its 8 pairs --
// and writes them to q_out / k_out and to the cache.  Bound by HBM for
// prompts (4 x 8192 tokens of 32 + 8 + 8 heads, 806 MB: 146 us, 5.5 TB/s; with
// one item of a thread at a time 167, with 3 blocks an SM 211), by latency for
// a decode step (64 tokens: 4.4 us, 0.8 of them the 64-bit power).

namespace {
constexpr int kAppThreads = 256;
constexpr int kBatch = 2;        // items of a thread whose loads are on their way together

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
}  // namespace

struct AppendArgs {
  const __nv_bfloat16* x[3];     // q, k, v
  long long sb[3], sh[3], st[3]; // strides of batch, head, token in elements
  const int32_t* positions;
  const int32_t* slots;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  int B, Hq, Hkv, N, page_size, num_pages;
  int heads;                     // Hq + Hkv (+ Hkv with v)
  int slabs;
  double base;
};

template <int D, bool kRope, bool kAdjacent, int TT>
__global__ void __launch_bounds__(kAppThreads, 4) kv_append_kernel(AppendArgs a) {
  constexpr int kHalf = D / 2;
  constexpr int kChunks = D / 16;                  // 32-byte items of a row
  constexpr int kRows = kAppThreads / kChunks;     // rows that the block takes at once
  __shared__ __align__(16) float2 tab[kRope ? TT * kHalf : 2];
  __shared__ long long s_src[3][TT];   // a token's row in q, k, v (elements)
  __shared__ int s_b[TT], s_i[TT];
  __shared__ long long s_cache[TT];    // its row in the cache, or -1 (elements)
  __shared__ int s_list[TT];           // the tokens that are stored
  __shared__ int s_kept;
  const int tid = threadIdx.x;
  const long long T = (long long)a.B * a.N;
  const long long t0 = (long long)blockIdx.x * TT;
  const int nt = T - t0 < TT ? (int)(T - t0) : TT;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < 32) {
    const long long rows = (long long)a.num_pages * a.page_size;
    int slot = -1;
    if (tid < nt) {
      if (a.slots) slot = a.slots[t0 + tid];
      const int b = (int)((unsigned)(t0 + tid) / (unsigned)a.N);   // (B * N < 2^31)
      const int i = (int)(t0 + tid - (long long)b * a.N);
      s_b[tid] = b;
      s_i[tid] = i;
#pragma unroll
      for (int p = 0; p < 3; ++p) s_src[p][tid] = b * a.sb[p] + i * a.st[p];
      if (slot >= rows) {
        slot = -1;
        atomicExch(&g_device_status, (int)ATTN_ERANGE);
      }
      const int page = slot < 0 ? 0 : slot / a.page_size;
      s_cache[tid] = slot < 0 ? -1
                              : ((long long)page * a.Hkv * a.page_size + (slot - page * a.page_size)) * D;
    }
    const unsigned m = __ballot_sync(0xffffffffu, slot >= 0);
    if (slot >= 0) s_list[__popc(m & ((1u << tid) - 1))] = tid;
    if (tid == 0) s_kept = __popc(m);
  }
  if constexpr (kRope) {
    const int i = tid % kHalf;
    const double theta = pow(a.base, -2.0 * (double)i / (double)D);
    for (int t = tid / kHalf; t < nt; t += kAppThreads / kHalf) {
      double s, c;
      sincos((double)a.positions[t0 + t] * theta, &s, &c);
      tab[t * kHalf + i] = make_float2((float)c, (float)s);
    }
  }
  __syncthreads();
  const int kept = s_kept;
  const int h0 = (int)((long long)a.heads * blockIdx.y / a.slabs);
  const int h1 = (int)((long long)a.heads * (blockIdx.y + 1) / a.slabs);
  const int c = tid % kChunks;

#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    // head rows of this part in the slab
    const int p0 = part == 0 ? 0 : (part == 1 ? a.Hq : a.Hq + a.Hkv);
    const int p1 = part == 0 ? a.Hq : (part == 1 ? a.Hq + a.Hkv : a.heads);
    const int f = (h0 > p0 ? h0 : p0) - p0, e = (h1 < p1 ? h1 : p1) - p0;
    __nv_bfloat16* out = part == 0 ? a.q_out : (part == 1 ? a.k_out : nullptr);
    __nv_bfloat16* cache = part == 0 ? nullptr : (part == 1 ? a.kc : a.vc);
    const int H = part == 0 ? a.Hq : a.Hkv;
    // without a copy outside the cache only the stored tokens matter
    const int n = out ? nt : kept;
    if (f >= e || n == 0) continue;
    const bool rot = kRope && part < 2;
    // chunks of an item: pairs (i, i + D/2) sit in chunk c of each half,
    // adjacent pairs and plain copies in two neighbouring chunks
    const bool halves = rot && !kAdjacent;
    const int e0 = halves ? 8 * c : 16 * c, e1 = halves ? kHalf + 8 * c : 16 * c + 8;
    const __nv_bfloat16* x = a.x[part];
    const long long sh = a.sh[part];
    // rows (head, token) side by side; a thread steps kRows rows on
    const int dh = kRows / n, dl = kRows % n;
    int h = f + (tid / kChunks) / n, li = (tid / kChunks) % n;
    // several items at a time, their loads first: outputs may be the inputs
    // themselves, so no load can be moved above an earlier item's stores
    while (h < e) {
      uint4 va[kBatch], vb[kBatch];
      int ts[kBatch], hs[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        hs[u] = h;
        ts[u] = 0;
        if (h < e) {
          ts[u] = out ? li : s_list[li];
          const __nv_bfloat16* src = x + s_src[part][ts[u]] + h * sh;
          va[u] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
          vb[u] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
        }
        h += dh;
        li += dl;
        if (li >= n) { li -= n; ++h; }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (hs[u] >= e) break;
        const int t = ts[u];
        if (rot) {
          const uint32_t wa[4] = {va[u].x, va[u].y, va[u].z, va[u].w};
          const uint32_t wb[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
          uint32_t oa[4], ob[4];
          const float4* cs = reinterpret_cast<const float4*>(tab + t * kHalf + 8 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kAdjacent) {
              const float4 p = cs[k >> 1], w = cs[2 + (k >> 1)];
              const float2 cp = (k & 1) ? make_float2(p.z, p.w) : make_float2(p.x, p.y);
              const float2 cw = (k & 1) ? make_float2(w.z, w.w) : make_float2(w.x, w.y);
              float r0, r1;
              rope_rotate(lo_bf16(wa[k]), hi_bf16(wa[k]), cp, r0, r1);
              oa[k] = pack_bf16x2(r0, r1);
              rope_rotate(lo_bf16(wb[k]), hi_bf16(wb[k]), cw, r0, r1);
              ob[k] = pack_bf16x2(r0, r1);
            } else {
              const float4 p = cs[k];
              float ra0, rb0, ra1, rb1;
              rope_rotate(lo_bf16(wa[k]), lo_bf16(wb[k]), make_float2(p.x, p.y), ra0, rb0);
              rope_rotate(hi_bf16(wa[k]), hi_bf16(wb[k]), make_float2(p.z, p.w), ra1, rb1);
              oa[k] = pack_bf16x2(ra0, ra1);
              ob[k] = pack_bf16x2(rb0, rb1);
            }
          }
          va[u] = make_uint4(oa[0], oa[1], oa[2], oa[3]);
          vb[u] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
        }
        if (out) {
          __nv_bfloat16* o = out + (((size_t)s_b[t] * H + hs[u]) * a.N + s_i[t]) * D;
          *reinterpret_cast<uint4*>(o + e0) = va[u];
          *reinterpret_cast<uint4*>(o + e1) = vb[u];
        }
        if (cache && s_cache[t] >= 0) {
          __nv_bfloat16* o = cache + s_cache[t] + (size_t)hs[u] * a.page_size * D;
          *reinterpret_cast<uint4*>(o + e0) = va[u];
          *reinterpret_cast<uint4*>(o + e1) = vb[u];
        }
      }
    }
  }
}

namespace {
template <int D, bool kRope, bool kAdjacent>
int launch_append_t(AppendArgs a, cudaStream_t st) {
  const long long T = (long long)a.B * a.N;
  // a tile of 16 tokens fills the machine from some 5k tokens on (8, 24 and 32
  // took 1 to 6% longer on 32k); below that smaller tiles and slabs of heads
  // spread the rows over the SMs
  const bool small = T <= 1024;
  const long long tiles = (T + (small ? 4 : 16) - 1) / (small ? 4 : 16);
  long long slabs = (296 + tiles - 1) / tiles;
  if (slabs > a.heads) slabs = a.heads;
  a.slabs = (int)slabs;
  const dim3 grid((unsigned)tiles, (unsigned)slabs);
  return small ? launch_programmatic(kv_append_kernel<D, kRope, kAdjacent, 4>, grid,
                                     dim3(kAppThreads), 0, st, a)
               : launch_programmatic(kv_append_kernel<D, kRope, kAdjacent, 16>, grid,
                                     dim3(kAppThreads), 0, st, a);
}
}  // namespace

int launch_kv_append(const void* q, const void* k, const void* v, const int64_t* strides,
                     const int32_t* positions, float rope_base, int rope_pairing, void* q_out,
                     void* k_out, const int32_t* slots, void* k_cache, void* v_cache, int B,
                     int Hq, int Hkv, int N, int d, int page_size, int num_pages,
                     cudaStream_t st) {
  AppendArgs a;
  const void* x[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    a.x[i] = static_cast<const __nv_bfloat16*>(x[i]);
    a.sb[i] = strides[3 * i];
    a.sh[i] = strides[3 * i + 1];
    a.st[i] = strides[3 * i + 2];
  }
  a.positions = positions;
  a.slots = slots;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.kc = static_cast<__nv_bfloat16*>(k_cache);
  a.vc = static_cast<__nv_bfloat16*>(v_cache);
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.N = N;
  a.page_size = page_size; a.num_pages = num_pages;
  a.heads = Hq + Hkv + (slots ? Hkv : 0);
  a.base = (double)rope_base;
  if (d == 128) {
    if (!positions) return launch_append_t<128, false, false>(a, st);
    return rope_pairing ? launch_append_t<128, true, true>(a, st)
                        : launch_append_t<128, true, false>(a, st);
  }
  if (!positions) return launch_append_t<64, false, false>(a, st);
  return rope_pairing ? launch_append_t<64, true, true>(a, st)
                      : launch_append_t<64, true, false>(a, st);
}

}  // namespace attn
