// tree.cu -- attention for a tree of drafted tokens over a cache: node i of a
// sequence sees every cached key, itself and its ancestors.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "tile_plan.cuh"

namespace attn {

// One warp per query row: the lanes hold the row's head dimension, the keys
// pass one at a time through the running maximum and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(TreeArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.Hq * a.Nq) return;
  const int i = (int)(row % a.Nq);
  const int hq = (int)(row / a.Nq % a.Hq), b = (int)(row / a.Nq / a.Hq);
  const int h = hq / (a.Hq / a.Hkv);
  const int L = clamp_len(a.key_lens ? a.key_lens[b] : a.Nk, a.Nk);
  const int n = clamp_len(a.new_lens ? a.new_lens[b] : a.Nq, a.Nq);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[row * D + lane * E + e]) * a.scale_log2;
    o[e] = 0.f;
  }
  auto add = [&](const __nv_bfloat16* kr, const __nv_bfloat16* vr) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kr[lane * E + e]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2_approx(m - mn), p = exp2_approx(s - mn);
    l = fmaf(l, f, p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, __bfloat162float(vr[lane * E + e]), o[e] * f);
    m = mn;
  };
  if (i < n) {
    for (int j = 0; j < L; ++j) {
      long long r;
      if (a.block_table) {
        const int page = a.block_table[(size_t)b * a.max_pages + j / a.page_size];
        if ((unsigned)page >= (unsigned)a.num_pages) {   // its keys and values read as zeros
          if (lane == 0) atomicExch(&g_device_status, (int)ATTN_ERANGE);
          const float mn = fmaxf(m, 0.f);
          const float f = m == -INFINITY ? 0.f : exp2_approx(m - mn);
          l = fmaf(l, f, exp2_approx(-mn));
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= f;
          m = mn;
          continue;
        }
        r = ((long long)page * a.Hkv + h) * a.page_size + j % a.page_size;
      } else {
        r = ((long long)b * a.Hkv + h) * a.Nk + j;
      }
      add(a.kc + r * D, a.vc + r * D);
    }
    for (int j = i; j >= 0;) {
      const long long r = ((long long)b * a.Hkv + h) * a.Nq + j;
      add(a.kn + r * D, a.vn + r * D);
      const int p = a.parents[(size_t)b * a.Nq + j];
      if (p < -1 || p >= j) {
        if (lane == 0) atomicExch(&g_device_status, (int)ATTN_ERANGE);
        break;
      }
      j = p;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.o[row * D + lane * E + e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

bool tree_supported(int B, int Nq, int d) {
  return (d == 64 || d == 128) && Nq <= 1024 && B <= 2048;
}

size_t tree_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int num_sms) {
  (void)B; (void)Hq; (void)Hkv; (void)Nq; (void)d; (void)num_sms;
  return 256;
}

int launch_tree(const TreeArgs& a, int d, void* workspace, int num_sms, cudaStream_t st) {
  (void)workspace; (void)num_sms;
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (d == 128) tree_rows_kernel<128><<<grid, 128, 0, st>>>(a);
  else tree_rows_kernel<64><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ECUDA;
}

}  // namespace attn
