// The merge of the split kernels' partial records, for the 16-bit and the 4-bit paged cache.
#pragma once
#include "swa_paged_attend.cuh"

namespace swa {
#ifdef __CUDACC__

// ---------------------------------------------------------------------------
// Merge: block (c, r) joins, for the rows r, r + gridDim.y, .., the records of the item that CTA c left unfinished at
// its end: slot 2c + 1, then slot 2c' of the following CTAs up to the one that ended
// it. 8 features a lane; the thread groups take the records in turn.
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedAttendParams p, int rows) {
  constexpr int L = D / 8, NG = kMergeThreads / L;
  __shared__ __align__(16) float s_acc[NG][D];
  __shared__ float s_l[NG];
  pdl_wait();
  pdl_trigger();
  const int4 dsc = p.ws_desc[blockIdx.x];
  if (dsc.x < 0) return;
  for (int row = blockIdx.y; row < dsc.w * p.hpg; row += gridDim.y) {
    const int c0 = blockIdx.x, n = dsc.z - c0 + 1;
    const int tid = threadIdx.x, grp = tid / L, c = tid % L;
    auto rec = [&](int i) { return ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * rows + row; };
    float y[8];                               // a group's first record, asked for before the maximum is known
    if (grp < n) load8(p.ws_acc + rec(grp) * D + c * 8, y);
    float mt = -INFINITY;
    for (int i = tid; i < n; i += kMergeThreads) mt = fmaxf(mt, p.ws_ml[rec(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    if ((tid & 31) == 0) s_l[tid >> 5] = mt;
    __syncthreads();
    mt = fmaxf(fmaxf(s_l[0], s_l[1]), fmaxf(s_l[2], s_l[3]));
    __syncthreads();
    float lt = 0.f, acc[8] = {};
#pragma unroll 4
    for (int i = grp; i < n; i += NG) {
      const float2 ml = p.ws_ml[rec(i)];
      const float a = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt);
      if (i > grp) load8(p.ws_acc + rec(i) * D + c * 8, y);
      lt += a * ml.y;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += a * y[j];
    }
    store8(&s_acc[grp][c * 8], acc);
    if (c == 0) s_l[grp] = lt;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int w = 1; w < NG; ++w) {
        float y[8];
        load8(&s_acc[w][c * 8], y);
        lt += s_l[w];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += y[j];
      }
      paged_store_row<T>(p, dsc.x + row / p.hpg, dsc.y * p.hpg + row % p.hpg, D, c * 8, mt, lt, PScale<T>::kLog2, acc, c == 0);
    }
    __syncthreads();                          // s_acc and s_l are read
  }
}

#endif
}  // namespace swa
