// Shared by the attention kernels over the paged cache: parameters, the weights'
// scale and the last step of a row.
#pragma once
#include <type_traits>

#include "swa_paged.cuh"

namespace swa {

template <int N>
using Int = std::integral_constant<int, N>;

struct PagedAttendParams {
  PagedMap map;
  int T, nh, hpg, max_rows;
  int whole;                   // split kernel: a CTA per (sequence, KV head), nothing to merge
  int most;                    // split kernel: sequences with more query vectors are not its
  float qmul;                  // scale * log2(e): scores in log2 units
  const void* q;
  long long q_row;
  void* out;
  int out_f32;
  float* lse;
  float* ws_acc;               // [records][rows][hd] (split kernel)
  float2* ws_ml;               // [records][rows] (m in log2 units, l)
  int4* ws_desc;               // per CTA: the item it left unfinished (b, g, last CTA, 0), b < 0: none
  uint32_t* err;
};

// Weights are 2^(s - max) times 2^kLog2 before they are rounded to T: f16 has no
// exponents below 2^-24, and weights under it would count in the sum but not in the
// product. Times 2^15 (the largest weight is then 2^15 < 65504) a weight loses 2^-40 of the
// largest at most. bf16 has f32's exponents.
template <typename T>
struct PScale {
  static constexpr float kLog2 = 0.f;
};
template <>
struct PScale<__half> {
  static constexpr float kLog2 = 15.f;
};

// The tensor-core kernel for chunks of many query vectors (swa_paged_chunk.cu)
struct ChunkPlan {
  int tile_tok, splits;        // chunk rows of a query tile, shares of an item's keys
  long long items;             // upper bound of its items (grid)
  size_t off_ml, off_desc, bytes;
};
ChunkPlan chunk_plan(const swa_paged_attend_args* a, int max_rows);
int launch_paged_chunk(const swa_paged_attend_args* a, const PagedAttendParams& p, const ChunkPlan& plan, int small,
                       char* ws, cudaStream_t s);

#ifdef __CUDACC__
// Features [f, f + 8) of a finished row: out = acc / l, and its lse (the weights in l
// carry 2^log2_scale).
template <typename T>
__device__ __forceinline__ void paged_store_row(const PagedAttendParams& p, int row, int head, int hd, int f, float m,
                                                float l, float log2_scale, float (&acc)[8], bool first) {
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no key: zeros; NaN stays
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = l == 0.f ? 0.f : acc[j] * inv;
  const size_t at = ((size_t)row * p.nh + head) * hd + f;
  if (p.out_f32)
    store8(static_cast<float*>(p.out) + at, acc);
  else
    store8(static_cast<T*>(p.out) + at, acc);
  if (first && p.lse)
    p.lse[(size_t)row * p.nh + head] = l == 0.f ? -INFINITY : (m - log2_scale + log2f(l)) * 0.6931471805599453f;
}
#endif

}  // namespace swa
