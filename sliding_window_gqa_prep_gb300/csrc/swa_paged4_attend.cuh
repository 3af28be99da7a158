// Shared by the attention kernels over the 4-bit paged cache: parameters, which tiles of keys a
// sequence's rows see, and the queries' scales.
#pragma once
#include "swa_paged4.cuh"
#include "swa_paged_attend.cuh"
#include "swa_paged_tc.cuh"

namespace swa {

struct Attend4Params {
  PagedAttendParams a;         // qmul: scale * log2(e) * 2^k_exp; q of type bf or f16
  Pools4 c;
  int bf;                      // q (and a 16-bit out) is bf16, else f16
  int window, sinks;           // window: 2^30 and more where there is none (sinks is then 0)
  int rows;                    // split kernel: query vectors of a record
  float rec_log2;              // log2 of the records' factor: PScale<type>, as the merge takes it
};

// Weights are 2^(s - max) times 2^kLog24; the running maximum is raised when a score passes it by
// kLazy4, so they stay below 2^15 < 65504, and one below 2^-14 loses 2^-25: 2^-36 of the row's scale.
constexpr float kLazy4 = 4.f, kLog24 = 11.f;

// The tensor-core kernel for chunks of many query vectors (swa_paged4_chunk.cuh)
ChunkPlan chunk4_plan(const swa_paged4_attend_args* a, int max_rows);
int launch_paged4_chunk(int hd, const Attend4Params& p, const ChunkPlan& plan, int small, char* ws, cudaStream_t s);

#ifdef __CUDACC__
// First key in the window of a row that sees the slots below lim (none: lim <= 0)
__device__ __forceinline__ int first_key(int lim, int window) { return max(0, max(0, lim) - window); }

// Tiles of kt keys that a sequence's rows see: the sinks', then those from the first row's window on.
struct Tiles4 {
  int sink, first, n;          // tiles of sinks in front of tile `first`; all
  __device__ __forceinline__ int at(int x) const { return x < sink ? x : x - sink + first; }
};
__device__ __forceinline__ Tiles4 key_tiles(const PagedSeq& s, const Attend4Params& p, int kt) {
  Tiles4 t;
  const int lo = first_key(s.len - s.t + 1, p.window);      // the first row's
  t.first = lo / kt;
  t.sink = min((min(p.sinks, s.len) + kt - 1) / kt, t.first);
  t.n = s.len > 0 ? t.sink + (s.len + kt - 1) / kt - t.first : 1;   // a row without keys is still written
  return t;
}

// The power of two that brings a vector's largest value to [2^14, 2^15) (as far as f32 has it; 1 for
// zeros, infinities and NaN), and its inverse
__device__ __forceinline__ float query_scale(float top, float& inv) {
  const int e = (int)(__float_as_uint(top) >> 23);          // biased; 0: below 2^-126
  const int shift = top == 0.f || e == 255 ? 0 : min(127, 14 + 127 - e);
  inv = __uint_as_float(shift >= 127 ? 0x00400000u : (uint32_t)(127 - shift) << 23);   // 2^-127 is subnormal
  return __uint_as_float((uint32_t)(127 + shift) << 23);
}

// Loads from shared memory by its own addresses (a pointer that was rounded up is a generic one): W words,
// aligned to their number; 16 and 8 bits. Volatile: they stay behind the waits.
template <int W>
__device__ __forceinline__ void lds_words(uint32_t (&r)[W], uint32_t at) {
  if constexpr (W == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(at));
  else if constexpr (W == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  uint32_t r;
  asm volatile("{\n\t.reg .b16 a;\n\tld.shared.b16 a, [%1];\n\tcvt.u32.u16 %0, a;\n\t}" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ void sts_words(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
#endif

}  // namespace swa
