// Shared by the kernels of the 4-bit paged cache: its pools, and the conversions of its
// codes (e2m1) and scales (e4m3).
#pragma once
#include "swa_paged.cuh"

namespace swa {

constexpr int kBlock4 = 16;              // features of a scale

struct Pools4 {
  uint8_t* k;                            // [num_pages][nk][page][hd / 2]
  uint8_t* ks;                           // [num_pages][nk][page][hd / 16]
  uint8_t* v;
  uint8_t* vs;
  float k_mul, v_mul;                    // 2^k_exp, 2^v_exp
};

// Host checks shared by the calls (swa_paged4_rows.cu).
int paged4_cache_status(const swa_paged4_cache* c);
PagedMap paged4_map(const swa_paged4_cache* c);
Pools4 paged4_pools(const swa_paged4_cache* c);
// The four pools and their bytes
struct Span4 {
  const void* at;
  size_t bytes;
};
void paged4_spans(const swa_paged4_cache* c, Span4 (&s)[4]);

#ifdef __CUDACC__
// Two codes of a byte (the lower half first) as f16x2: byte B of w
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t d;
  if constexpr (B == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (B == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (B == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
// Two scales as f16x2, the lower byte first (e4m3 is exact in f16)
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
  const uint32_t h = e4m3x2_f16x2(byte);
  return __half2float(__ushort_as_half((unsigned short)h));
}
// The nearest e4m3 (ties to even, 448 at most; NaN stays)
__device__ __forceinline__ uint32_t f32_e4m3(float x) {
  uint32_t d;
  asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %1, %2;\n\tcvt.u32.u16 %0, a;\n\t}" : "=r"(d) : "f"(0.f), "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
#endif

}  // namespace swa
