// Pieces of the paged kernels on the tensor cores (tcgen05, pages copied by TMA).
#pragma once
#include <cuda.h>

#include "swa_paged_attend.cuh"
#include "swa_tcgen05.cuh"

namespace swa {

// Tensor map of a page pool (K or V of a swa_paged_cache): rows of hd elements, boxes of
// 64 features x min(page, kt) rows, 128-byte swizzle, zeros out of range (swa_paged.cu).
int pool_map(const swa_paged_cache& c, void* base, int kt, CUtensorMap* m);
// Tensor map of packed rows q [T][nh][hd], `row` elements apart, of the cache's type: boxes of
// 64 features x `heads` heads x `rows` rows, 128-byte swizzle (swa_paged.cu).
int rows_map(const swa_paged_cache& c, const void* q, int T, int nh, long long row, int heads, int rows, CUtensorMap* m);

#ifdef __CUDACC__
// kind::f16 with D in f32, A and B both f16 or both bf16, A K-major, B K-major or not
__host__ __device__ constexpr uint32_t tc_idesc_16(bool bf16, bool b_mn_major, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// Shared-memory matrix descriptor, 128-byte swizzle (rows of 128 bytes, groups of 8
// rows every 1024 bytes). K-major: sbo = 1024. MN-major: sbo = 1024 between groups of
// 8 K rows, lbo between columns of 64 MN elements.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0) : "memory");
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// packed pairs of f32
__device__ __forceinline__ uint64_t pack64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void unpack64(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Waits for this thread's TMEM loads; the registers are operands, so that nothing that
// reads them moves ahead of the wait.
#define SWA_RW32(r) "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]), \
  "+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15]), \
  "+r"(r[16]),"+r"(r[17]),"+r"(r[18]),"+r"(r[19]),"+r"(r[20]),"+r"(r[21]),"+r"(r[22]),"+r"(r[23]), \
  "+r"(r[24]),"+r"(r[25]),"+r"(r[26]),"+r"(r[27]),"+r"(r[28]),"+r"(r[29]),"+r"(r[30]),"+r"(r[31])
template <int N>
__device__ __forceinline__ void wait_ld(uint32_t (&x)[N][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SWA_RW32(x[0]) :: "memory");
#pragma unroll
  for (int i = 1; i < N; ++i) asm volatile("" : SWA_RW32(x[i]) :: "memory");
}
__device__ __forceinline__ void wait_ld(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SWA_RW32(x) :: "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
               :: "r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
               :: "r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z) : "memory");
}

// A wait that gives up after kWaitLimitNs, for the whole CTA; the clock is read every 64th try only (the
// read takes longer than a try).
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) *(volatile int*)abort_flag = 1;
      if (*(volatile int*)abort_flag) return false;
    }
  }
}

#endif  // __CUDACC__

}  // namespace swa
