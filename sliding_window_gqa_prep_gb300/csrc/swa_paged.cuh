// Shared by the paged-cache and rotary kernels: element types, the page map and
// a sequence's rows and length as the kernels read them (all bounds applied).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "swa_internal.cuh"

namespace swa {

// The page map of a swa_paged_cache as the kernels take it (by value).
struct PagedMap {
  int B, nk, page_shift, num_pages, max_pages, cap;   // cap = max_pages << page_shift
  const int32_t* table;
  const int32_t* row_start;
  const int32_t* lens;
};

// Host checks shared by the paged calls (swa_paged.cu). rows: row_start is read.
int paged_cache_status(const swa_paged_cache* c, bool rows);
PagedMap paged_map(const swa_paged_cache* c);
// [a, a + an) and [b, b + bn) share a byte
bool bytes_overlap(const void* a, size_t an, const void* b, size_t bn);
// Elements that T >= 1 rows of n elements, `row` apart, span; -1 when rows overlap or the
// span passes 2^44 (no memory holds it, and products of offsets stay in 64 bits)
inline long long rows_span(long long T, long long n, long long row) {
  if (n < 1 || row < n || row > (1LL << 40) || row > (1LL << 44) / T) return -1;
  return (T - 1) * row + n;
}
inline bool aligned16p(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t up256s(size_t x) { return (x + 255) & ~(size_t)255; }

// Dynamic shared memory of a kernel, allowed once per device (an attribute call costs as
// much host time as the rest of a launch's preparation). With min_regs the kernel has to have been
// compiled to that many registers a thread.
template <auto Kernel>
cudaError_t allow_smem(int bytes, int min_regs = 0) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  if (min_regs) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, Kernel)) != cudaSuccess) return e;
    if (fa.numRegs < min_regs) return cudaErrorLaunchOutOfResources;
  }
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

#ifdef __CUDACC__

// Rows and keys of sequence b. Rows out of range leave t = 0, a length out of
// range is clamped; `bits` collects the SWA_DERR_* of what was found.
struct PagedSeq {
  int r0, t, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedMap& m, int b, int T, int max_rows, uint32_t& bits) {
  PagedSeq s;
  const int r0 = m.row_start[b], r1 = m.row_start[b + 1];
  int len = m.lens[b];
  s.r0 = r0;
  s.t = r1 - r0;
  if (r0 < 0 || r1 < r0 || r1 > T || s.t > max_rows) {
    bits |= SWA_DERR_SEGMENT;
    s.r0 = 0;
    s.t = 0;
  }
  if (len < 0 || len > m.cap) {
    bits |= SWA_DERR_META;
    len = len < 0 ? 0 : m.cap;
  }
  s.len = len;
  return s;
}

__device__ __forceinline__ bool page_ok(const PagedMap& m, int page) {
  return (unsigned)page < (unsigned)m.num_pages;
}

// Eight elements of a 16-bit or f32 row, 16-byte aligned, to and from f32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of its f32
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b, const __nv_bfloat16*) {
  a = __uint_as_float(v << 16);
  b = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b, const __half*) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1], p), pack2(x[2], x[3], p), pack2(x[4], x[5], p),
                                            pack2(x[6], x[7], p));
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void round_to(float& d, float x) { d = x; }
__device__ __forceinline__ void round_to(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void round_to(__half& d, float x) { d = __float2half_rn(x); }

// N = 1, 2, 4 or 8 elements at a multiple of N, as they lie in memory (accesses of up to
// 16 bytes) and as f32
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T e[N];
};
template <int N, typename T>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) { return *reinterpret_cast<const Pack<T, N>*>(p); }
template <int N, typename T>
__device__ __forceinline__ void unpack(const Pack<T, N>& v, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f32(v.e[i]);
}
template <int N, typename T>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[N]) {
  Pack<T, N> v;
#pragma unroll
  for (int i = 0; i < N; ++i) round_to(v.e[i], x[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

#endif  // __CUDACC__

}  // namespace swa
