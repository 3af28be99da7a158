// Attention of a ragged chunk over the 4-bit paged cache (swa_paged4_attend).
//
// A warp takes a query vector and walks the keys that its row sees, one at a time: the lanes hold
// hd / 32 features each, the softmax runs along.
#include <cmath>

#include "swa_paged4.cuh"
#include "swa_paged_attend.cuh"

namespace swa {

struct Attend4Params {
  PagedMap map;
  Pools4 c;
  int T, nh, hpg, max_rows, window, sinks, out_f32;
  float qmul;                  // scale * log2(e) * 2^k_exp: scores in log2 units
  const void* q;
  long long q_row;
  void* out;
  float* lse;
  uint32_t* err;
};

template <typename T, int E>
__global__ void __launch_bounds__(128) paged4_plain_kernel(const Attend4Params p) {
  constexpr int HD = 32 * E;
  const int lane = threadIdx.x & 31;
  const long long v = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y;
  uint32_t bits = 0;
  const PagedSeq s = paged_seq(p.map, b, p.T, p.max_rows, bits);
  const int i = (int)(v / p.nh), h = (int)(v % p.nh), g = h / p.hpg;
  if (i < s.t) {
    const int lim = min(s.len, s.len - s.t + i + 1), lo = p.window ? max(0, lim - p.window) : 0;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    unpack(load_pack<E>(static_cast<const T*>(p.q) + (long long)(s.r0 + i) * p.q_row + (long long)h * HD + lane * E), q);
    for (int j = 0; j < lim; ++j) {
      if (j < lo && j >= p.sinks) j = lo;
      const int page = p.map.table[(size_t)b * p.map.max_pages + (j >> p.map.page_shift)];
      const bool ok = page_ok(p.map, page);
      if (!ok) bits |= SWA_DERR_PAGE;
      const long long key = ok ? ((((long long)page * p.map.nk + g) << p.map.page_shift) + (j & ((1 << p.map.page_shift) - 1))) : 0;
      float k[E], w[E], x = 0.f;
      auto value = [&](const uint8_t* codes, const uint8_t* scales, float (&y)[E]) {
        const float u = ok ? e4m3_f32(scales[key * (HD / 16) + lane * E / 16]) : 0.f;
        for (int e = 0; e < E; e += 2) {
          const uint32_t f = e2m1x2_f16x2<0>(codes[key * (HD / 2) + (lane * E + e) / 2]);
          const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&f));
          y[e] = t.x * u;
          y[e + 1] = t.y * u;
        }
      };
      value(p.c.k, p.c.ks, k);
      value(p.c.v, p.c.vs, w);
      for (int e = 0; e < E; ++e) x += q[e] * k[e];
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= p.qmul;
      const float mn = fmaxf(m, x), a = ex2(m - mn), e1 = ex2(x - mn);
      m = mn;
      l = l * a + e1;
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + e1 * w[e];
    }
    const float inv = l > 0.f ? p.c.v_mul / l : l;
    for (int e = 0; e < E; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
    const long long at = ((long long)(s.r0 + i) * p.nh + h) * HD + lane * E;
    if (p.out_f32) store_pack(static_cast<float*>(p.out) + at, o);
    else store_pack(static_cast<T*>(p.out) + at, o);
    if (lane == 0 && p.lse) p.lse[(long long)(s.r0 + i) * p.nh + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
  if (bits) set_err(p.err, bits);
}

// Sizes alone (the workspace query); pointers are checked by the call.
static bool attend4_sizes_ok(const swa_paged4_attend_args* a) {
  const swa_paged4_cache& c = a->cache;
  if (c.B < 1 || c.B > 65535 || c.nk < 1 || c.nk > 65535 || (long long)c.B * c.nk > (1 << 24)) return false;
  if (c.hd != 64 && c.hd != 128 && c.hd != 256) return false;
  if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1))) return false;
  if (c.max_pages < 1 || c.max_pages > (1 << 30) / c.page) return false;
  if (a->T < 0 || a->max_rows < 1 || a->nh < 1 || a->nh % c.nk || a->nh / c.nk > 32) return false;
  if (a->window < 0 || a->sinks < 0 || (a->q_dtype != SWA_BF16 && a->q_dtype != SWA_F16)) return false;
  return (long long)a->T * a->nh < (1LL << 31) - 256;
}

}  // namespace swa

using namespace swa;

extern "C" {

size_t swa_paged4_attend_workspace_size(const swa_paged4_attend_args* a) {
  return a && attend4_sizes_ok(a) ? 1 : 0;
}

int swa_paged4_attend(const swa_paged4_attend_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged4_cache& c = a->cache;
  int rc = paged4_cache_status(&c);
  if (rc != SWA_OK) return rc;
  if (!attend4_sizes_ok(a) || !(a->scale >= 0.f) || std::isinf(a->scale)) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->q || !a->out) return SWA_E_NULL;
  const long long qn = rows_span(a->T, (long long)a->nh * c.hd, a->q_row);
  if (qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->q) || !aligned16p(a->out) || (a->q_row & 7) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
    return SWA_E_ALIGN;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return SWA_E_ALIGN;
  const size_t rows = (size_t)a->T * a->nh, on = rows * c.hd * (a->out_f32 ? 4 : 2), ln = a->lse ? rows * 4 : 0;
  if (bytes_overlap(a->q, (size_t)qn * 2, a->out, on) ||
      (a->lse && (bytes_overlap(a->q, (size_t)qn * 2, a->lse, ln) || bytes_overlap(a->out, on, a->lse, ln))))
    return SWA_E_SHAPE;
  Attend4Params p{};
  p.map = paged4_map(&c);
  p.c = paged4_pools(&c);
  p.T = a->T; p.nh = a->nh; p.hpg = a->nh / c.nk; p.max_rows = a->max_rows < a->T ? a->max_rows : a->T;
  p.window = a->window; p.sinks = a->window ? a->sinks : 0;
  p.qmul = a->scale * 1.4426950408889634f * p.c.k_mul;
  p.q = a->q; p.q_row = a->q_row;
  p.out = a->out; p.out_f32 = a->out_f32 != 0; p.lse = a->lse;
  p.err = a->err;
  cudaError_t e;
  if (a->ev_start && (e = cudaEventRecord(a->ev_start, stream)) != cudaSuccess) return cuda_status(e);
  const dim3 grid((unsigned)(((long long)p.max_rows * p.nh + 3) / 4), c.B), block(128);
  const bool bf = a->q_dtype == SWA_BF16;
  e = c.hd == 64    ? (bf ? launch_pdl(paged4_plain_kernel<__nv_bfloat16, 2>, grid, block, 0, stream, p) : launch_pdl(paged4_plain_kernel<__half, 2>, grid, block, 0, stream, p))
      : c.hd == 128 ? (bf ? launch_pdl(paged4_plain_kernel<__nv_bfloat16, 4>, grid, block, 0, stream, p) : launch_pdl(paged4_plain_kernel<__half, 4>, grid, block, 0, stream, p))
                    : (bf ? launch_pdl(paged4_plain_kernel<__nv_bfloat16, 8>, grid, block, 0, stream, p) : launch_pdl(paged4_plain_kernel<__half, 8>, grid, block, 0, stream, p));
  rc = finish_launch(e);
  if (rc != SWA_OK) return rc;
  if (a->ev_stop && (e = cudaEventRecord(a->ev_stop, stream)) != cudaSuccess) return cuda_status(e);
  return SWA_OK;
}

}  // extern "C"
