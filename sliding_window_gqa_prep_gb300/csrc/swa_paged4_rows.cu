// Rows into and out of the 4-bit paged cache: swa_paged4_append (rotary positions, encoding,
// and the rotation of q) and swa_paged4_read.
//
// Encoding is exact in the sense that the stored codes are those of the formula, not of its
// f32 arithmetic: the borders between two levels (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5 times
// scale * 2^exp) have seven bits and a comparison of an f32 with them is exact, and a block's
// largest value / 6 in f32 falls on the same side of a border between two scales as the exact
// quotient (a border times 6 has seven bits, so a value next to it is at least 2/3 of an ulp of
// the quotient away). Values that were not rotated are thus encoded exactly. A rotated value is
// known up to kTol * (|u| + |v|); where that leaves a scale or a code open (one head in some
// hundreds) the warp takes the angles and the encoding again in f64.
#include <cmath>

#include "swa_paged4.cuh"

namespace swa {

struct Rows4Params {
  PagedMap map;
  Pools4 c;
  int T, hd, R;                // rows of a block
  // append: heads [0, nh) are q, [nh, nh + nk) k, [nh + nk, H) v
  int nh, H, Hg, rot;          // heads of a block
  float mag;
  const void* q;
  const void* k;
  const void* v;
  long long q_row, k_row, v_row;
  void* q_out;
  const int32_t* pos;
  const uint64_t* turns;
  float k_div, v_div;          // 2^-exp
  // read
  void* k_out;
  void* v_out;
  uint32_t* err;
};

constexpr int kRThreads = 256, kRWarps = kRThreads / 32;
constexpr int kRRows = 4;          // most rows of a block (append)
constexpr int kRPairs = 128;       // most pairs of a head
// The angle's fraction of a turn rounded to f32 (2^-25 half turns: 9.4e-8), sincospif (2 ulp at most:
// 1.2e-7), mag, two products and their sum (2^-24 each): below 4e-7 of |u| + |v|.
constexpr float kTol = 0x1p-20f;

// The last b with row_start[b] <= row (0 if none), by a whole warp: 32 probes a step.
__device__ __forceinline__ int find_seq4(const int32_t* row_start, int B, int row) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lo + (int)(threadIdx.x & 31) * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < lo + n && row_start[i] <= row);
    const int k = m ? 31 - __clz(m) : 0;   // ascending: the last probe at or below the row
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// Where a packed row lies: the pool's row of (page, head 0, slot), -1 where it lies nowhere; live:
// it belongs to a sequence. By a whole warp.
struct RowSlot {
  bool live;
  long long at;
  uint32_t bits;
};
__device__ __forceinline__ RowSlot row_slot(const PagedMap& m, int T, int row) {
  const int b = find_seq4(m.row_start, m.B, row);
  const int r0 = m.row_start[b], r1 = m.row_start[b + 1], len = m.lens[b];
  // a row behind the last sequence or before the first belongs to none
  const bool none = (row >= r1 && b == m.B - 1 && r1 >= r0 && r1 >= 0) || (row < r0 && b == 0);
  const bool bad = !none && (r0 < 0 || r1 > T || row < r0 || row >= r1);
  RowSlot s{!none && !bad, -1, bad ? SWA_DERR_SEGMENT : 0u};
  if (!s.live) return s;
  const long long slot = (long long)len - r1 + row;
  if (len < 0 || len > m.cap || slot < 0) {
    s.bits |= SWA_DERR_META;
    return s;
  }
  const int page = m.table[(size_t)b * m.max_pages + (size_t)(slot >> m.page_shift)];
  if (page_ok(m, page))
    s.at = ((long long)page * m.nk << m.page_shift) + (slot & ((1 << m.page_shift) - 1));
  else
    s.bits |= SWA_DERR_PAGE;
  return s;
}

// Lower three bits of the code of y >= 0 in units u (scale * 2^exp): two borders at a time; each
// comparison is one with a border next to y or one that y is far from. near: y is within tol of one.
template <typename F>
__device__ __forceinline__ uint32_t level_code(F y, F u, F tol, bool& near) {
  const F b4 = F(1.75) * u;
  const bool c4 = y >= b4;
  const F b2 = (c4 ? F(3.5) : F(0.75)) * u;
  const bool c2 = y >= b2;
  const F b1 = (c4 ? (c2 ? F(5) : F(2.5)) : (c2 ? F(1.25) : F(0.25))) * u;
  const bool c1 = y > b1;
  near |= fabs(y - b4) <= tol || fabs(y - b2) <= tol || fabs(y - b1) <= tol;
  return c4 * 4 + c2 * 2 + c1;
}

// The same from angles in f64, for a warp whose head f32 left open. x, b: this lane's features and
// their partners; sign: how the partner enters; e: the feature's pair, -1 where it does not turn.
template <int E>
__device__ __noinline__ void encode_exact(const float (&x)[E], const float (&b)[E], const int (&e)[E], const float (&sign)[E],
                                          int pos, const uint64_t* turns, float mag, float div, float mul, uint32_t& codes,
                                          uint32_t& scale) {
  constexpr int L = kBlock4 / E;
  double y[E], top = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    y[j] = x[j];
    if (e[j] >= 0) {
      double sn, cs;
      sincospi((double)(int64_t)((uint64_t)(int64_t)pos * turns[e[j]]) * 0x1p-63, &sn, &cs);
      y[j] = (x[j] * cs + (double)sign[j] * b[j] * sn) * mag;
    }
    top = fmax(top, fabs(y[j]));
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  const double t = fmin(top * div / 6.0, 448.0);
  const int k = t < 0x1p-6 ? -9 : ilogb(t) - 3;          // three bits behind the leading one
  const double s = scalbn(rint(scalbn(t, -k)), k);
  scale = f32_e4m3((float)s);
  codes = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    bool near = false;
    const uint32_t c = s > 0 ? level_code<double>(fabs(y[j]), s * mul, 0.0, near) | (y[j] < 0 ? 8u : 0u) : 0u;
    codes |= c << (4 * j);
  }
}

template <typename TI, typename TQ, int E>
__global__ void __launch_bounds__(kRThreads) paged4_append_kernel(const Rows4Params p, const int inter) {
  constexpr int HD = 32 * E, L = kBlock4 / E;            // lanes of a block
  __shared__ __align__(16) float s_cos[kRRows * kRPairs], s_sin[kRRows * kRPairs];
  __shared__ long long s_at[kRRows];
  __shared__ bool s_live[kRRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x * p.R, nr = min(p.R, p.T - row0), h0 = blockIdx.y * p.Hg, nh = min(p.Hg, p.H - h0);
  const int half = p.rot >> 1, f0 = lane * E, items = nr * nh;
  const bool whole = half % E == 0;                      // a lane's partners are as consecutive and as aligned as its features
  // Head x of the block: this lane's features, and their partners where pairs are halves apart
  struct Item {
    int r, h, kind;                                      // 0: q, 1: k, 2: v
    Pack<TI, E> a, b;
  };
  auto load = [&](int x, Item& it) {
    if (x >= items) return;
    it.r = x / nh;
    it.h = h0 + x - it.r * nh;
    it.kind = it.h < p.nh ? 0 : it.h < p.nh + p.map.nk ? 1 : 2;
    const long long row = row0 + it.r;
    const TI* src;
    if (it.kind == 0) {
      src = static_cast<const TI*>(p.q) + row * p.q_row;
    } else if (it.kind == 1) {
      it.h -= p.nh;
      src = static_cast<const TI*>(p.k) + row * p.k_row;
    } else {
      it.h -= p.nh + p.map.nk;
      src = static_cast<const TI*>(p.v) + row * p.v_row;
    }
    src += (long long)it.h * HD;
    it.a = load_pack<E>(src + f0);
    if (inter || it.kind == 2 || f0 >= p.rot) return;
    if (whole) {
      it.b = load_pack<E>(src + (f0 < half ? f0 + half : f0 - half));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (f0 + j < p.rot) it.b.e[j] = src[f0 + j < half ? f0 + j + half : f0 + j - half];
    }
  };
  pdl_wait();
  pdl_trigger();
  Item cur, next;
  load(warp, cur);
  for (int i = tid; i < nr * half; i += kRThreads) {
    const int r = i / half, e = i % half;
    const uint64_t frac = (uint64_t)(int64_t)p.pos[row0 + r] * p.turns[e];   // modulo 2^64: the fraction of a turn
    float sn, cs;
    sincospif((float)(int32_t)(uint32_t)(frac >> 32) * 0x1p-31f, &sn, &cs);
    s_cos[i] = cs * p.mag;
    s_sin[i] = sn * p.mag;
  }
  const int r = kRWarps - 1 - warp;                      // the last warps: the first ones hold angles
  if (r < nr) {
    const RowSlot s = row_slot(p.map, p.T, row0 + r);
    if (lane == 0) {
      s_live[r] = s.live;
      s_at[r] = s.at;
      if (s.bits && blockIdx.y == 0) set_err(p.err, s.bits);
    }
  }
  __syncthreads();

  for (int x = warp; x < items; x += kRWarps) {
    load(x + kRWarps, next);
    const long long at = s_at[cur.r];
    if (s_live[cur.r] && (cur.kind == 0 || at >= 0)) {
      float a[E], b[E], y[E], sign[E];
      int e[E];
      unpack(cur.a, a);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int f = f0 + j;
        e[j] = -1;
        sign[j] = 0.f;
        b[j] = 0.f;
        y[j] = a[j];
        if (cur.kind == 2 || f >= p.rot) continue;
        if (inter) {
          e[j] = f >> 1;
          sign[j] = f & 1 ? 1.f : -1.f;
          b[j] = a[j ^ 1];
        } else {
          e[j] = f < half ? f : f - half;
          sign[j] = f < half ? -1.f : 1.f;
          b[j] = to_f32(cur.b.e[j]);
        }
        const int i = cur.r * half + e[j];
        y[j] = a[j] * s_cos[i] + sign[j] * b[j] * s_sin[i];
      }
      if (cur.kind == 0) {
        store_pack(static_cast<TQ*>(p.q_out) + ((long long)(row0 + cur.r) * p.nh + cur.h) * HD + f0, y);
      } else {
        const bool is_k = cur.kind == 1;
        const float div = is_k ? p.k_div : p.v_div, mul = is_k ? p.c.k_mul : p.c.v_mul;
        float top = 0.f, tol[E], tol_top = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          top = fmaxf(top, fabsf(y[j]));
          bad |= !(fabsf(y[j]) <= 3.402823466e38f);
          tol[j] = e[j] >= 0 ? kTol * fabsf(p.mag) * (fabsf(a[j]) + fabsf(b[j])) : 0.f;
          tol_top = fmaxf(tol_top, tol[j]);
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          tol_top = fmaxf(tol_top, __shfl_xor_sync(0xffffffffu, tol_top, o));
          bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
        }
        uint32_t scale = f32_e4m3(top * div / 6.f), codes = 0;
        bool open = tol_top > 0.f && f32_e4m3((top - tol_top) * div / 6.f) != f32_e4m3((top + tol_top) * div / 6.f);
        const float u = e4m3_f32(scale) * mul;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          bool near = false;
          const uint32_t c = u > 0.f ? level_code<float>(fabsf(y[j]), u, tol[j], near) | (y[j] < 0.f ? 8u : 0u) : 0u;
          codes |= c << (4 * j);
          open |= near && tol[j] > 0.f;
        }
        if (__any_sync(0xffffffffu, open && !bad))
          encode_exact<E>(a, b, e, sign, p.pos[row0 + cur.r], p.turns, p.mag, div, mul, codes, scale);
        if (bad) {
          codes = 0;
          scale = 0x7f;
        }
        const long long key = at + ((long long)cur.h << p.map.page_shift);
        uint8_t* const to = (is_k ? p.c.k : p.c.v) + key * (HD / 2) + lane * (E / 2);
        if constexpr (E == 2) *to = (uint8_t)codes;
        else if constexpr (E == 4) *reinterpret_cast<uint16_t*>(to) = (uint16_t)codes;
        else *reinterpret_cast<uint32_t*>(to) = codes;
        if (lane % L == 0) (is_k ? p.c.ks : p.c.vs)[key * (HD / kBlock4) + lane / L] = (uint8_t)scale;
      }
    }
    cur = next;
  }
}

// A thread takes 8 features at a time.
template <typename TO, int HD>
__global__ void __launch_bounds__(kRThreads) paged4_read_kernel(const Rows4Params p) {
  constexpr int U = HD / 8;
  __shared__ long long s_at[kRWarps];
  __shared__ bool s_live[kRWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nk = p.map.nk;
  const int row0 = blockIdx.x * p.R, nr = min(p.R, p.T - row0);
  pdl_wait();
  pdl_trigger();
  if (warp < nr) {
    const RowSlot s = row_slot(p.map, p.T, row0 + warp);
    if (lane == 0) {
      s_live[warp] = s.live;
      s_at[warp] = s.at;
      if (s.bits) set_err(p.err, s.bits);
    }
  }
  __syncthreads();
  const int units = 2 * nr * nk * U;                     // K of all rows, then V: below 2^26
  for (int x = tid; x < units; x += kRThreads) {
    const int u = x % U, y = x / U, z = y / nk, g = y - z * nk, r = z < nr ? z : z - nr;
    const bool is_v = z >= nr;
    TO* const out = static_cast<TO*>(is_v ? p.v_out : p.k_out);
    if (!out || !s_live[r]) continue;
    float f[8] = {};
    if (s_at[r] >= 0) {
      const long long key = s_at[r] + ((long long)g << p.map.page_shift);
      const uint32_t c = *reinterpret_cast<const uint32_t*>((is_v ? p.c.v : p.c.k) + key * (HD / 2) + u * 4);
      const float s = e4m3_f32((is_v ? p.c.vs : p.c.ks)[key * (HD / kBlock4) + u / 2]) * (is_v ? p.c.v_mul : p.c.k_mul);
      const uint32_t h[4] = {e2m1x2_f16x2<0>(c), e2m1x2_f16x2<1>(c), e2m1x2_f16x2<2>(c), e2m1x2_f16x2<3>(c)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = t.x * s;
        f[2 * i + 1] = t.y * s;
      }
    }
    store_pack(out + ((long long)(row0 + r) * nk + g) * HD + u * 8, f);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int paged4_cache_status(const swa_paged4_cache* c) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->lens || !c->row_start) return SWA_E_NULL;
  if (c->B < 1 || c->B > 65535 || c->nk < 1 || c->nk > 65535 || (long long)c->B * c->nk > (1 << 24)) return SWA_E_SHAPE;
  if (c->hd != 64 && c->hd != 128 && c->hd != 256) return SWA_E_SHAPE;
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return SWA_E_SHAPE;
  if (c->num_pages < 1 || (long long)c->num_pages * c->nk >= (1LL << 31) / c->page) return SWA_E_SHAPE;
  if (c->max_pages < 1 || c->max_pages > (1 << 30) / c->page) return SWA_E_SHAPE;
  if (c->k_exp < -32 || c->k_exp > 32 || c->v_exp < -32 || c->v_exp > 32) return SWA_E_SHAPE;
  if (!aligned16p(c->k) || !aligned16p(c->v) || !aligned16p(c->k_scale) || !aligned16p(c->v_scale) ||
      (reinterpret_cast<uintptr_t>(c->table) & 3u) || (reinterpret_cast<uintptr_t>(c->row_start) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->lens) & 3u))
    return SWA_E_ALIGN;
  return SWA_OK;
}

PagedMap paged4_map(const swa_paged4_cache* c) {
  PagedMap m{};
  m.B = c->B; m.nk = c->nk; m.num_pages = c->num_pages; m.max_pages = c->max_pages;
  while ((1 << m.page_shift) < c->page) ++m.page_shift;
  m.cap = c->max_pages << m.page_shift;
  m.table = c->table; m.row_start = c->row_start; m.lens = c->lens;
  return m;
}

Pools4 paged4_pools(const swa_paged4_cache* c) {
  return {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->k_scale), static_cast<uint8_t*>(c->v),
          static_cast<uint8_t*>(c->v_scale), std::ldexp(1.f, c->k_exp), std::ldexp(1.f, c->v_exp)};
}

void paged4_spans(const swa_paged4_cache* c, Span4 (&s)[4]) {
  const size_t keys = (size_t)c->num_pages * c->nk * c->page;
  s[0] = {c->k, keys * c->hd / 2};
  s[1] = {c->k_scale, keys * c->hd / kBlock4};
  s[2] = {c->v, keys * c->hd / 2};
  s[3] = {c->v_scale, keys * c->hd / kBlock4};
}

template <typename TI, typename TQ>
static int launch_append(Rows4Params& p, int inter, cudaStream_t s) {
  // all heads of kRRows rows once that gives every SM four blocks, else a row and a head a warp
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  p.R = p.T >= 4 * sms * kRRows ? kRRows : 1;
  p.Hg = p.T >= 4 * sms ? p.H : kRWarps;
  if ((p.H + p.Hg - 1) / p.Hg > 65535) p.Hg = (p.H + 65534) / 65535;
  const dim3 grid((unsigned)((p.T + p.R - 1) / p.R), (unsigned)((p.H + p.Hg - 1) / p.Hg)), block(kRThreads);
  return finish_launch(p.hd == 64    ? launch_pdl(paged4_append_kernel<TI, TQ, 2>, grid, block, 0, s, p, inter)
                       : p.hd == 128 ? launch_pdl(paged4_append_kernel<TI, TQ, 4>, grid, block, 0, s, p, inter)
                                     : launch_pdl(paged4_append_kernel<TI, TQ, 8>, grid, block, 0, s, p, inter));
}

template <typename TO>
static int launch_read(Rows4Params& p, cudaStream_t s) {
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  p.R = p.T >= 8 * sms * kRWarps ? kRWarps : p.T >= 16 * sms ? 2 : 1;
  const dim3 grid((unsigned)((p.T + p.R - 1) / p.R)), block(kRThreads);
  return finish_launch(p.hd == 64    ? launch_pdl(paged4_read_kernel<TO, 64>, grid, block, 0, s, p)
                       : p.hd == 128 ? launch_pdl(paged4_read_kernel<TO, 128>, grid, block, 0, s, p)
                                     : launch_pdl(paged4_read_kernel<TO, 256>, grid, block, 0, s, p));
}

static int type_bytes4(int t) { return t == SWA_F32 ? 4 : 2; }
static bool type_ok(int t) { return t == SWA_F32 || t == SWA_BF16 || t == SWA_F16; }

}  // namespace swa

using namespace swa;

extern "C" {

int swa_paged4_append(const swa_paged4_append_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged4_cache& c = a->cache;
  const int rc = paged4_cache_status(&c);
  if (rc != SWA_OK) return rc;
  const int nh = a->q || a->q_out ? a->nh : 0;
  if (a->T < 0 || a->nh < 0 || a->nh >= (1 << 20) || a->rot < 0 || (a->rot & 1) || a->rot > c.hd) return SWA_E_SHAPE;
  if (!type_ok(a->src) || !std::isfinite(a->mag)) return SWA_E_SHAPE;
  const long long H = (long long)nh + 2LL * c.nk;
  if (H >= (1 << 21) || (long long)a->T * H >= (1LL << 40) / c.hd) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->k || !a->v || (a->q != nullptr) != (a->q_out != nullptr)) return SWA_E_NULL;
  if (a->rot > 0 && (!a->pos || !a->turns)) return SWA_E_NULL;
  if (a->q && (a->nh < 1 || (a->q_dtype != SWA_BF16 && a->q_dtype != SWA_F16))) return SWA_E_SHAPE;
  const int w = type_bytes4(a->src);
  const long long kd = (long long)c.nk * c.hd, qd = (long long)nh * c.hd;
  const long long kn = rows_span(a->T, kd, a->k_row), vn = rows_span(a->T, kd, a->v_row);
  const long long qn = a->q ? rows_span(a->T, qd, a->q_row) : 0;
  if (kn < 0 || vn < 0 || qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->k) || !aligned16p(a->v) || !aligned16p(a->q) || !aligned16p(a->q_out) ||
      ((a->k_row | a->v_row | (a->q ? a->q_row : 0)) * w & 15) || (reinterpret_cast<uintptr_t>(a->pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->turns) & 7u))
    return SWA_E_ALIGN;
  if (a->q) {
    const bool same = a->q == a->q_out && a->src == a->q_dtype && a->q_row == qd;
    const size_t on = (size_t)a->T * qd * 2;
    if ((!same && bytes_overlap(a->q, (size_t)qn * w, a->q_out, on)) ||
        bytes_overlap(a->k, (size_t)kn * w, a->q_out, on) || bytes_overlap(a->v, (size_t)vn * w, a->q_out, on))
      return SWA_E_SHAPE;
  }
  Span4 pool[4];
  paged4_spans(&c, pool);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (bytes_overlap(pool[i].at, pool[i].bytes, pool[j].at, pool[j].bytes)) return SWA_E_SHAPE;
  Rows4Params p{};
  p.map = paged4_map(&c);
  p.c = paged4_pools(&c);
  p.T = a->T; p.hd = c.hd; p.nh = nh; p.H = (int)H; p.rot = a->rot; p.mag = a->mag;
  p.q = a->q; p.k = a->k; p.v = a->v; p.q_row = a->q_row; p.k_row = a->k_row; p.v_row = a->v_row;
  p.q_out = a->q_out; p.pos = a->pos; p.turns = a->turns;
  p.k_div = 1.f / p.c.k_mul; p.v_div = 1.f / p.c.v_mul;
  p.err = a->err;
  const int inter = a->interleaved != 0;
  const bool bf = a->q_dtype == SWA_BF16;
  switch (a->src) {
    case SWA_F32: return bf ? launch_append<float, __nv_bfloat16>(p, inter, stream) : launch_append<float, __half>(p, inter, stream);
    case SWA_BF16: return bf ? launch_append<__nv_bfloat16, __nv_bfloat16>(p, inter, stream) : launch_append<__nv_bfloat16, __half>(p, inter, stream);
    default: return bf ? launch_append<__half, __nv_bfloat16>(p, inter, stream) : launch_append<__half, __half>(p, inter, stream);
  }
}

int swa_paged4_read(const swa_paged4_read_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged4_cache& c = a->cache;
  const int rc = paged4_cache_status(&c);
  if (rc != SWA_OK) return rc;
  if (a->T < 0 || !type_ok(a->dtype) || (long long)a->T * c.nk >= (1LL << 40) / c.hd) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->k_out && !a->v_out) return SWA_E_NULL;
  if (!aligned16p(a->k_out) || !aligned16p(a->v_out)) return SWA_E_ALIGN;
  const size_t n = (size_t)a->T * c.nk * c.hd * type_bytes4(a->dtype);
  Span4 pool[4];
  paged4_spans(&c, pool);
  for (const Span4& s : pool)
    if ((a->k_out && bytes_overlap(a->k_out, n, s.at, s.bytes)) || (a->v_out && bytes_overlap(a->v_out, n, s.at, s.bytes)))
      return SWA_E_SHAPE;
  if (a->k_out && a->v_out && bytes_overlap(a->k_out, n, a->v_out, n)) return SWA_E_SHAPE;
  Rows4Params p{};
  p.map = paged4_map(&c);
  p.c = paged4_pools(&c);
  p.T = a->T; p.hd = c.hd;
  p.k_out = a->k_out; p.v_out = a->v_out;
  p.err = a->err;
  return a->dtype == SWA_F32 ? launch_read<float>(p, stream) : a->dtype == SWA_BF16 ? launch_read<__nv_bfloat16>(p, stream)
                                                                                   : launch_read<__half>(p, stream);
}

}  // extern "C"
