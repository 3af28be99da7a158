// Rows into and out of the 4-bit paged cache: swa_paged4_append (rotary positions, encoding,
// and the rotation of q) and swa_paged4_read.
//
// Encoding is exact in the sense that the stored codes are those of the formula, not of its f32
// arithmetic. A border between two levels (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5) times a scale has seven
// bits, and so has six times a border between two scales: an f32 that is not on the border is so far
// from it that the quotient, correctly rounded, is on the same side. The quotients x / 6 and x / scale
// are correctly rounded by a product with the rounded reciprocal and one step of correction (all 2^23
// mantissas were compared, for 6 and for the eight mantissas of a scale). Values that were not rotated
// are thus encoded exactly. A rotated value is known up to kTol * (|u| + |v|); where that leaves
// a scale or a code open (one head in some hundreds) the warp takes the angles and the encoding again in f64.
//
// Bound by memory and by the instructions of the encoding: a lane takes half a block of a row's head, a warp one head
// of one to four rows, so that a pair's other half is in a lane of the same warp, a block's largest value one shuffle away,
// and every access consecutive. 8192 rows of 32 heads of q and 8 of k and v, hd 128, from f32: 62 us, where their bytes
// take 41; 24 of them are the encoding of k and v (33 with positions).
#include <cmath>
#include <cstring>

#include "swa_paged4.cuh"

namespace swa {

struct Rows4Params {
  PagedMap map;
  Pools4 c;
  int T, hd, R;                // rows of a block
  // append: heads [0, nh) are q, [nh, nh + nk) k, [nh + nk, H) v
  int nh, H, Hg, rot, q_bf;    // Hg heads of a block; q_out is bf16, else f16
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
constexpr int kE = 8;              // features of a lane (append): half a block
template <int HD>
struct AppendCfg {
  static constexpr int LANES = HD / kE, ROWS_WARP = 32 / LANES;   // of a head; rows that a warp takes at once
  static constexpr int ROWS = HD == 64 ? 8 : 4;                   // most rows of a block
};
// How far a rotated value, the quotients made of it and the ends of their interval may be off in f32, in all and at most, as
// a part of |u| + |v| (times mag), in units of 2^-24: sincospif an ulp (1), the step that adds what the angle's f32 lacks 0.5,
// mag 1, the product and the fused sum 1 each: 4.5. For codes the quotient and an end, which has to pass the border: 3. For scales
// an end's sum, 1 / 6, the product with it, and passing the border: 5. (tests/test_paged4_encoding_cpu.py)
constexpr float kTol = 0x1.4p-21f;       // 10 of these

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

// Codes -0 become 0, in all nibbles
__device__ __forceinline__ uint32_t plain_zeros(uint32_t c) { return c & (((c & 0x77777777u) + 0x77777777u) | 0x77777777u); }
// The codes of two values in units of their scale (ties to even, 6 at most), the first in the lower half
__device__ __forceinline__ uint32_t f32x2_e2m1(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %1, %2;\n\tcvt.u32.u8 %0, a;\n\t}" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The largest of three, NaN if one is
__device__ __forceinline__ float nan_max(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int E>
__device__ __forceinline__ uint32_t codes_of(const float (&z)[E]) {
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < E; j += 2) c |= f32x2_e2m1(z[j], z[j + 1]) << (4 * j);
  return plain_zeros(c);
}

// The encoding of the blocks that f32 left open, from angles in f64, by a warp. x, b: a lane's features and their
// partners with the sign that they enter by; e: the feature's pair, -1 where it does not turn; pos: its row's.
// A lane takes one feature of a block: a chain of f64 operations takes long.
__device__ __noinline__ void encode_exact(const float (&x)[kE], const float (&b)[kE], const int (&e)[kE], unsigned open, int pos,
                                          const uint64_t* turns, float mag, float div, uint32_t& codes, uint32_t& scale) {
  constexpr int L = kBlock4 / kE;
  const int lane = threadIdx.x & 31;
  while (open) {
    const int block = (__ffs(open) - 1) / L, i = lane & 15, owner = block * L + i / kE;
    open &= ~(((1u << L) - 1) << (block * L));
    float xi = 0.f, bi = 0.f;
    int ei = -1;
    const int at = __shfl_sync(0xffffffffu, pos, owner);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const float xj = __shfl_sync(0xffffffffu, x[j], owner), bj = __shfl_sync(0xffffffffu, b[j], owner);
      const int ej = __shfl_sync(0xffffffffu, e[j], owner);
      if (i % kE == j) {
        xi = xj;
        bi = bj;
        ei = ej;
      }
    }
    double y = xi;
    if (ei >= 0) {
      double sn, cs;
      sincospi((double)(int64_t)((uint64_t)(int64_t)at * turns[ei]) * 0x1p-63, &sn, &cs);
      y = ((double)xi * cs + (double)bi * sn) * mag;
    }
    y *= div;
    const double m = fabs(y);
    double top = m;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    const double t = fmin(top / 6.0, 448.0);
    const int k = t < 0x1p-6 ? -9 : ilogb(t) - 3;        // three bits behind the leading one
    const double s = scalbn(rint(scalbn(t, -k)), k);
    uint32_t c = 0;
    if (s > 0) c = (m > 0.25 * s) + (m >= 0.75 * s) + (m > 1.25 * s) + (m >= 1.75 * s) + (m > 2.5 * s) + (m >= 3.5 * s) + (m > 5.0 * s);
    if (c && y < 0) c |= 8u;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kE; ++j) mine |= __shfl_sync(0xffffffffu, c, (lane % L) * kE + j) << (4 * j);
    if (lane / L == block) {
      codes = mine;
      scale = f32_e4m3((float)s);
    }
  }
}

// PAIRS: how the features of a pair lie. 0: half of the turned ones apart, and a lane's partners are those
// of one other lane; 1: next to each other; 2: as 0 with partners in two lanes (half % kE != 0).
template <typename TI, int HD, int PAIRS>
__global__ void __launch_bounds__(kRThreads, sizeof(TI) == 2 ? 4 : 3) paged4_append_kernel(const __grid_constant__ Rows4Params p) {
  using C = AppendCfg<HD>;
  constexpr int LH = C::LANES, RP = C::ROWS_WARP, TIMES = C::ROWS / RP, L = kBlock4 / kE;   // L: lanes of a block
  __shared__ __align__(16) float s_cos[C::ROWS * (HD / 2)], s_sin[2][C::ROWS * (HD / 2)];   // [0]: -sin, of a pair's first feature
  __shared__ long long s_at[C::ROWS];      // -2: of no sequence, -1: not stored
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x * p.R, nr = min(p.R, p.T - row0), h0 = blockIdx.y * p.Hg, n = min(p.Hg, p.H - h0);
  const int half = p.rot >> 1, sub = lane % LH, f0 = sub * kE, row_w = lane / LH, nq = p.nh, nqk = p.nh + p.map.nk;
  // A warp takes the heads warp, warp + 8, .. of the block, of each all rows. The next head's are loaded while these
  // are worked on where they lie in more than 16 bytes a lane; else another CTA fits (8192 rows of 32 + 16 heads, hd 128:
  // f32 62 us, 65 the other way; bf16 62, 66).
  constexpr bool AHEAD = sizeof(TI) == 4 && HD < 256;
  struct Rows {
    Pack<TI, kE> a[TIMES];
  };
  auto load = [&](Rows& t, int x) {
    const int h = h0 + x;
    const TI* src;
    long long row;
    if (h < nq) {
      src = static_cast<const TI*>(p.q) + (long long)h * HD;
      row = p.q_row;
    } else if (h < nqk) {
      src = static_cast<const TI*>(p.k) + (long long)(h - nq) * HD;
      row = p.k_row;
    } else {
      src = static_cast<const TI*>(p.v) + (long long)(h - nqk) * HD;
      row = p.v_row;
    }
    src += (row0 + row_w) * row + f0;
#pragma unroll
    for (int i = 0; i < TIMES; ++i, src += RP * row) {
      t.a[i] = Pack<TI, kE>{};
      if (i * RP + row_w < nr) t.a[i] = load_pack<kE>(src);
    }
  };
  // The largest of a block's values (NaN where one is) in units of 2^exp; its scale and the reciprocal
  struct Scale {
    float top, u, inv;
    uint32_t bits;
    bool bad;
  };
  // y in units of 2^exp afterwards
  auto scale_of = [&](float (&y)[kE], float div) {
    float m = fabsf(y[0]);
#pragma unroll
    for (int j = 1; j + 1 < kE; j += 2) m = nan_max(m, fabsf(y[j]), fabsf(y[j + 1]));
    m = nan_max(m, fabsf(y[kE - 1]), m);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, o), m);
    Scale s;
    s.bad = !(m < INFINITY);
    s.top = m * div;
    if (div != 1.f) {
#pragma unroll
      for (int j = 0; j < kE; ++j) y[j] *= div;
    }
    if (__any_sync(0xffffffffu, s.top > 4096.f)) {       // 448 * 6 and more take the largest scale
      s.top = fminf(s.top, 4096.f);
#pragma unroll
      for (int j = 0; j < kE; ++j) y[j] = fminf(fmaxf(y[j], -4096.f), 4096.f);
    }
    float q = s.top * (1.f / 6.f);
    q = fmaf(fmaf(-6.f, q, s.top), 1.f / 6.f, q);
    s.bits = f32_e4m3(q);
    s.u = e4m3_f32(s.bits);
    // correctly rounded: one step from an ulp away (tests/test_gpu_paged4.py has every scale)
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s.u));
    s.inv = s.u > 0.f ? fmaf(fmaf(-s.u, inv, 1.f), inv, inv) : 0.f;
    return s;
  };
  auto quotients = [&](float (&y)[kE], const Scale& s) {
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const float q = y[j] * s.inv;
      y[j] = fmaf(fmaf(-q, s.u, y[j]), s.inv, q);
    }
  };
  auto store = [&](uint8_t* to_codes, uint8_t* to_scales, long long at, int g, uint32_t codes, uint32_t scale) {
    if (at < 0) return;
    const long long key = at + ((long long)g << p.map.page_shift);
    *reinterpret_cast<uint32_t*>(to_codes + key * (HD / 2) + sub * (kE / 2)) = codes;
    if (sub % L == 0) to_scales[key * (HD / kBlock4) + sub / L] = (uint8_t)scale;
  };
  auto row_of = [&](int i) { return min(i * RP + row_w, nr - 1); };   // a lane without a row takes the last one's place
  auto at_of = [&](int i) { return i * RP + row_w < nr ? s_at[i * RP + row_w] : -2; };
  auto work_v = [&](int i, int g, const Pack<TI, kE>& raw) {
    const long long at = at_of(i);
    float x[kE];
    unpack(raw, x);
    const Scale s = scale_of(x, p.v_div);
    quotients(x, s);
    store(p.c.v, p.c.vs, at, g, s.bad ? 0u : codes_of(x), s.bad ? 0x7fu : s.bits);
  };
  // the rotation: y = x cos + b sin, b the partner with its sign; f0 < half and the partner's lane are the same
  // for all rows
  const bool low = f0 < half;
  const int partner = (low ? lane + half / kE : lane - half / kE) & 31, pair0 = low ? f0 : f0 - half;
  auto pair_of = [&](int j) {              // of feature f0 + j, -1: it does not turn
    const int f = f0 + j;
    if (f >= p.rot) return -1;
    return PAIRS == 1 ? f >> 1 : f < half ? f : f - half;
  };
  auto first_of = [&](int j) { return PAIRS == 1 ? !(j & 1) : PAIRS == 0 ? low : f0 + j < half; };   // of its pair
  auto rotate = [&](int r, const Pack<TI, kE>& raw, const TI* src, float (&x)[kE], float (&b)[kE], float (&y)[kE]) {
    unpack(raw, x);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      y[j] = x[j];
      b[j] = 0.f;
    }
    if (PAIRS == 0) {
      Pack<TI, kE> other;                                // of lane +- half / kE
      constexpr int W = sizeof(raw) / 4;
      uint32_t mine[W], theirs[W];
      memcpy(mine, &raw, sizeof(raw));
#pragma unroll
      for (int i = 0; i < W; ++i) theirs[i] = __shfl_sync(0xffffffffu, mine[i], partner);
      memcpy(&other, theirs, sizeof(other));
      if (f0 < p.rot) {
        float c[kE], sn[kE];
        unpack(load_pack<kE>(s_cos + r * half + pair0), c);
        unpack(load_pack<kE>(s_sin[!low] + r * half + pair0), sn);
        unpack(other, b);
#pragma unroll
        for (int j = 0; j < kE; ++j) y[j] = fmaf(b[j], sn[j], x[j] * c[j]);
      }
    } else if (PAIRS == 1) {
#pragma unroll
      for (int j = 0; j < kE; j += 2) {
        if (f0 + j >= p.rot) continue;
        const int i = r * half + (f0 + j) / 2;
        const float c = s_cos[i], sn = s_sin[1][i];
        b[j] = x[j + 1];
        b[j + 1] = x[j];
        y[j] = fmaf(-x[j + 1], sn, x[j] * c);
        y[j + 1] = fmaf(x[j], sn, x[j + 1] * c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        const int f = f0 + j, e = pair_of(j);
        if (e < 0) continue;
        b[j] = to_f32(src[f < half ? f + half : f - half]);
        y[j] = fmaf(b[j], s_sin[f >= half][r * half + e], x[j] * s_cos[r * half + e]);
      }
    }
  };
  auto work_q = [&](int i, int h, const Pack<TI, kE>& raw) {
    const int r = row_of(i);
    float x[kE], b[kE], y[kE];
    rotate(r, raw, static_cast<const TI*>(p.q) + (row0 + r) * p.q_row + (long long)h * HD, x, b, y);
    if (PAIRS == 2) __syncwarp();                        // q_out may be q, whose partners other lanes read
    if (at_of(i) == -2) return;
    const long long to = ((long long)(row0 + r) * nq + h) * HD + f0;
    if (p.q_bf) store_pack(static_cast<__nv_bfloat16*>(p.q_out) + to, y);
    else store_pack(static_cast<__half*>(p.q_out) + to, y);
  };
  auto work_k = [&](int i, int g, const Pack<TI, kE>& raw) {
    const int r = row_of(i);
    const long long at = at_of(i);
    float x[kE], b[kE], y[kE];
    rotate(r, raw, static_cast<const TI*>(p.k) + (row0 + r) * p.k_row + (long long)g * HD, x, b, y);
    Scale s = scale_of(y, p.k_div);
    // how far y may be from the rotated value; at position 0 it is that
    const int pos = p.rot ? p.pos[row0 + r] : 0;
    float t = 0.f;                                       // |u| + |v| is 2 t at most; NaN where one is
#pragma unroll
    for (int j = 0; j < kE; j += 1 + (PAIRS == 1)) t = nan_max(t, fabsf(x[j]), fabsf(PAIRS == 1 ? x[j + 1] : b[j]));
    const float tol = (pos == 0 && p.mag == 1.f) || f0 >= p.rot ? 0.f : t * (2.f * kTol * fabsf(p.mag) * p.k_div);
    float tol_top = tol;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) tol_top = fmaxf(tol_top, __shfl_xor_sync(0xffffffffu, tol_top, o));
    quotients(y, s);
    float hi[kE];
    const float d = tol * s.inv;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      hi[j] = y[j] + d;
      y[j] -= d;
    }
    uint32_t codes = codes_of(y), scale = s.bits;
    const bool two = codes != codes_of(hi);
    if (__any_sync(0xffffffffu, s.bad)) {                // an infinity or NaN, or finite features whose rotation passes f32's range: open
#pragma unroll
      for (int o = 1; o < L; o <<= 1) t = nan_max(t, __shfl_xor_sync(0xffffffffu, t, o), t);
      if (s.bad && t < INFINITY) {
        s.bad = false;
        s.top = 0.f;
        tol_top = INFINITY;
      }
    }
    const bool open = at >= 0 && !s.bad && tol_top > 0.f &&
                      (two || f32_e4m3((s.top - tol_top) * (1.f / 6.f)) != f32_e4m3((s.top + tol_top) * (1.f / 6.f)));
    const unsigned any = __ballot_sync(0xffffffffu, open);
    if (any) {
      int e[kE];
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        e[j] = pair_of(j);
        if (first_of(j)) b[j] = -b[j];
      }
      encode_exact(x, b, e, any, pos, p.turns, p.mag, p.k_div, codes, scale);
    }
    store(p.c.k, p.c.ks, at, g, s.bad ? 0u : codes, s.bad ? 0x7fu : scale);
  };
  pdl_wait();
  pdl_trigger();
  Rows cur;
  if (warp < n) load(cur, warp);
  for (int i = tid; i < nr * half; i += kRThreads) {
    const int r = i / half, e = i % half;
    const uint64_t frac = (uint64_t)(int64_t)p.pos[row0 + r] * p.turns[e];   // modulo 2^64: the fraction of a turn
    const int32_t turn = (int32_t)(uint32_t)(frac >> 32);                    // in 2^-31 half turns
    const float f = (float)turn;
    float sn, cs;
    sincospif(f * 0x1p-31f, &sn, &cs);
    // what f lacks, in radians: below 2^-24, and 0 only where the angle is a whole number of half turns
    const float rest = fmaf((float)(turn - (int32_t)f), 0x1p-31f * 3.14159265f, (float)(uint32_t)frac * (0x1p-63f * 3.14159265f));
    s_cos[i] = fmaf(-sn, rest, cs) * p.mag;
    sn = fmaf(cs, rest, sn) * p.mag;
    s_sin[0][i] = -sn;
    s_sin[1][i] = sn;
  }
  if (const int r = kRWarps - 1 - warp; r < nr) {        // the last warps: the first ones hold angles
    const RowSlot s = row_slot(p.map, p.T, row0 + r);
    if (lane == 0) {
      s_at[r] = s.live ? s.at : -2;
      if (s.bits && blockIdx.y == 0) set_err(p.err, s.bits);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int x = warp; x < n; x += kRWarps) {
    Rows next;
    if (AHEAD && x + kRWarps < n) load(next, x + kRWarps);
    const int h = h0 + x;
    if (h < nq) {
#pragma unroll
      for (int i = 0; i < TIMES; ++i)
        if (i * RP < nr) work_q(i, h, cur.a[i]);
    } else if (h < nqk) {
#pragma unroll
      for (int i = 0; i < TIMES; ++i)
        if (i * RP < nr) work_k(i, h - nq, cur.a[i]);
    } else {
#pragma unroll
      for (int i = 0; i < TIMES; ++i)
        if (i * RP < nr) work_v(i, h - nqk, cur.a[i]);
    }
    if (AHEAD) cur = next;
    else if (x + kRWarps < n) load(cur, x + kRWarps);
  }
}

// A block takes some rows and heads (all of them, or one row's) in the order of the output; their keys' numbers
// stand in shared memory. A thread has the same 8 features of every head that it takes.
constexpr int kReadRows = 32, kReadHeads = 256, kReadKeys = 1024;   // most rows, heads and keys of a block
template <typename TO, int HD>
__global__ void __launch_bounds__(kRThreads, 6) paged4_read_kernel(const __grid_constant__ Rows4Params p) {
  constexpr int U = HD / 8, STEP = kRThreads / U, N = 4;
  __shared__ int s_key[kReadKeys];         // -2: of no sequence, -1: zeros
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x * p.R, nr = min(p.R, p.T - row0), h0 = blockIdx.y * p.Hg, nh = min(p.Hg, p.map.nk - h0);
  pdl_wait();
  pdl_trigger();
  for (int r = warp; r < nr; r += kRWarps) {
    const RowSlot s = row_slot(p.map, p.T, row0 + r);
    for (int g = lane; g < nh; g += 32)
      s_key[r * nh + g] = !s.live ? -2 : s.at < 0 ? -1 : (int)(s.at + ((long long)(h0 + g) << p.map.page_shift));   // below 2^31
    if (lane == 0 && s.bits && blockIdx.y == 0) set_err(p.err, s.bits);
  }
  __syncthreads();
  const int u = tid % U, keys = nr * nh;
  const long long base = ((long long)row0 * p.map.nk + h0) * HD + u * 8;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    TO* const out = static_cast<TO*>(side ? p.v_out : p.k_out) + base;
    if (!(side ? p.v_out : p.k_out)) continue;
    const uint8_t* const codes = (side ? p.c.v : p.c.k) + u * 4;
    const uint8_t* const scales = (side ? p.c.vs : p.c.ks) + u / 2;
    const float mul = side ? p.c.v_mul : p.c.k_mul;
    for (int y0 = tid / U; y0 < keys; y0 += N * STEP) {
      uint32_t c[N], s[N];
      int key[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int y = y0 + i * STEP;
        key[i] = y < keys ? s_key[y] : -2;
        c[i] = s[i] = 0;
        if (key[i] >= 0) {
          c[i] = *reinterpret_cast<const uint32_t*>(codes + (long long)key[i] * (HD / 2));
          s[i] = scales[(long long)key[i] * (HD / kBlock4)];
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (key[i] == -2) continue;
        const float m = e4m3_f32(s[i]) * mul;
        const uint32_t h[4] = {e2m1x2_f16x2<0>(c[i]), e2m1x2_f16x2<1>(c[i]), e2m1x2_f16x2<2>(c[i]), e2m1x2_f16x2<3>(c[i])};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
          f[2 * k] = t.x * m;
          f[2 * k + 1] = t.y * m;
        }
        store_pack(out + (long long)(y0 + i * STEP) * HD, f);
      }
    }
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

template <typename TI, int HD>
static cudaError_t launch_pairs(Rows4Params& p, int inter, cudaStream_t s) {
  // All heads of the most rows a block once that gives every SM four blocks, else the rows that a warp takes at once, and
  // a head a warp. (8192 rows of 32 + 16 heads in f32: 62 us, with fewer rows 72, with 8 heads a block 86.)
  using C = AppendCfg<HD>;
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  p.R = p.T >= 4 * sms * C::ROWS ? C::ROWS : C::ROWS_WARP;
  p.Hg = p.T >= 4 * sms * p.R ? p.H : kRWarps;
  if ((p.H + p.Hg - 1) / p.Hg > 65535) p.Hg = (p.H + 65534) / 65535;
  const dim3 grid((unsigned)((p.T + p.R - 1) / p.R), (unsigned)((p.H + p.Hg - 1) / p.Hg)), block(kRThreads);
  if (inter) return launch_pdl(paged4_append_kernel<TI, HD, 1>, grid, block, 0, s, p);
  if (p.rot / 2 % kE == 0) return launch_pdl(paged4_append_kernel<TI, HD, 0>, grid, block, 0, s, p);
  return launch_pdl(paged4_append_kernel<TI, HD, 2>, grid, block, 0, s, p);
}

template <typename TI>
static int launch_append(Rows4Params& p, int inter, cudaStream_t s) {
  return finish_launch(p.hd == 64 ? launch_pairs<TI, 64>(p, inter, s) : p.hd == 128 ? launch_pairs<TI, 128>(p, inter, s)
                                                                                   : launch_pairs<TI, 256>(p, inter, s));
}

template <typename TO>
static int launch_read(Rows4Params& p, cudaStream_t s) {
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  // rows of a block: 8 heads a thread and array, if that leaves every SM two blocks (46000 rows of 8 heads, hd 128: 43 us, with
  // one row a block 112)
  const long long row = (long long)p.map.nk * p.hd / 8, most = 8 * kRThreads / row;
  long long R = p.T / (2 * sms);
  R = R > most ? most : R;
  R = R > kReadRows ? kReadRows : R < 1 || p.map.nk > kReadHeads ? 1 : R;
  p.Hg = p.map.nk < kReadHeads ? p.map.nk : kReadHeads;
  p.R = (int)(R * p.Hg > kReadKeys ? kReadKeys / p.Hg : R);
  const dim3 grid((unsigned)((p.T + p.R - 1) / p.R), (unsigned)((p.map.nk + p.Hg - 1) / p.Hg)), block(kRThreads);
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
  p.q_bf = a->q_dtype == SWA_BF16;
  switch (a->src) {
    case SWA_F32: return launch_append<float>(p, inter, stream);
    case SWA_BF16: return launch_append<__nv_bfloat16>(p, inter, stream);
    default: return launch_append<__half>(p, inter, stream);
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
