// Rotary positions of packed rows (swa_rotary) and of a chunk that enters the
// paged cache (swa_paged_append).
//
// u' = u cos a - v sin a, v' = v cos a + u sin a with a = pos * f. The angle is
// taken modulo one turn in integers: turns = f / 2 pi as a 64-bit fraction, and
// pos * turns modulo 2^64 is the angle's fraction of a turn, exact but for the
// fraction's own last bit (2^-33 turns at 2^31 positions). Its upper 32 bits, signed (2^-32 turns),
// times 2^-31 are half turns in [-1, 1) once rounded to f32 (2^-26 turns at most), what sincospif
// takes: no f64 arithmetic (two lanes an SM here) and no range reduction, at any position.
//
// Memory bound: each element is read and written once. A block takes R rows and a group
// of heads: its threads first compute the rows' sines and cosines into shared memory (one
// or two a thread, used by all the heads) and, for the cache, the rows' slots; then each
// thread takes units (8 pairs, or 8 features when interleaved: 16-byte accesses for 16-bit
// types) of the rows' heads in turn. With the angles in registers instead, recomputed for
// every few heads, a prompt of 6000 f32 rows of 48 heads entered the cache at 3.6 TB/s.
// Halves that do not start at multiples of 8 features take units of 4, 2 or 1 pairs.
// Measured: 16383 f32 rows of 40 heads of 128: 101 us, 6.7 TB/s; 6000 f32 rows of 48 heads
// into the cache: 34 us, 5.8 TB/s.
#include <cmath>

#include "swa_paged.cuh"

namespace swa {

struct RotaryParams {
  int T, H, hd, rot, R, Hg, units, inverse;   // R rows and Hg heads a block
  uint64_t units_inv, heads_inv;              // ceil(2^32 / d) of units and Hg: x / d = x * inv >> 32, x < 2^20, d <= 2^11
  float mag;
  const void* x;               // rows of heads [0, H) (swa_rotary) or of q (append)
  long long x_row, x_head;
  void* out;
  long long out_row, out_head;
  const int32_t* pos;
  const uint64_t* turns;
  // append: heads [0, nh) are q, [nh, nh + nk) k, [nh + nk, nh + 2 nk) v
  int nh, nk, hd_page;         // hd_page = page * hd
  const void* k;
  const void* v;
  long long k_row, v_row;
  void* cache_k;
  void* cache_v;
  PagedMap map;
  int32_t* slot_pos;
  float* weight;
  uint32_t* err;
};

constexpr int kRotThreads = 256;
constexpr int kRotRows = 4;        // most rows of a block
constexpr int kRotPairs = 512;     // most pairs of a head

// The last b with row_start[b] <= row (0 if none), by a whole warp: 32 probes a step.
__device__ __forceinline__ int find_seq(const int32_t* row_start, int B, int row) {
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

// V: pairs (half layout: 1, 2, 4 or 8) or features (interleaved: 8) of a unit
template <typename TI, typename TO, bool INTER, int V, bool APPEND>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  __shared__ __align__(16) float s_cos[kRotRows * kRotPairs], s_sin[kRotRows * kRotPairs];
  __shared__ long long s_slot[kRotRows], s_aux[kRotRows];   // cache element of (page, head 0, slot); slot_pos entry
  __shared__ int s_live[kRotRows];
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * p.R, nr = min(p.R, p.T - row0), h0 = blockIdx.y * p.Hg, h1 = min(h0 + p.Hg, p.H);
  const int half = p.rot >> 1;
  constexpr int NP = INTER ? V / 2 : V;                 // pairs of a unit
  const int rot_units = INTER ? (p.rot + V - 1) / V : half / V;   // interleaved: the last may be turned in part
  const int nh = h1 - h0, items = nr * nh * p.units;
  // Unit x of the block: row, head and first feature
  struct Unit {
    int u, h, r, f0;
    bool turn;
  };
  auto unit = [&](int x) {
    Unit q;
    const int y = (int)((uint64_t)(unsigned)x * p.units_inv >> 32);
    q.u = x - y * p.units;
    q.r = (int)((uint64_t)(unsigned)y * p.heads_inv >> 32);
    if (nh != p.Hg) q.r = y / nh;                       // the last group of heads
    q.h = h0 + y - q.r * nh;
    q.turn = q.u < rot_units;
    q.f0 = INTER ? q.u * V : q.turn ? q.u * NP : p.rot + (q.u - rot_units) * V;
    return q;
  };
  // U units of a thread at a time. Those of the next step are loaded before this step's are
  // stored, and the first ones before the angles: out may be x, so the compiler keeps every
  // load behind the stores before it.
  constexpr int U = sizeof(TI) == 4 ? 1 : 2, STEP = U * kRotThreads;
  struct Loaded {
    Pack<TI, V> a[U], b[U];
  };
  auto load = [&](int x0, Loaded& l) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int x = x0 + k * kRotThreads;
      if (x >= items) continue;
      const Unit q = unit(x);
      const long long row = row0 + q.r;
      const TI* src;
      if (!APPEND || q.h < p.nh)
        src = static_cast<const TI*>(p.x) + row * p.x_row + (long long)q.h * p.x_head;
      else if (q.h < p.nh + p.nk)
        src = static_cast<const TI*>(p.k) + row * p.k_row + (long long)(q.h - p.nh) * p.hd;
      else
        src = static_cast<const TI*>(p.v) + row * p.v_row + (long long)(q.h - p.nh - p.nk) * p.hd;
      l.a[k] = load_pack<V>(src + q.f0);
      if (!INTER && q.turn) l.b[k] = load_pack<V>(src + half + q.f0);
    }
  };
  pdl_wait();
  pdl_trigger();
  Loaded cur;
  load(tid, cur);

  for (int i = tid; i < nr * half; i += kRotThreads) {
    const int r = i / half, e = i % half;
    const uint64_t frac = (uint64_t)(int64_t)p.pos[row0 + r] * p.turns[e];   // modulo 2^64: the fraction of a turn
    float sn, cs;
    sincospif((float)(int32_t)(uint32_t)(frac >> 32) * 0x1p-31f, &sn, &cs);
    s_cos[i] = cs * p.mag;
    s_sin[i] = p.inverse ? -sn * p.mag : sn * p.mag;
  }
  if constexpr (APPEND) {
    // the rows' sequences and slots, a warp a row (the last warps: the first ones hold angles)
    const int r = kRotThreads / 32 - 1 - (tid >> 5);
    if (r < nr) {
      const int row = row0 + r, b = find_seq(p.map.row_start, p.map.B, row);
      const int r0 = p.map.row_start[b], r1 = p.map.row_start[b + 1], len = p.map.lens[b];
      // a row behind the last sequence or before the first belongs to none
      const bool none = (row >= r1 && b == p.map.B - 1 && r1 >= r0 && r1 >= 0) || (row < r0 && b == 0);
      const bool bad = !none && (r0 < 0 || r1 > p.T || row < r0 || row >= r1);
      uint32_t bits = bad ? SWA_DERR_SEGMENT : 0u;
      const long long slot = (long long)len - r1 + row;
      long long at = -1;
      if (!none && !bad) {
        if (len < 0 || len > p.map.cap || slot < 0) {
          bits |= SWA_DERR_META;
        } else {
          const int page = p.map.table[(size_t)b * p.map.max_pages + (size_t)(slot >> p.map.page_shift)];
          if (page_ok(p.map, page))
            at = (long long)page * p.nk * p.hd_page + (slot & ((1 << p.map.page_shift) - 1)) * p.hd;
          else
            bits |= SWA_DERR_PAGE;
        }
      }
      if ((tid & 31) == 0) {
        s_live[r] = !none && !bad;
        s_slot[r] = at;
        s_aux[r] = (long long)b * p.nk * p.map.cap + slot;
        if (bits && blockIdx.y == 0) set_err(p.err, bits);
      }
    }
  }
  __syncthreads();

  for (int x0 = tid; x0 < items; x0 += STEP) {
    Loaded next;
    load(x0 + STEP, next);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int x = x0 + k * kRotThreads;
      if (x >= items) continue;
      const Unit q = unit(x);
      const long long row = row0 + q.r;
      TO* dst;
      bool rotate = q.turn;
      if constexpr (APPEND) {
        if (!s_live[q.r]) continue;
        if (q.h < p.nh) {
          dst = static_cast<TO*>(p.out) + row * p.out_row + (long long)q.h * p.hd;
        } else {
          const bool is_k = q.h < p.nh + p.nk;
          const int g = q.h - p.nh - (is_k ? 0 : p.nk);
          if (s_slot[q.r] < 0) continue;
          dst = static_cast<TO*>(is_k ? p.cache_k : p.cache_v) + s_slot[q.r] + (long long)g * p.hd_page;
          rotate = q.turn && is_k;
          if (is_k && q.u == 0) {
            if (p.slot_pos) p.slot_pos[s_aux[q.r] + (long long)g * p.map.cap] = p.pos[row];
            if (p.weight) p.weight[s_aux[q.r] + (long long)g * p.map.cap] = 0.f;
          }
        }
      } else {
        dst = static_cast<TO*>(p.out) + row * p.out_row + (long long)q.h * p.out_head;
      }
      const int e0 = q.u * NP;                          // first pair
      const float* cs = s_cos + q.r * half + e0;
      const float* sn = s_sin + q.r * half + e0;
      float a[V];
      unpack(cur.a[k], a);
      if constexpr (INTER) {
        if (rotate) {
          const int np = min(NP, half - e0);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            if (i < np) {
              const float c = cs[i], s = sn[i], u0 = a[2 * i], v0 = a[2 * i + 1];
              a[2 * i] = u0 * c - v0 * s;
              a[2 * i + 1] = v0 * c + u0 * s;
            }
          }
        }
      } else if (q.turn) {
        float b[V];
        unpack(cur.b[k], b);
        if (rotate) {
          float c[V], s[V];
          unpack(load_pack<V>(cs), c);
          unpack(load_pack<V>(sn), s);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float u0 = a[i], v0 = b[i];
            a[i] = u0 * c[i] - v0 * s[i];
            b[i] = v0 * c[i] + u0 * s[i];
          }
        }
        store_pack(dst + half + q.f0, b);
      }
      store_pack(dst + q.f0, a);
    }
    cur = next;
  }
}

// Units of a row (pairs of the rotated part, then the copied part), and the block's rows
// and heads: all heads of kRotRows rows once that gives every SM four blocks, else one
// row and as many heads as give each thread a unit.
static bool rotary_units(RotaryParams& p, bool inter, int* v) {
  const int half = p.rot / 2, rest = p.hd - p.rot;
  // the halves start at multiples of v, and then the rest does (hd is a multiple of 8)
  *v = inter || half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
  p.units = inter ? p.hd / 8 : half / *v + rest / *v;
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  p.R = p.T >= 4 * sms * kRotRows ? kRotRows : 1;
  p.Hg = p.R > 1 || p.T >= 4 * sms ? p.H : (kRotThreads + p.units - 1) / p.units;
  if (p.Hg > p.H) p.Hg = p.H;
  const long long most = (1 << 18) / p.units < 2048 ? (1 << 18) / p.units : 2048;   // items of a block: 2^20 at most
  if (p.Hg > most) p.Hg = (int)most;
  p.units_inv = ((1ull << 32) + p.units - 1) / p.units;
  p.heads_inv = ((1ull << 32) + p.Hg - 1) / p.Hg;
  return (p.H + p.Hg - 1) / p.Hg <= 65535;
}

template <typename TI, typename TO, bool APPEND>
static int launch_rotary(const RotaryParams& p, bool inter, int v, cudaStream_t s) {
  const dim3 grid((unsigned)((p.T + p.R - 1) / p.R), (unsigned)((p.H + p.Hg - 1) / p.Hg)), block(kRotThreads);
  cudaError_t e;
  if (inter)
    e = launch_pdl(rotary_kernel<TI, TO, true, 8, APPEND>, grid, block, 0, s, p);
  else if (v == 8)
    e = launch_pdl(rotary_kernel<TI, TO, false, 8, APPEND>, grid, block, 0, s, p);
  else if (v == 4)
    e = launch_pdl(rotary_kernel<TI, TO, false, 4, APPEND>, grid, block, 0, s, p);
  else if (v == 2)
    e = launch_pdl(rotary_kernel<TI, TO, false, 2, APPEND>, grid, block, 0, s, p);
  else
    e = launch_pdl(rotary_kernel<TI, TO, false, 1, APPEND>, grid, block, 0, s, p);
  return finish_launch(e);
}

static int type_bytes(int t) { return t == SWA_F32 ? 4 : 2; }

// Frequencies of a schedule in f64 (declared and explained in swa.h).
static int rotary_freqs(const swa_rotary_schedule* s, int e, double* f) {
  double theta = s->theta;
  if (s->kind == SWA_ROTARY_BASE) theta *= std::pow(s->factor, (double)s->rot / (s->rot - 2));
  double v = std::pow(theta, -2.0 * e / s->rot);
  if (s->kind == SWA_ROTARY_LINEAR) v /= s->factor;
  if (s->kind == SWA_ROTARY_PARTS) {
    const double r = s->orig_len * v / 6.283185307179586476925;
    double keep = (r - s->low) / (s->high - s->low);
    keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
    v = keep * v + (1 - keep) * v / s->factor;
  }
  *f = v;
  return v >= 0 && v < 0x1p64;             // false for NaN too
}

// floor(frac(f / 2 pi) * 2^64) of the f64 f >= 0, f < 2^64, in integers: f = m 2^e with m < 2^53,
// and m floor(2^256 / 2 pi) 2^(e - 256) is below f / 2 pi by less than 2^-192. (A quotient in f64
// is off by 2^-53 of itself, which 2^31 positions make 2^-25 turns.)
static uint64_t turn_fraction(double f) {
  static const uint64_t inv[4] = {0x7f9458eaf7aef158u, 0x36d8a5664f10e410u, 0x7f09d5f47d4d3770u, 0x28be60db9391054au};
  int e;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(f, &e), 53);
  uint64_t prod[5], carry = 0;             // m * inv, the lowest word first
  for (int i = 0; i < 4; ++i) {
    const unsigned __int128 t = (unsigned __int128)m * inv[i] + carry;
    prod[i] = (uint64_t)t;
    carry = (uint64_t)(t >> 64);
  }
  prod[4] = carry;
  const int bit = 256 - 64 - (e - 53);     // its bit of weight 2^-64: 181 at least
  if (bit >= 320) return 0;
  const int w = bit >> 6, r = bit & 63;
  return prod[w] >> r | (r && w < 4 ? prod[w + 1] << (64 - r) : 0);
}

}  // namespace swa

using namespace swa;

extern "C" {

int swa_rotary_turns(const swa_rotary_schedule* s, double* freqs, uint64_t* turns) {
  if (!s) return SWA_E_NULL;
  if (s->kind < SWA_ROTARY_PLAIN || s->kind > SWA_ROTARY_PARTS) return SWA_E_SHAPE;
  if (s->rot < 2 || s->rot > 1024 || (s->rot & 1) || !(s->theta > 0.0) || !std::isfinite(s->theta))
    return SWA_E_SHAPE;
  if (s->kind != SWA_ROTARY_PLAIN && !(s->factor >= 1.0 && std::isfinite(s->factor))) return SWA_E_SHAPE;
  if (s->kind == SWA_ROTARY_BASE && s->rot <= 2) return SWA_E_SHAPE;
  if (s->kind == SWA_ROTARY_PARTS &&
      !(s->orig_len > 0.0 && std::isfinite(s->orig_len) && s->high > s->low && std::isfinite(s->high) &&
        std::isfinite(s->low)))
    return SWA_E_SHAPE;
  for (int e = 0; e < s->rot / 2; ++e) {   // nothing is written unless every frequency is one
    double f;
    if (!rotary_freqs(s, e, &f)) return SWA_E_SHAPE;
  }
  for (int e = 0; e < s->rot / 2; ++e) {
    double f;
    rotary_freqs(s, e, &f);
    if (freqs) freqs[e] = f;
    if (turns) turns[e] = turn_fraction(f);
  }
  return SWA_OK;
}

// Extent in elements of T rows of H heads, or -1 when rows and heads overlap.
static long long extent(long long T, long long H, long long hd, long long row, long long head) {
  const long long heads = rows_span(H, hd, head), rows = rows_span(T, hd, row);
  if (heads < 0 || rows < 0 || !(row >= heads || head >= rows)) return -1;
  return (T - 1) * row + heads;
}

int swa_rotary(const swa_rotary_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  if (a->T < 0 || a->H < 1 || a->hd < 8 || a->hd > 1024 || a->hd % 8 || a->rot < 2 || (a->rot & 1) || a->rot > a->hd)
    return SWA_E_SHAPE;
  if (a->dtype != SWA_F32 && a->dtype != SWA_BF16 && a->dtype != SWA_F16) return SWA_E_SHAPE;
  if (!std::isfinite(a->mag)) return SWA_E_SHAPE;
  if (a->H >= (1 << 21) || (long long)a->T * a->H >= (1LL << 40) / a->hd) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->x || !a->out || !a->pos || !a->turns) return SWA_E_NULL;
  const long long nx = extent(a->T, a->H, a->hd, a->x_row, a->x_head);
  const long long no = extent(a->T, a->H, a->hd, a->out_row, a->out_head);
  if (nx < 0 || no < 0) return SWA_E_SHAPE;
  const int w = type_bytes(a->dtype);
  if (!aligned16p(a->x) || !aligned16p(a->out) || ((a->x_row | a->x_head | a->out_row | a->out_head) * w & 15) ||
      (reinterpret_cast<uintptr_t>(a->pos) & 3u) || (reinterpret_cast<uintptr_t>(a->turns) & 7u))
    return SWA_E_ALIGN;
  const bool same = a->x == a->out && a->x_row == a->out_row && a->x_head == a->out_head;
  if (!same && bytes_overlap(a->x, (size_t)nx * w, a->out, (size_t)no * w)) return SWA_E_SHAPE;
  RotaryParams p{};
  p.T = a->T; p.H = a->H; p.hd = a->hd; p.rot = a->rot; p.inverse = a->inverse != 0; p.mag = a->mag;
  p.x = a->x; p.x_row = a->x_row; p.x_head = a->x_head;
  p.out = a->out; p.out_row = a->out_row; p.out_head = a->out_head;
  p.pos = a->pos; p.turns = a->turns;
  const bool inter = a->interleaved != 0;
  int v;
  if (!rotary_units(p, inter, &v)) return SWA_E_SHAPE;
  switch (a->dtype) {
    case SWA_F32: return launch_rotary<float, float, false>(p, inter, v, stream);
    case SWA_BF16: return launch_rotary<__nv_bfloat16, __nv_bfloat16, false>(p, inter, v, stream);
    default: return launch_rotary<__half, __half, false>(p, inter, v, stream);
  }
}

int swa_paged_append(const swa_paged_append_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged_cache& c = a->cache;
  const int rc = paged_cache_status(&c, true);
  if (rc != SWA_OK) return rc;
  const int nh = a->q || a->q_out ? a->nh : 0;
  if (a->T < 0 || a->nh < 0 || a->nh >= (1 << 20) || a->rot < 0 || (a->rot & 1) || a->rot > c.hd) return SWA_E_SHAPE;
  if (a->src != SWA_F32 && a->src != c.dtype) return SWA_E_SHAPE;
  if (!std::isfinite(a->mag)) return SWA_E_SHAPE;
  const long long H = (long long)nh + 2LL * c.nk;
  if (H >= (1 << 21) || (long long)a->T * H >= (1LL << 40) / c.hd) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->k || !a->v || (a->q != nullptr) != (a->q_out != nullptr)) return SWA_E_NULL;
  if (a->rot > 0 && (!a->pos || !a->turns)) return SWA_E_NULL;
  if (a->slot_pos && !a->pos) return SWA_E_NULL;
  if (a->q && a->nh < 1) return SWA_E_SHAPE;
  const int w = type_bytes(a->src);
  const long long kd = (long long)c.nk * c.hd, qd = (long long)nh * c.hd;
  const long long kn = rows_span(a->T, kd, a->k_row), vn = rows_span(a->T, kd, a->v_row);
  const long long qn = a->q ? rows_span(a->T, qd, a->q_row) : 0;
  if (kn < 0 || vn < 0 || qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->k) || !aligned16p(a->v) || !aligned16p(a->q) || !aligned16p(a->q_out) ||
      ((a->k_row | a->v_row | (a->q ? a->q_row : 0)) * w & 15) || (reinterpret_cast<uintptr_t>(a->pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->turns) & 7u) || (reinterpret_cast<uintptr_t>(a->slot_pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->weight) & 3u))
    return SWA_E_ALIGN;
  if (a->q) {
    const bool same = a->q == a->q_out && a->src == c.dtype && a->q_row == qd;
    const size_t on = (size_t)a->T * qd * 2;
    if ((!same && bytes_overlap(a->q, (size_t)qn * w, a->q_out, on)) ||
        bytes_overlap(a->k, (size_t)kn * w, a->q_out, on) || bytes_overlap(a->v, (size_t)vn * w, a->q_out, on))
      return SWA_E_SHAPE;
  }
  const size_t pool = (size_t)c.num_pages * c.nk * c.page * c.hd * 2;
  if (bytes_overlap(c.k, pool, c.v, pool)) return SWA_E_SHAPE;
  RotaryParams p{};
  p.T = a->T; p.H = (int)H; p.hd = c.hd; p.rot = a->rot; p.mag = a->mag;
  p.x = a->q; p.x_row = a->q_row; p.x_head = c.hd;
  p.out = a->q_out; p.out_row = qd;
  p.pos = a->pos; p.turns = a->turns;
  p.nh = nh; p.nk = c.nk; p.hd_page = c.page * c.hd;
  p.k = a->k; p.v = a->v; p.k_row = a->k_row; p.v_row = a->v_row;
  p.cache_k = c.k; p.cache_v = c.v;
  p.map = paged_map(&c);
  p.slot_pos = a->slot_pos; p.weight = a->weight; p.err = a->err;
  const bool inter = a->interleaved != 0;
  int v;
  if (!rotary_units(p, inter, &v)) return SWA_E_SHAPE;
  if (a->src == SWA_F32)
    return c.dtype == SWA_BF16 ? launch_rotary<float, __nv_bfloat16, true>(p, inter, v, stream)
                               : launch_rotary<float, __half, true>(p, inter, v, stream);
  return c.dtype == SWA_BF16 ? launch_rotary<__nv_bfloat16, __nv_bfloat16, true>(p, inter, v, stream)
                             : launch_rotary<__half, __half, true>(p, inter, v, stream);
}

}  // extern "C"
