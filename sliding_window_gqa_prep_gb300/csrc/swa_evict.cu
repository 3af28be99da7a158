// The weight each cached key received (swa_paged_weigh) and the eviction of keys by it
// (swa_paged_evict).
#include <cmath>

#include "swa_mma16.cuh"
#include "swa_paged_attend.cuh"

namespace swa {

// ---------------------------------------------------------------------------
// Weigh. w_j += sum over query vectors of 2^(qmul <q, k_j> - lse log2 e): with the
// row's lse known every weight stands alone, so a CTA takes 64 keys of one KV head,
// holds them as A operands (16 keys a warp) and streams the query vectors that see
// them through shared memory as B operands; S has a key a row, and the sum over its
// columns stays in registers until the end. K is read once; bound by that while a
// sequence has few rows.
// ---------------------------------------------------------------------------
struct PagedWeighParams {
  PagedMap map;
  int T, nh, hpg, max_rows;
  float qmul;
  const void* q;
  long long q_row;
  const void* ck;
  const float* lse;
  const float* weight;
  float* out;
  uint32_t* err;
};

constexpr int kWThreads = 128;
constexpr int kWKeys = 64;     // keys of a CTA
constexpr int kWVecs = 32;     // query vectors of a tile

template <typename T, int D>
__global__ void __launch_bounds__(kWThreads) paged_weigh_kernel(const PagedWeighParams p) {
  constexpr int CH = D / 8;
  extern __shared__ __align__(128) unsigned char sm[];       // K tile, two Q tiles
  __shared__ float s_lse[2][kWVecs];
  __shared__ int s_lim[2][kWVecs];
  const uint32_t smk = smem_u32(sm), smq = smk + kWKeys * D * 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z, g = blockIdx.y, k0 = blockIdx.x * kWKeys;
  pdl_wait();
  pdl_trigger();
  uint32_t bits = 0;
  const PagedSeq s = paged_seq(p.map, b, p.T, p.max_rows, bits);
  if (bits && tid == 0 && g == 0 && blockIdx.x == 0) set_err(p.err, bits);
  if (k0 >= s.len) return;

  const int32_t* table = p.map.table + (size_t)b * p.map.max_pages;
  const T* const kp = static_cast<const T*>(p.ck);
  const T* const qp = static_cast<const T*>(p.q);
#pragma unroll
  for (int i = 0; i < kWKeys * CH / kWThreads; ++i) {
    const int x = tid + i * kWThreads, r = x / CH, c = x % CH, key = k0 + r;
    int id = -1;
    if (key < s.len) {
      id = table[key >> p.map.page_shift];
      if (!page_ok(p.map, id)) {
        set_err(p.err, SWA_DERR_PAGE);
        id = -1;
      }
    }
    const size_t off =
        id >= 0 ? ((((size_t)id * p.map.nk + g) << p.map.page_shift) + (key & ((1 << p.map.page_shift) - 1))) * D + c * 8 : 0;
    cp16_or_zero(smk + tile_off<D>(r, c), kp + off, id >= 0);
  }
  // rows that see some key of the block: limit > k0
  const int i_first = max(0, k0 - (s.len - s.t));
  const int v0 = i_first * p.hpg, nv = s.t * p.hpg;
  auto load_q = [&](int buf, int v) {
    for (int x = tid; x < kWVecs * CH; x += kWThreads) {
      const int r = x / CH, c = x % CH, vec = v + r;
      const bool ok = vec < nv;
      const int i = ok ? vec / p.hpg : 0, h = ok ? vec % p.hpg : 0;
      cp16_or_zero(smq + (uint32_t)(buf * kWVecs * D * 2) + tile_off<D>(r, c),
                   qp + (ok ? (size_t)(s.r0 + i) * p.q_row + (size_t)(g * p.hpg + h) * D + c * 8 : 0), ok);
    }
    if (tid < kWVecs) {
      const int vec = v + tid;
      float lse = 0.f;
      int lim = 0;
      if (vec < nv) {
        const int i = vec / p.hpg;
        lse = p.lse[(size_t)(s.r0 + i) * p.nh + g * p.hpg + vec % p.hpg] * 1.4426950408889634f;
        lim = min(s.len, s.len - s.t + i + 1);
      }
      s_lse[buf][tid] = lse;
      s_lim[buf][tid] = lim;
    }
  };
  if (v0 < nv) load_q(0, v0);
  cp_commit();
  float w[2] = {0.f, 0.f};
  uint32_t kf[D / 16][4];
  int buf = 0;
  for (int v = v0; v < nv; v += kWVecs, buf ^= 1) {
    cp_wait<0>();
    __syncthreads();
    if (v == v0) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ldsm4(kf[k], smk + tile_off<D>(warp * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), k * 2 + (lane >> 4)));
    }
    if (v + kWVecs < nv) load_q(buf ^ 1, v + kWVecs);
    cp_commit();
    const uint32_t qb = smq + (uint32_t)(buf * kWVecs * D * 2);
    float sc[kWVecs / 8][4];
#pragma unroll
    for (int n = 0; n < kWVecs / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[n][j] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int n = 0; n < kWVecs / 16; ++n) {
        uint32_t f[4];
        ldsm4(f, qb + tile_off<D>(n * 16 + ((lane >> 4) << 3) + (lane & 7), k * 2 + ((lane >> 3) & 1)));
        mma16816<T>(sc[2 * n], kf[k], f[0], f[1]);
        mma16816<T>(sc[2 * n + 1], kf[k], f[2], f[3]);
      }
    const int key = k0 + warp * 16 + (lane >> 2);
#pragma unroll
    for (int n = 0; n < kWVecs / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n * 8 + (lane & 3) * 2 + (j & 1);
        const float x = ex2(fmaf(sc[n][j], p.qmul, -s_lse[buf][c]));
        if (key + (j >> 1) * 8 < s_lim[buf][c]) w[j >> 1] += x;
      }
  }
  cp_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    w[r] += __shfl_xor_sync(0xffffffffu, w[r], 1);
    w[r] += __shfl_xor_sync(0xffffffffu, w[r], 2);
    const int key = k0 + warp * 16 + r * 8 + (lane >> 2);
    if ((lane & 3) == 0 && key < s.len) {
      const size_t at = ((size_t)b * p.map.nk + g) * p.map.cap + key;
      p.out[at] = (p.weight ? p.weight[at] : 0.f) + w[r];
    }
  }
}

template <typename T, int D>
static int launch_weigh(const PagedWeighParams& p, cudaStream_t s) {
  constexpr int smem = (kWKeys + 2 * kWVecs) * D * 2;
  cudaError_t e = allow_smem<paged_weigh_kernel<T, D>>(smem);
  if (e != cudaSuccess) return cuda_status(e);
  const dim3 grid((unsigned)((p.map.cap + kWKeys - 1) / kWKeys), (unsigned)p.map.nk, (unsigned)p.map.B);
  return finish_launch(launch_pdl(paged_weigh_kernel<T, D>, grid, dim3(kWThreads), smem, s, p));
}

// ---------------------------------------------------------------------------
// Evict. select: one CTA per (sequence, KV head) finds the threshold key of the n'
// first slots by a radix select over an order-preserving 32-bit key (four histogram
// passes of 8 bits), then numbers the freed and the moved slots in slot order with
// block scans, and writes the kept slots' weights and positions. move: a warp a moved
// row copies K, V, weight and position; its source lies at or behind n', its
// destination before it, so no row is both read and written.
// ---------------------------------------------------------------------------
struct PagedEvictParams {
  PagedMap map;
  int hd, keep, sinks, list_cap;
  const float* weight;
  const int32_t* slot_pos;
  const int32_t* recent_from;
  float* weight_out;
  int32_t* slot_pos_out;
  int32_t* lens_out;
  void* ck;
  void* cv;
  int* ws_count;               // [B][nk]
  int* ws_dst;                 // [B][nk][list_cap]
  int* ws_src;                 // [B][nk][list_cap]
  uint32_t* err;
};

constexpr int kEThreads = 1024;

// Descending order of slots as descending order of this key: protected slots first,
// then NaN, then the weights (-0 as 0).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sinks, int recent) {
  if (pos < sinks || pos >= recent) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;     // +inf: 0xff800000
}

// Exclusive sum of a small per-thread count over the block, and the block's total.
__device__ __forceinline__ int block_rank(bool flag, int* warp_sums, int& total) {
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) warp_sums[warp] = __popc(m);
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kEThreads / 32; ++w) {
    const int c = warp_sums[w];
    if (w < warp) before += c;
    total += c;
  }
  return before + __popc(m & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kEThreads) paged_evict_select_kernel(const PagedEvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kEThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, g = blockIdx.x, b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  int n = p.map.lens[b];
  if (n < 0 || n > p.map.cap) {
    if (tid == 0 && g == 0) set_err(p.err, SWA_DERR_META);
    n = n < 0 ? 0 : p.map.cap;
  }
  const int keep = min(n, p.keep);
  const size_t bg = (size_t)b * p.map.nk + g;
  const float* w = p.weight + bg * p.map.cap;
  const int32_t* pos = p.slot_pos + bg * p.map.cap;
  float* wo = p.weight_out + bg * p.map.cap;
  int32_t* po = p.slot_pos_out + bg * p.map.cap;
  if (tid == 0 && g == 0) p.lens_out[b] = keep;
  if (n <= p.keep) {                       // everything stays
    for (int j = tid; j < n; j += kEThreads) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    if (tid == 0) p.ws_count[bg] = 0;
    return;
  }
  const int recent = p.recent_from ? p.recent_from[b] : 0x7fffffff;
  const bool any_recent = p.recent_from != nullptr;
  auto key_of = [&](int j) {
    const int ps = pos[j];
    return evict_key(w[j], any_recent ? ps : min(ps, 0x7ffffffe), p.sinks, recent);
  };
  // the keep-th largest key, eight bits at a time
  uint32_t prefix = 0;
  int need = keep;                         // slots still to take among keys with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kEThreads) {
      const uint32_t k = key_of(j);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int c = 0, d = 255;
      for (; d > 0; --d) {
        if (c + hist[d] >= need) break;
        c += hist[d];
      }
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = need - c;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // keys above `prefix` stay, and the first `need` slots that equal it
  int* const dst = p.ws_dst + bg * p.list_cap;
  int* const src = p.ws_src + bg * p.list_cap;
  int eq_seen = 0, n_dst = 0, n_src = 0;
  for (int j0 = 0; j0 < n; j0 += kEThreads) {
    const int j = j0 + tid;
    const bool in = j < n;
    const uint32_t k = in ? key_of(j) : 0u;
    const bool eq = in && k == prefix;
    int total;
    const int rank = block_rank(eq, warp_sums, total);
    const bool kept = in && (k > prefix || (eq && eq_seen + rank < need));
    eq_seen += total;
    const bool freed = in && j < keep && !kept, moved = kept && j >= keep;
    if (kept && j < keep) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    if (j0 < keep) {
      const int r = block_rank(freed, warp_sums, total);
      if (freed) dst[n_dst + r] = j;
      n_dst += total;
    }
    if (j0 + kEThreads > keep) {
      const int r = block_rank(moved, warp_sums, total);
      if (moved) src[n_src + r] = j;
      n_src += total;
    }
  }
  if (tid == 0) p.ws_count[bg] = n_src;    // = n_dst: keep slots stay in all
}

constexpr int kMoveWarps = 8;
constexpr int kMoveRows = 4;               // rows of a warp

__global__ void __launch_bounds__(kMoveWarps * 32) paged_evict_move_kernel(const PagedEvictParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const size_t bg = (size_t)b * p.map.nk + g;
  const int count = p.ws_count[bg];
  const int32_t* table = p.map.table + (size_t)b * p.map.max_pages;
  const int ch = p.hd / 8;                 // 16-byte chunks of a row: 8, 16 or 32
  for (int r = 0; r < kMoveRows; ++r) {
    const int i = (blockIdx.x * kMoveWarps + warp) * kMoveRows + r;
    if (i >= count) return;
    const int to = p.ws_dst[bg * p.list_cap + i], of = p.ws_src[bg * p.list_cap + i];
    const int pt = table[to >> p.map.page_shift], pf = table[of >> p.map.page_shift];
    const int mask = (1 << p.map.page_shift) - 1;
    if (lane == 0) {
      p.weight_out[bg * p.map.cap + to] = p.weight[bg * p.map.cap + of];
      p.slot_pos_out[bg * p.map.cap + to] = p.slot_pos[bg * p.map.cap + of];
    }
    if (!page_ok(p.map, pt) || !page_ok(p.map, pf)) {
      if (lane == 0) set_err(p.err, SWA_DERR_PAGE);
      continue;
    }
    const size_t at = ((((size_t)pt * p.map.nk + g) << p.map.page_shift) + (to & mask)) * ch;
    const size_t from = ((((size_t)pf * p.map.nk + g) << p.map.page_shift) + (of & mask)) * ch;
    for (int c = lane; c < 2 * ch; c += 32) {
      uint4* base = static_cast<uint4*>(c < ch ? p.ck : p.cv);
      const int cc = c < ch ? c : c - ch;
      base[at + cc] = base[from + cc];
    }
  }
}

static size_t evict_list_cap(const swa_paged_evict_args* a) {
  const long long cap = (long long)a->cache.max_pages * a->cache.page;
  return (size_t)(a->keep < cap ? a->keep : cap);
}
static bool evict_sizes_ok(const swa_paged_evict_args* a) {
  const swa_paged_cache& c = a->cache;
  return c.B >= 1 && c.B <= 65535 && c.nk >= 1 && c.nk <= 65535 && c.page >= 16 && c.page <= 256 &&
         (c.page & (c.page - 1)) == 0 && c.max_pages >= 1 && c.max_pages <= (1 << 30) / c.page && a->keep >= 1 &&
         a->sinks >= 0;
}

}  // namespace swa

using namespace swa;

extern "C" {

int swa_paged_weigh(const swa_paged_weigh_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged_cache& c = a->cache;
  const int rc = paged_cache_status(&c, true);
  if (rc != SWA_OK) return rc;
  if (!a->out || (a->T > 0 && (!a->q || !a->lse))) return SWA_E_NULL;
  if (a->T < 0 || a->max_rows < 1 || a->nh < 1 || a->nh % c.nk || a->nh / c.nk > 32) return SWA_E_SHAPE;
  if ((long long)a->T * a->nh >= (1LL << 31) || (long long)a->max_rows * (a->nh / c.nk) >= (1LL << 31) - 64) return SWA_E_SHAPE;
  if (!(a->scale >= 0.f) || std::isinf(a->scale)) return SWA_E_SHAPE;
  if (a->T > 0 && (a->q_row < (long long)a->nh * c.hd || a->q_row > (1LL << 40))) return SWA_E_SHAPE;
  if (!aligned16p(a->q) || (a->T > 0 && (a->q_row & 7)) || (reinterpret_cast<uintptr_t>(a->lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->weight) & 3u) || (reinterpret_cast<uintptr_t>(a->out) & 3u))
    return SWA_E_ALIGN;
  PagedWeighParams p{};
  p.map = paged_map(&c);
  const size_t bytes = (size_t)c.B * c.nk * p.map.cap * 4;
  if (a->weight && a->weight != a->out && bytes_overlap(a->weight, bytes, a->out, bytes)) return SWA_E_SHAPE;
  p.T = a->T; p.nh = a->nh; p.hpg = a->nh / c.nk; p.max_rows = a->max_rows;
  p.qmul = a->scale * 1.4426950408889634f;
  p.q = a->q; p.q_row = a->q_row; p.ck = c.k;
  p.lse = a->lse; p.weight = a->weight; p.out = a->out; p.err = a->err;
  if (c.dtype == SWA_BF16)
    return c.hd == 64 ? launch_weigh<__nv_bfloat16, 64>(p, stream)
                      : c.hd == 128 ? launch_weigh<__nv_bfloat16, 128>(p, stream) : launch_weigh<__nv_bfloat16, 256>(p, stream);
  return c.hd == 64 ? launch_weigh<__half, 64>(p, stream)
                    : c.hd == 128 ? launch_weigh<__half, 128>(p, stream) : launch_weigh<__half, 256>(p, stream);
}

size_t swa_paged_evict_workspace_size(const swa_paged_evict_args* a) {
  if (!a || !evict_sizes_ok(a)) return 0;
  const size_t items = (size_t)a->cache.B * a->cache.nk;
  return up256s(items * 4) + 2 * up256s(items * evict_list_cap(a) * 4);
}

int swa_paged_evict(const swa_paged_evict_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged_cache& c = a->cache;
  const int rc = paged_cache_status(&c, false);
  if (rc != SWA_OK) return rc;
  if (!a->weight || !a->slot_pos || !a->weight_out || !a->slot_pos_out || !a->lens_out) return SWA_E_NULL;
  if (!evict_sizes_ok(a)) return SWA_E_SHAPE;
  const void* words[] = {a->weight, a->slot_pos, a->recent_from, a->weight_out, a->slot_pos_out, a->lens_out};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return SWA_E_ALIGN;
  PagedEvictParams p{};
  p.map = paged_map(&c);
  const size_t items = (size_t)c.B * c.nk, bytes = items * p.map.cap * 4, lens = (size_t)c.B * 4;
  const struct { const void* p; size_t n; } in[] = {{a->weight, bytes}, {a->slot_pos, bytes}, {c.lens, lens},
                                                    {a->recent_from, a->recent_from ? lens : 0}},
                                            out[] = {{a->weight_out, bytes}, {a->slot_pos_out, bytes}, {a->lens_out, lens}};
  for (const auto& o : out) {
    for (const auto& i : in)
      if (bytes_overlap(o.p, o.n, i.p, i.n)) return SWA_E_SHAPE;
    for (const auto& o2 : out)
      if (&o2 != &o && bytes_overlap(o.p, o.n, o2.p, o2.n)) return SWA_E_SHAPE;
  }
  const size_t need = swa_paged_evict_workspace_size(a);
  if (!a->workspace || a->workspace_bytes < need) return SWA_E_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return SWA_E_ALIGN;
  p.hd = c.hd; p.keep = a->keep; p.sinks = a->sinks; p.list_cap = (int)evict_list_cap(a);
  p.weight = a->weight; p.slot_pos = a->slot_pos; p.recent_from = a->recent_from;
  p.weight_out = a->weight_out; p.slot_pos_out = a->slot_pos_out; p.lens_out = a->lens_out;
  p.ck = c.k; p.cv = c.v;
  char* ws = static_cast<char*>(a->workspace);
  p.ws_count = reinterpret_cast<int*>(ws);
  p.ws_dst = reinterpret_cast<int*>(ws + up256s(items * 4));
  p.ws_src = reinterpret_cast<int*>(ws + up256s(items * 4) + up256s(items * evict_list_cap(a) * 4));
  p.err = a->err;
  const int rc2 = finish_launch(launch_pdl(paged_evict_select_kernel, dim3(c.nk, c.B), dim3(kEThreads), 0, stream, p));
  if (rc2 != SWA_OK) return rc2;
  const unsigned per = kMoveWarps * kMoveRows;
  return finish_launch(launch_pdl(paged_evict_move_kernel, dim3(((unsigned)p.list_cap + per - 1) / per, c.nk, c.B),
                                  dim3(kMoveWarps * 32), 0, stream, p));
}

}  // extern "C"
