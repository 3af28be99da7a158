// Eviction of cached keys by their accumulated weight (swa_paged_evict).
#include "swa_paged.cuh"

namespace swa {

// ---------------------------------------------------------------------------
// select: one CTA per (sequence, KV head) finds the threshold key of the n'
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
