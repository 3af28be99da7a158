// Eviction of cached keys by their accumulated weight (swa_paged_evict).
//
// One cluster per (sequence, KV head) does the whole eviction in one launch, each CTA a
// contiguous share of the slots:
//   1. keys of its slots (an order-preserving 32-bit key), 8 slots a thread in registers
//      (longer shares in shared memory), all loads under way together;
//   2. the n'-th largest key by histogram passes over its digits; the CTAs' histograms are
//      summed through distributed shared memory;
//   3. each warp counts its run of slots that stay before and behind n'; sums over the warps
//      and CTAs number the freed and the moved slots, and a walk in slot order writes the
//      kept slots' weights and positions and the two lists (slots and rows);
//   4. the rows that move are copied. A source lies at or
//      behind n', its destination before it: no row is both read and written.
// Steps 1 to 3 are chains of barriers and short passes, so the CTAs' shares stay small
// (kSlotsPerCta) while the cluster may grow (8 CTAs at most) and the passes are kept short in
// instructions; copies are bound by memory.
// Measured: 32 sequences, 8 heads, 64 of 2112 slots: 12.4 us (keys 2.6, passes 2.2, counts and
// walk 2.8, copies 2.5); four of 16384 to 32768 slots down to 4096: 35.4 us, of them copies
// 17.5 at 6.6 TB/s, passes 5.7, counts and walk 5, keys 3. (Keys of a slot at a time, kept in
// shared memory, and two walks: 17 and 46.7 us; all passes always: 13.5 and 36.7.)
#include <cooperative_groups.h>

#include "swa_paged.cuh"

namespace swa {
namespace cg = cooperative_groups;

struct PagedEvictParams {
  PagedMap map;
  int hd, keep, sinks, list_cap;
  int key_slots;               // keys of a CTA that fit in its shared memory
  const float* weight;
  const int32_t* slot_pos;
  const int32_t* recent_from;
  float* weight_out;
  int32_t* slot_pos_out;
  int32_t* lens_out;
  void* ck;
  void* cv;
  int2* ws_dst;                // [B][nk][list_cap]: freed slots and their rows in the pool
  int4* ws_src;                // [B][nk][list_cap]: moved ones: row, weight, position
  uint32_t* err;
};

constexpr int kEThreads = 512, kEWarps = kEThreads / 32;
constexpr int kEN = 8;                      // slots of a thread at a time: 32 kEN in a row a warp
constexpr int kSlotsPerCta = kEThreads * kEN;   // 4096: a cluster of (capacity / this), 1 to 8, CTAs
constexpr int kMaxKeySlots = 40960;         // keys of a CTA in shared memory; longer shares are read again
constexpr int kMaxCluster = 8;

// Descending order of slots as descending order of this key: protected slots first,
// then NaN, then the weights (-0 as 0).
__device__ __forceinline__ uint32_t evict_key(float w, bool safe) {
  if (safe) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;     // +inf: 0xff800000
}

// CL: a cluster of CTAs a (sequence, KV head), else one CTA. REG: a CTA has kSlotsPerCta
// slots at most, whose keys stay in its threads' registers.
template <bool CL, bool REG>
__global__ void __launch_bounds__(kEThreads, 2) paged_evict_kernel(const PagedEvictParams p) {
  extern __shared__ uint32_t s_keys[];      // not REG
  __shared__ __align__(16) int hist[CL ? 4 : 3][CL ? 256 : 2048];
  __shared__ int s_sums[kEWarps];
  __shared__ int4 s_cnt[kEWarps];
  __shared__ int2 s_tot;                    // this CTA's freed and moved slots
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  __shared__ bool s_all;                    // every key of the bin stays
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CS = CL ? (int)cluster.num_blocks() : 1, rank = CL ? (int)cluster.block_rank() : 0;
  constexpr int MC = CL ? kMaxCluster : 1;
  auto sync_all = [&]() {
    if constexpr (CL) cluster.sync();
    else __syncthreads();
  };
  // shared memory of CTA r of the cluster
  auto peer = [&](auto* x, int r) {
    if constexpr (CL) return cluster.map_shared_rank(x, r);
    else return x;
  };
  const int item = blockIdx.x / CS, b = item / p.map.nk, g = item % p.map.nk;
  pdl_wait();
  pdl_trigger();
  int n = p.map.lens[b];
  const bool any_recent = p.recent_from != nullptr;
  const int recent = any_recent ? p.recent_from[b] : 0;
  if (n < 0 || n > p.map.cap) {
    if (tid == 0 && g == 0 && rank == 0) set_err(p.err, SWA_DERR_META);
    n = n < 0 ? 0 : p.map.cap;
  }
  const int keep = min(n, p.keep);
  const size_t base = (size_t)item * p.map.cap;
  const float* w = p.weight + base;
  const int32_t* pos = p.slot_pos + base;
  float* wo = p.weight_out + base;
  int32_t* po = p.slot_pos_out + base;
  if (tid == 0 && g == 0 && rank == 0) p.lens_out[b] = keep;
  // this CTA's slots [lo, hi), a multiple of 32 a CTA
  const int share = ((n + CS - 1) / CS + 31) & ~31;
  const int lo = min(n, rank * share), hi = min(n, lo + share);
  if (n <= p.keep) {                        // everything stays (the same for the whole cluster)
    for (int j = lo + tid; j < hi; j += kEThreads) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    return;
  }
  // warp w takes slots [wlo, whi) of the CTA's
  const int run = ((hi - lo + kEWarps - 1) / kEWarps + 31) & ~31;
  const int wlo = min(hi, lo + warp * run), whi = min(hi, wlo + run);
  // key of slot j; 0, which is no slot's, behind the warp's last one
  auto make_key = [&](int j, float x, int ps) {
    return j < whi ? evict_key(x, ps < p.sinks || (any_recent && ps >= recent)) : 0u;
  };
  uint32_t key[kEN];
  float wv[kEN];
  int pv[kEN], pg[kEN];
  auto load_slots = [&](int base) {         // all under way together
#pragma unroll
    for (int u = 0; u < kEN; ++u) {
      wv[u] = 0.f;
      pv[u] = 0;
      if (base + u * 32 + lane < whi) {
        wv[u] = (w + base + lane)[u * 32];
        pv[u] = (pos + base + lane)[u * 32];
      }
    }
  };
  const int32_t* table = p.map.table + (size_t)b * p.map.max_pages;
  auto load_pages = [&](int base) {
#pragma unroll
    for (int u = 0; u < kEN; ++u) {
      pg[u] = -1;
      if (base + u * 32 + lane < whi) pg[u] = table[(base + u * 32 + lane) >> p.map.page_shift];
    }
  };
  const bool cached = !REG && share <= p.key_slots;
  auto load_keys = [&](int base) {
    if (!cached) load_slots(base);
#pragma unroll
    for (int u = 0; u < kEN; ++u) {
      const int j = base + u * 32 + lane;
      key[u] = !cached ? make_key(j, wv[u], pv[u]) : j < whi ? s_keys[j - lo] : 0u;
    }
  };
  // f(slot, key) of the warp's slots in order, 32 at a time
  auto each = [&](auto f) {
    for (int base = wlo; base < whi; base += 32 * kEN) {
      if constexpr (!REG) load_keys(base);
#pragma unroll
      for (int u = 0; u < kEN; ++u)
        if (base + u * 32 < whi) f(base + u * 32 + lane, key[u]);
      if constexpr (REG) break;
    }
  };
  // Digits of the key: 11, 11 and 10 bits in a CTA alone (evict of 64 of 2112 slots: 18.5
  // instead of 20.8 us); four of 8 bits in a cluster, which reads every CTA's bins (30 and 21
  // thousand clk for 8 CTAs)
  const int n_pass = CL ? 4 : 3;
  for (int i = tid; i < (int)(sizeof(hist) / 4); i += kEThreads) (&hist[0][0])[i] = 0;
  if constexpr (REG) {
    load_slots(wlo);
    // the pages of these slots are looked up at the end: called into the cache now
    if (lane < kEN) asm volatile("prefetch.global.L1 [%0];" :: "l"(table + (min(wlo + lane * 32, n - 1) >> p.map.page_shift)));
#pragma unroll
    for (int u = 0; u < kEN; ++u) key[u] = make_key(wlo + u * 32 + lane, wv[u], pv[u]);
  } else if (cached) {
    for (int base = wlo; base < whi; base += 32 * kEN) {
      load_slots(base);
#pragma unroll
      for (int u = 0; u < kEN; ++u) {
        const int j = base + u * 32 + lane;
        if (j < whi) s_keys[j - lo] = make_key(j, wv[u], pv[u]);
      }
    }
  }
  __syncthreads();

  // the keep-th largest key, a digit at a time
  uint32_t prefix = 0;
  int need = keep;                          // slots still to take among keys with this prefix
#pragma unroll 1
  for (int pass = 0; pass < n_pass; ++pass) {
    const int bits = CL ? 8 : pass < 2 ? 11 : 10, shift = CL ? 24 - 8 * pass : pass == 0 ? 21 : pass == 1 ? 10 : 0;
    each([&](int, uint32_t k) {
      if (pass == 0 ? k != 0 : k >> (shift + bits) == prefix) atomicAdd(&hist[pass][(k >> shift) & ((1u << bits) - 1)], 1);
    });
    sync_all();
    // thread t holds the bins 4t .. 4t + 3 counted from the top, summed over the cluster
    const int threads = 1 << (bits - 2), top = 4 * (threads - 1 - tid);
    if (tid < threads) {
      int c[4] = {0, 0, 0, 0};
      int4 v[MC];
#pragma unroll
      for (int i = 0; i < MC; ++i) {   // all under way together; each CTA starts at its own
        v[i] = make_int4(0, 0, 0, 0);
        if (i < CS)
          v[i] = *reinterpret_cast<const int4*>(peer(&hist[pass][top], (rank + i) & (CS - 1)));
      }
#pragma unroll
      for (int i = 0; i < MC; ++i) {
        c[0] += v[i].w;
        c[1] += v[i].z;
        c[2] += v[i].y;
        c[3] += v[i].x;
      }
      const int sum = c[0] + c[1] + c[2] + c[3];
      int before = sum;                     // of the warp's threads up to this one, then of all before it
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
      }
      if (lane == 31) s_sums[warp] = before;
      named_barrier(1, threads);
      before += __reduce_add_sync(0xffffffffu, lane < warp ? s_sums[lane] : 0) - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < need && need <= before + c[i]) {
          s_digit = (uint32_t)(top + 3 - i);
          s_need = need - before;
          s_all = need == before + c[i];
        }
        before += c[i];
      }
    }
    __syncthreads();
    prefix = prefix << bits | s_digit;
    need = s_need;
    // all keys with this prefix stay: those above the greatest key below it (of weights
    // without ties: the last pass falls away 9 times in 10)
    if (s_all && prefix != 0 && shift > 0) {
      prefix = (prefix << shift) - 1;
      need = 0;
      break;
    }
  }
  // keys above `prefix` stay, and of those that equal it the first `need` in slot order;
  // the CTAs before this one hold eq_before of them
  const uint32_t digit = prefix & (CL ? 255u : 1023u);
  int eq_before = 0;
#pragma unroll
  for (int r = 0; r < MC; ++r)
    if (r < rank) eq_before += *peer(&hist[n_pass - 1][digit], r);

  // counts of the warp's slots: equal to prefix below and from `keep` on, above it the same
  int4 cnt = make_int4(0, 0, 0, 0);
  each([&](int j, uint32_t k) {
    const bool e = k == prefix, a = k > prefix, low = j < keep;
    cnt.x += e && low;
    cnt.y += e && !low;
    cnt.z += a && low;
    cnt.w += a && !low;
  });
  cnt.x = __reduce_add_sync(0xffffffffu, cnt.x);
  cnt.y = __reduce_add_sync(0xffffffffu, cnt.y);
  cnt.z = __reduce_add_sync(0xffffffffu, cnt.z);
  cnt.w = __reduce_add_sync(0xffffffffu, cnt.w);
  if (lane == 0) s_cnt[warp] = cnt;
  __syncthreads();
  // Each warp finds, lane i for warp i, how many slots are freed and moved: of its equal
  // slots the first `take` stay, those below `keep` before the others.
  int eq, n_freed, n_moved;                 // equal, freed and moved slots before this warp's
  bool any_eq;                              // some of this warp's slots are equal
  {
    const int4 c = lane < kEWarps ? s_cnt[lane] : make_int4(0, 0, 0, 0);
    const int i0 = min(hi, lo + lane * run), i1 = min(hi, i0 + run);
    int incl = c.x + c.y;
#pragma unroll
    for (int o = 1; o < kEWarps; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int before = eq_before + incl - c.x - c.y;
    const int take = max(0, min(need - before, c.x + c.y)), take_low = min(take, c.x);
    const int freed = lane < kEWarps ? max(0, min(i1, keep) - i0) - c.z - take_low : 0, moved = c.w + take - take_low;
    int f = freed, m = moved;
#pragma unroll
    for (int o = 1; o < kEWarps; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, f, o), y = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) {
        f += x;
        m += y;
      }
    }
    if (tid == kEWarps - 1) s_tot = make_int2(f, m);
    eq = __shfl_sync(0xffffffffu, before, warp);
    any_eq = __shfl_sync(0xffffffffu, c.x + c.y, warp) != 0;
    n_freed = __shfl_sync(0xffffffffu, f - freed, warp);
    n_moved = __shfl_sync(0xffffffffu, m - moved, warp);
  }
  sync_all();
  int count = 0;                            // rows that move, in the whole cluster
  int2 tot[MC];
#pragma unroll
  for (int r = 0; r < MC; ++r) tot[r] = r < CS ? *peer(&s_tot, r) : make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < MC; ++r) {
    if (r < rank) {
      n_freed += tot[r].x;
      n_moved += tot[r].y;
    }
    count += tot[r].y;
  }
  int2* const dst = p.ws_dst + (size_t)item * p.list_cap;
  int4* const src = p.ws_src + (size_t)item * p.list_cap;
  const int mask = (1 << p.map.page_shift) - 1;
  const unsigned below = (1u << lane) - 1;
  for (int base = wlo; base < whi; base += 32 * kEN) {
    load_pages(base);
    load_slots(base);
    if constexpr (!REG) {
#pragma unroll
      for (int u = 0; u < kEN; ++u) key[u] = make_key(base + u * 32 + lane, wv[u], pv[u]);
    }
#pragma unroll
    for (int u = 0; u < kEN; ++u) {
      const int j0 = base + u * 32, j = j0 + lane;
      if (j0 >= whi) continue;
      bool kept = key[u] > prefix;
      if (any_eq) {
        const bool is_eq = key[u] == prefix;
        const unsigned m = __ballot_sync(0xffffffffu, is_eq);
        kept |= is_eq && eq + __popc(m & below) < need;
        eq += __popc(m);
      }
      const bool ok = page_ok(p.map, pg[u]);
      const int row = ok ? ((pg[u] * p.map.nk + g) << p.map.page_shift) + (j & mask) : -1;   // below 2^31
      if (!ok && j < whi && kept == (j >= keep)) set_err(p.err, SWA_DERR_PAGE);   // a freed or a moved slot's
      if (j0 < keep) {
        const bool freed = j < min(whi, keep) && !kept;
        const unsigned m = __ballot_sync(0xffffffffu, freed);
        if (freed) dst[n_freed + __popc(m & below)] = make_int2(j, row);
        n_freed += __popc(m);
        if (kept && j < keep) {
          (wo + base + lane)[u * 32] = wv[u];
          (po + base + lane)[u * 32] = pv[u];
        }
      }
      if (j0 + 31 >= keep) {
        const bool moved = kept && j >= keep;
        const unsigned m = __ballot_sync(0xffffffffu, moved);
        if (moved) src[n_moved + __popc(m & below)] = make_int4(row, __float_as_int(wv[u]), pv[u], 0);
        n_moved += __popc(m);
      }
    }
    if constexpr (REG) break;
  }
  sync_all();                           // the lists are complete (and no histogram is read any more)

  // weights and positions of the moved slots
  for (int i = rank * kEThreads + tid; i < count; i += CS * kEThreads) {
    const int to = dst[i].x;
    const int4 x = src[i];
    wo[to] = __int_as_float(x.y);
    po[to] = x.z;
  }
  // rows: ch = 8, 16 or 32 lanes a row of K (job 2 i) or V (2 i + 1), kRows of them under way
  constexpr int kRows = 8;
  const int ch = p.hd / 8, lc = tid % ch, stride = CS * kEThreads / ch, jobs = 2 * count;
  for (int q = rank * (kEThreads / ch) + tid / ch; q < jobs; q += kRows * stride) {
    int to[kRows], of[kRows];
    uint4 v[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int job = min(q + k * stride, jobs - 1);
      to[k] = dst[job >> 1].y;
      of[k] = src[job >> 1].x;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int job = q + k * stride;
      if (job >= jobs || of[k] < 0) to[k] = -1;
      if (to[k] >= 0) v[k] = static_cast<const uint4*>(job & 1 ? p.cv : p.ck)[(size_t)of[k] * ch + lc];
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (to[k] >= 0) static_cast<uint4*>((q + k * stride) & 1 ? p.cv : p.ck)[(size_t)to[k] * ch + lc] = v[k];
  }
}

static size_t evict_list_cap(const swa_paged_evict_args* a) {
  const long long cap = (long long)a->cache.max_pages * a->cache.page;
  return (size_t)(a->keep < cap ? a->keep : cap);
}
static bool evict_sizes_ok(const swa_paged_evict_args* a) {
  const swa_paged_cache& c = a->cache;
  return c.B >= 1 && c.B <= 65535 && c.nk >= 1 && c.nk <= 65535 && (long long)c.B * c.nk <= (1 << 24) &&
         c.page >= 16 && c.page <= 256 && (c.page & (c.page - 1)) == 0 && c.max_pages >= 1 &&
         c.max_pages <= (1 << 30) / c.page && a->keep >= 1 && a->sinks >= 0;
}

}  // namespace swa

using namespace swa;

extern "C" {

size_t swa_paged_evict_workspace_size(const swa_paged_evict_args* a) {
  if (!a || !evict_sizes_ok(a)) return 0;
  const size_t items = (size_t)a->cache.B * a->cache.nk;
  return up256s(items * evict_list_cap(a) * sizeof(int2)) + up256s(items * evict_list_cap(a) * sizeof(int4));
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
  p.ws_dst = reinterpret_cast<int2*>(ws);
  p.ws_src = reinterpret_cast<int4*>(ws + up256s(items * p.list_cap * sizeof(int2)));
  p.err = a->err;
  // a CTA for every kSlotsPerCta slots of the capacity, 1, 2, 4 or 8 of them a cluster
  int cs = 1;
  while (cs < kMaxCluster && (long long)cs * kSlotsPerCta < p.map.cap) cs *= 2;
  if (cs == 1)
    return finish_launch(launch_pdl(paged_evict_kernel<false, true>, dim3((unsigned)items), dim3(kEThreads), 0, stream, p));
  const int share = ((p.map.cap + cs - 1) / cs + 31) & ~31;
  const bool reg = share <= kSlotsPerCta;
  if (!reg) {
    p.key_slots = share < kMaxKeySlots ? share : kMaxKeySlots;
    const cudaError_t e = allow_smem<paged_evict_kernel<true, false>>(kMaxKeySlots * 4);
    if (e != cudaSuccess) return cuda_status(e);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * cs));
  cfg.blockDim = dim3(kEThreads);
  cfg.dynamicSmemBytes = (size_t)p.key_slots * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return finish_launch(reg ? cudaLaunchKernelEx(&cfg, paged_evict_kernel<true, true>, p)
                           : cudaLaunchKernelEx(&cfg, paged_evict_kernel<true, false>, p));
}

}  // extern "C"
