// Pages that sequences share: swa_paged_fork (the next batch's tables, counts of holders,
// copies of pages about to be written) and swa_paged_compact (pages in use to the front).
//
// Both are integer work over the tables and the counts, a few passes with sums in between,
// and then copies of whole pages. The passes are bound by latency, not by what they read, the copies by
// memory. Where the counts fit in shared memory and the tables are short, one launch does everything: every SM's CTA
// makes the passes for itself, the first one writes the outputs (counts in place: the last one), and each copies its share (waiting for
// another launch, or for the other SMs, would take longer than the passes). Otherwise one cluster of 8 CTAs
// makes them in global memory, with the cluster's barrier (which orders it among them) in place of the block's, and a
// second launch copies from the list that it leaves in the workspace.
// Sums are of whole numbers and every list is in ascending order: the result does not
// depend on timing.
#include <cooperative_groups.h>

#include "swa_paged.cuh"

namespace swa {
namespace cg = cooperative_groups;

constexpr int kPCtas = 8, kPThreads = 512;    // of the cluster
constexpr int kOneThreads = 1024;             // of a CTA that makes all passes
// What it takes: pages and sequences that fit in shared memory, and table entries up to where the cluster is as fast (one
// launch against two, us: fork of 64 x 64 entries 8.4, 11.7; 256 x 64 21.1, 21.0; compact of 600 pages 5.4, 9.1; 6000 13.6, 15.8).
constexpr int kOnePages = 8192, kOneSeqs = 2048, kOneEntries = 32768;
constexpr int kCopyThreads = 256, kCopyUnit = kCopyThreads * 8 * 16;   // bytes that this many threads copy at a time

struct PageCopies {
  int pools;
  char* base[SWA_MAX_POOLS];
  long long bytes[SWA_MAX_POOLS];      // of a page
  long long units[SWA_MAX_POOLS];      // of a page, up to and with this pool
};

struct ForkParams {
  int B, R, num_pages, page_shift, max_pages, cap;
  uint64_t width_inv;                  // floor(2^64 / max_pages) + 1: x / max_pages = x * inv >> 64 for x < 2^32 (0: max_pages is 1)
  const int32_t* table;
  const int32_t* lens;
  const int32_t* parent;
  const int32_t* room;
  const int32_t* refs;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* refs_out;
  int32_t* left;
  int* children;                       // [B]
  int2* opens;                         // [num_pages]: new sequences that write the page next, the first of them
  int* free_list;                      // [num_pages]
  int* open_page;                      // [R]: the page that the sequence writes next, if it has begun, or -1
  int2* copies;                        // [R]
  int* count;
  int in_place;                        // refs_out is refs, and more than one CTA reads it
  uint32_t* err;
  PageCopies pages;
};

struct CompactParams {
  int num_pages;
  long long entries;                   // of the table
  const int32_t* table;
  const int32_t* refs;
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* moved;
  int32_t* used;
  int* refs_moved;                     // [num_pages] counts of the pages that move
  int2* copies;                        // [num_pages]
  int* count;
  int in_place;                        // refs_out is refs, and more than one CTA reads it
  uint32_t* err;
  PageCopies pages;
};

// Exclusive sums over the CTA's threads, and the totals (in every thread). s: an entry a warp.
template <int WARPS>
__device__ __forceinline__ int2 block_scan(int2 v, int2* s, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  __syncthreads();                     // s of the call before is read
  if (lane == 31) s[warp] = incl;
  __syncthreads();
  int2 w = lane < WARPS ? s[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  total = make_int2(__shfl_sync(0xffffffffu, w.x, WARPS - 1), __shfl_sync(0xffffffffu, w.y, WARPS - 1));
  const int2 front = make_int2(__shfl_sync(0xffffffffu, w.x, (warp - 1) & 31), __shfl_sync(0xffffffffu, w.y, (warp - 1) & 31));
  return make_int2(incl.x - v.x + (warp ? front.x : 0), incl.y - v.y + (warp ? front.y : 0));
}

// The CTAs of a launch: one, or a cluster
template <bool ONE>
struct Ctas {
  static constexpr int N = ONE ? 1 : kPCtas, THREADS = ONE ? kOneThreads : kPThreads, WARPS = THREADS / 32;
  __device__ __forceinline__ static int rank() {
    if constexpr (ONE) return 0;
    else return (int)cg::this_cluster().block_rank();
  }
  __device__ __forceinline__ static void sync() {
    if constexpr (ONE) __syncthreads();
    else cg::this_cluster().sync();
  }
};

// Sums of the CTAs before this one and of all, from a pair that each CTA has put into s_mine.
template <bool ONE>
__device__ __forceinline__ int2 cluster_base(int2* s_mine, int2& total) {
  if constexpr (ONE) {
    total = *s_mine;
    return make_int2(0, 0);
  } else {
    cg::cluster_group cl = cg::this_cluster();
    int2 before = make_int2(0, 0);
    total = make_int2(0, 0);
    for (int r = 0; r < kPCtas; ++r) {
      const int2 t = *cl.map_shared_rank(s_mine, r);
      if (r < (int)cl.block_rank()) {
        before.x += t.x;
        before.y += t.y;
      }
      total.x += t.x;
      total.y += t.y;
    }
    return before;
  }
}

// Group `who` of `all` groups of kCopyThreads threads copies its share of the listed pages (from, to) in all pools,
// kCopyUnit bytes at a time.
__device__ __forceinline__ void copy_pages(const PageCopies& p, const int2* list, int count, int who, int all, int thread) {
  if (!p.pools) return;
  const long long per = p.units[p.pools - 1], total = per * count;
  for (long long u = who; u < total; u += all) {
    const int2 c = list[u / per];
    if (c.y < 0) continue;             // there was no page for it
    const long long v = u % per;
    int i = 0;
    while (v >= p.units[i]) ++i;
    const long long at = (v - (i ? p.units[i - 1] : 0)) * kCopyUnit + thread * 16;
    const char* from = p.base[i] + c.x * p.bytes[i] + at;
    char* to = p.base[i] + c.y * p.bytes[i] + at;
    uint4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j * kCopyThreads * 16 < p.bytes[i]) x[j] = *reinterpret_cast<const uint4*>(from + j * kCopyThreads * 16);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j * kCopyThreads * 16 < p.bytes[i]) *reinterpret_cast<uint4*>(to + j * kCopyThreads * 16) = x[j];
  }
}

// Whether this CTA writes the counts (all have the same): the first one, or with the counts in place the last that has
// read them, by a ticket that was set to 0. No CTA waits for another.
__device__ __forceinline__ bool writes_counts(int in_place, int32_t* ticket) {
  if (!in_place) return blockIdx.x == 0;
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  return s_last;
}

template <bool ONE>
__global__ void __launch_bounds__(Ctas<ONE>::THREADS) paged_fork_kernel(const __grid_constant__ ForkParams p) {
  using C = Ctas<ONE>;
  extern __shared__ __align__(16) int s_one[];   // ONE: the parts below
  __shared__ int2 s_scan[C::WARPS];
  __shared__ int2 s_need, s_free;      // this CTA's sums: (pages, copies) its sequences need, (free pages, 0)
  const int rank = C::rank(), tid = threadIdx.x, all = C::N * C::THREADS, me = rank * C::THREADS + tid;
  int2* const opens = ONE ? reinterpret_cast<int2*>(s_one) : p.opens;
  int* const counts = ONE ? s_one + 2 * p.num_pages : p.refs_out;
  int* const free_list = ONE ? s_one + 3 * p.num_pages : p.free_list;
  int* const children = ONE ? s_one + 4 * p.num_pages + 2 * p.R : p.children;
  int2* const copies = ONE ? reinterpret_cast<int2*>(s_one + 4 * p.num_pages) : p.copies;
  int* const new_lens = ONE ? children + p.B : p.lens_out;
  int* const open_page = ONE ? new_lens + p.R : p.open_page;
  // ONE reads what is read again and again once, all of it at the start
  const int32_t* const lens = ONE ? open_page + p.R : p.lens;
  const int32_t* const parent = ONE ? lens + p.B : p.parent;
  const int32_t* const room = ONE ? parent + p.R : p.room;
  const bool writes = !ONE || blockIdx.x == 0;
  const int page = 1 << p.page_shift;
  uint32_t bits = 0;
  auto ok = [&](int e) { return (unsigned)e < (unsigned)p.num_pages; };
  auto keys = [&](int b) {             // of old sequence b
    const int n = lens[b];
    if (n < 0 || n > p.cap) bits |= SWA_DERR_META;
    return n < 0 ? 0 : min(n, p.cap);
  };
  auto over_width = [&](unsigned x) { return p.width_inv ? (int)__umul64hi(x, p.width_inv) : (int)x; };
  auto pages_of = [&](int n) { return (n >> p.page_shift) + ((n & (page - 1)) != 0); };   // n + page - 1 may pass 31 bits
  auto parent_of = [&](int r) {
    const int q = parent[r];
    if (q < -1 || q >= p.B) bits |= SWA_DERR_META;
    return q < -1 || q >= p.B ? -1 : q;
  };
  pdl_wait();
  pdl_trigger();

  for (int b = me; b < p.B; b += all) {
    children[b] = 0;
    if (ONE) const_cast<int32_t*>(lens)[b] = p.lens[b];
  }
  if (ONE)
    for (int r = me; r < p.R; r += all) {
      const_cast<int32_t*>(parent)[r] = p.parent[r];
      if (p.room) const_cast<int32_t*>(room)[r] = p.room[r];
    }
  if (counts != p.refs)
    for (int i = me; i < p.num_pages; i += all) counts[i] = p.refs[i];
  C::sync();

  for (int r = me; r < p.R; r += all) {
    const int q = parent_of(r), n = q < 0 ? 0 : keys(q);
    new_lens[r] = n;
    if (ONE && writes) p.lens_out[r] = n;
    open_page[r] = -1;
    if (q >= 0) atomicAdd(&children[q], 1);
  }
  C::sync();

  // the old rows let go, the new ones hold: a page changes by (children that keep it) - 1
  const unsigned width = p.max_pages, old_entries = p.B * width, new_entries = p.R * width;   // below 2^31
  for (unsigned x = me; x < old_entries; x += all) {
    const int e = p.table[x];
    if (!ok(e)) continue;
    const int b = over_width(x), i = x - b * width;
    const int d = (i < pages_of(keys(b)) ? children[b] : 0) - 1;
    if (d) atomicAdd(&counts[e], d);
  }
  for (unsigned x = me; x < new_entries; x += all) {
    const int r = over_width(x), i = x - r * width, n = new_lens[r];
    int e = -1;
    if (i < pages_of(n)) {
      e = p.table[(long long)parent_of(r) * p.max_pages + i];
      if (!ok(e)) {
        bits |= SWA_DERR_PAGE;
        e = -1;
      } else if (i == n >> p.page_shift) {
        opens[e] = make_int2(0, p.R);   // the page of slot n, begun: every writer of it sets the same
        open_page[r] = e;
      }
    }
    if (writes) p.table_out[x] = e;
  }
  C::sync();

  for (int r = me; r < p.R; r += all) {
    const int e = open_page[r];
    if (e < 0) continue;
    atomicAdd(&opens[e].x, 1);
    atomicMin(&opens[e].y, r);
  }
  C::sync();

  // what each sequence needs (CTAs and threads take consecutive ones), and the free pages
  auto copied = [&](int r) {           // the counts are those of step 2 until the barriers below
    const int e = open_page[r];
    if (e < 0 || counts[e] < 2) return false;
    const int2 o = opens[e];
    return !(o.x == counts[e] && o.y == r);
  };
  auto grows = [&](int r) {
    const int n = new_lens[r];
    int more = p.room ? room[r] : 0;
    if (more > p.cap - n) bits |= SWA_DERR_META;
    more = more < 0 ? 0 : min(more, p.cap - n);
    return pages_of(n + more) - pages_of(n);
  };
  const int r_share = (p.R + all - 1) / all, r0 = min(p.R, me * r_share), r1 = min(p.R, r0 + r_share);
  uint32_t gets = 0;                   // bit j: sequence r0 + j (16 a thread at most) gets a copy
  int2 need = make_int2(0, 0), need_cta;
  for (int r = r0; r < r1; ++r) {
    const bool c = copied(r);
    gets |= (uint32_t)c << (r - r0);
    need.x += grows(r) + c;
    need.y += c;
  }
  int2 at = block_scan<C::WARPS>(need, s_scan, need_cta);
  // pages: a CTA takes a run of them
  const int run = ((p.num_pages + C::N - 1) / C::N + 3) & ~3, p0 = min(p.num_pages, rank * run), p1 = min(p.num_pages, p0 + run);
  int2 free = make_int2(0, 0), free_cta;
  for (int i = p0 + tid; i < p1; i += C::THREADS) {
    const int c = counts[i];
    if (c < 0) bits |= SWA_DERR_META;
    free.x += c == 0;
  }
  block_scan<C::WARPS>(free, s_scan, free_cta);
  if (tid == 0) {
    s_need = need_cta;
    s_free = free_cta;
  }
  C::sync();
  int2 need_all, free_all;
  const int2 need_before = cluster_base<ONE>(&s_need, need_all);
  int k = cluster_base<ONE>(&s_free, free_all).x;     // free pages before this CTA's run
  for (int i0 = p0; i0 < p1 && k < need_all.x; i0 += 4 * C::THREADS) {
    const int i = i0 + 4 * tid;
    bool c[4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = i + j < p1 && counts[i + j] == 0;
      n += c[j];
    }
    int2 sum;
    int to = k + block_scan<C::WARPS>(make_int2(n, 0), s_scan, sum).x;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c[j]) free_list[to++] = i + j;
    k += sum.x;
  }
  C::sync();                           // and the sums of the other CTAs are read

  at.x += need_before.x;
  at.y += need_before.y;
  auto take = [&]() {
    const int e = at.x < free_all.x ? free_list[at.x] : -1;
    ++at.x;
    if (e < 0)
      bits |= SWA_DERR_FULL;
    else
      counts[e] = 1;
    return e;
  };
  for (int r = r0; r < r1; ++r) {
    const int g = grows(r), first = pages_of(new_lens[r]);
    int32_t* row = p.table_out + (long long)r * p.max_pages;
    if (gets >> (r - r0) & 1) {
      const int from = open_page[r], to = take();
      copies[at.y++] = make_int2(from, to);
      atomicSub(&counts[from], 1);
      if (writes) row[first - 1] = to;
    }
    for (int i = 0; i < g; ++i) {
      const int e = take();
      if (writes) row[first + i] = e;
    }
  }
  if (!ONE && me == 0) {
    *p.left = free_all.x - need_all.x;
    *p.count = need_all.y;
  }
  if (bits && writes) set_err(p.err, bits);
  if constexpr (ONE) {
    __syncthreads();
    if (writes_counts(p.in_place, p.left)) {
      for (int i = tid; i < p.num_pages; i += C::THREADS) p.refs_out[i] = counts[i];
      if (tid == 0) *p.left = free_all.x - need_all.x;
    }
    constexpr int G = C::THREADS / kCopyThreads;
    copy_pages(p.pages, copies, need_all.y, blockIdx.x * G + tid / kCopyThreads, gridDim.x * G, tid % kCopyThreads);
  }
}

template <bool ONE>
__global__ void __launch_bounds__(Ctas<ONE>::THREADS) paged_compact_kernel(const __grid_constant__ CompactParams p) {
  using C = Ctas<ONE>;
  extern __shared__ __align__(16) int s_one[];   // ONE: moves, counts, new places, counts of what moves
  __shared__ int2 s_scan[C::WARPS];
  __shared__ int2 s_used, s_lists;     // this CTA's sums: (pages in use, 0), (free ones below n, ones that move)
  const int rank = C::rank(), tid = threadIdx.x, all = C::N * C::THREADS, me = rank * C::THREADS + tid;
  // half of the pages move at most
  int2* const copies = ONE ? reinterpret_cast<int2*>(s_one) : p.copies;
  const int moves = (p.num_pages + 1) / 2;
  int* const s_refs = s_one + 2 * moves;
  const int32_t* const refs = ONE ? s_refs : p.refs;
  int* const moved = ONE ? s_refs + p.num_pages : p.moved;
  int* const refs_moved = ONE ? s_refs + 2 * p.num_pages : p.refs_moved;
  const bool writes = !ONE || blockIdx.x == 0;
  const int run = ((p.num_pages + C::N - 1) / C::N + 3) & ~3, p0 = min(p.num_pages, rank * run), p1 = min(p.num_pages, p0 + run);
  uint32_t bits = 0;
  pdl_wait();
  pdl_trigger();

  int2 used = make_int2(0, 0), used_cta, used_all;
  for (int i = p0 + tid; i < p1; i += C::THREADS) {
    const int c = p.refs[i];
    if (ONE) s_refs[i] = c;
    if (c < 0) bits |= SWA_DERR_META;
    used.x += c != 0;
  }
  block_scan<C::WARPS>(used, s_scan, used_cta);
  if (tid == 0) s_used = used_cta;
  C::sync();
  cluster_base<ONE>(&s_used, used_all);
  const int n = used_all.x;
  auto kind = [&](int i, int c) { return make_int2(c == 0 && i < n, c != 0 && i >= n); };

  int2 lists = make_int2(0, 0), lists_cta, lists_all;
  for (int i = p0 + tid; i < p1; i += C::THREADS) {
    const int2 w = kind(i, refs[i]);
    lists.x += w.x;
    lists.y += w.y;
  }
  block_scan<C::WARPS>(lists, s_scan, lists_cta);
  if (tid == 0) s_lists = lists_cta;
  C::sync();
  int2 k = cluster_base<ONE>(&s_lists, lists_all);
  for (int i0 = p0; i0 < p1; i0 += 4 * C::THREADS) {
    const int i = i0 + 4 * tid;
    int c[4];
    int2 w[4], sum = make_int2(0, 0), step;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = i + j < p1 ? refs[i + j] : 0;
      w[j] = i + j < p1 ? kind(i + j, c[j]) : make_int2(0, 0);
      sum.x += w[j].x;
      sum.y += w[j].y;
    }
    int2 to = block_scan<C::WARPS>(sum, s_scan, step);
    to.x += k.x;
    to.y += k.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j >= p1) continue;
      if (w[j].y) {                    // its count and new place: below
        copies[to.y].x = i + j;
        refs_moved[to.y++] = c[j];
        continue;
      }
      moved[i + j] = c[j] ? i + j : -1;
      if (w[j].x)
        copies[to.x++].y = i + j;
      else if (!ONE)
        p.refs_out[i + j] = c[j];
    }
    k.x += step.x;
    k.y += step.y;
  }
  C::sync();
  const bool writes_refs = !ONE || writes_counts(p.in_place, p.used);
  if (ONE && writes_refs)
    for (int i = tid; i < p.num_pages; i += C::THREADS) {
      const int c = refs[i];
      if (!kind(i, c).x && !kind(i, c).y) p.refs_out[i] = c;
    }
  for (int x = me; x < lists_all.y; x += all) {
    const int2 c = copies[x];
    moved[c.x] = c.y;
    if (writes_refs) {
      p.refs_out[c.y] = refs_moved[x];
      p.refs_out[c.x] = 0;
    }
  }
  C::sync();
  if (writes) {
    for (long long x = me; x < p.entries; x += all) {
      int e = p.table[x];
      if ((unsigned)e < (unsigned)p.num_pages) {
        e = moved[e];
        if (e < 0) bits |= SWA_DERR_PAGE;
      }
      p.table_out[x] = e;
    }
    if (ONE)
      for (int i = tid; i < p.num_pages; i += C::THREADS) p.moved[i] = moved[i];
    if (!ONE && me == 0) *p.count = lists_all.y;
    if (bits) set_err(p.err, bits);
  }
  if (writes_refs && me == 0) *p.used = n;
  if constexpr (ONE) {
    constexpr int G = C::THREADS / kCopyThreads;
    copy_pages(p.pages, copies, lists_all.y, blockIdx.x * G + tid / kCopyThreads, gridDim.x * G, tid % kCopyThreads);
  }
}

__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const __grid_constant__ PageCopies p, const int2* list, const int* count) {
  pdl_wait();
  pdl_trigger();
  copy_pages(p, list, *count, blockIdx.x, gridDim.x, threadIdx.x);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Span {
  const void* at;
  size_t bytes;
};

static bool pools_sizes_ok(const swa_page_pools& c) {
  return c.num_pages >= 1 && c.num_pages < (1 << 30) && c.pools >= 0 && c.pools <= SWA_MAX_POOLS;
}
// Status of the pools; their spans are added to s (n entries so far).
static int pools_status(const swa_page_pools& c, Span* s, int* n) {
  for (int i = 0; i < c.pools; ++i) {
    if (!c.base[i]) return SWA_E_NULL;
    if (c.page_bytes[i] < 16 || c.page_bytes[i] > (1LL << 46) / c.num_pages) return SWA_E_SHAPE;
    if (!aligned16p(c.base[i]) || (c.page_bytes[i] & 15)) return SWA_E_ALIGN;
    s[(*n)++] = {c.base[i], (size_t)c.page_bytes[i] * c.num_pages};
  }
  return SWA_OK;
}
// The first `written` spans are written: each is apart from all others.
static bool spans_apart(const Span* s, int n, int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (bytes_overlap(s[i].at, s[i].bytes, s[j].at, s[j].bytes)) return false;
  return true;
}
static bool words_aligned(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(s[i].at) & 3u) return false;
  return true;
}

static PageCopies copies_of(const swa_page_pools& c) {
  PageCopies p{};
  p.pools = c.pools;
  long long units = 0;
  for (int i = 0; i < c.pools; ++i) {
    p.base[i] = static_cast<char*>(c.base[i]);
    p.bytes[i] = c.page_bytes[i];
    p.units[i] = units += (c.page_bytes[i] + kCopyUnit - 1) / kCopyUnit;
  }
  return p;
}

// One launch of a CTA an SM with `smem` bytes of shared memory (`most` at most). With the counts in place `ticket`, an output, is
// set to 0 before it. (A grid that waits for itself needs every SM at once: it starts when no other stream holds one, and
// not at all where a process has fewer. Of 64 beams, and 32 prompts continued eight ways, on the GPU: apart 9.5 and 20.0 us, in place
// 14.9 and 25.4, with a second launch for the counts 16.7 and 29.6, as a grid that waits 11.0 and 21.4.)
template <auto One, typename P>
static int launch_one(size_t smem, int most, P& p, bool in_place, int32_t* ticket, cudaStream_t s) {
  cudaError_t e = allow_smem<One>(most);
  if (e != cudaSuccess) return cuda_status(e);
  const dim3 grid(p.pages.pools ? (num_sms() > 0 ? num_sms() : 148) : 1);
  p.in_place = in_place && grid.x > 1;
  if (p.in_place && (e = cudaMemsetAsync(ticket, 0, sizeof(int32_t), s)) != cudaSuccess) return cuda_status(e);
  return finish_launch(launch_pdl(One, grid, dim3(kOneThreads), smem, s, p));
}
// The passes on a cluster, then the copies of at most `most` pages
template <auto Many, typename P>
static int launch_many(const P& p, long long most, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPCtas);
  cfg.blockDim = dim3(kPThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const int rc = finish_launch(cudaLaunchKernelEx(&cfg, Many, p));
  if (rc != SWA_OK || !p.pages.pools) return rc;
  const long long sms = num_sms() > 0 ? num_sms() : 148, units = p.pages.units[p.pages.pools - 1] * most;
  const long long grid = units < 8 * sms ? units : 8 * sms;   // 8 CTAs an SM: 128 KB of loads under way
  return finish_launch(launch_pdl(paged_copy_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, s, p.pages,
                                  (const int2*)p.copies, (const int*)p.count));
}

// offsets of the fork's parts of the workspace, from the front; .. + total
struct ForkPlan {
  bool one;                            // everything in one launch, without a workspace (bytes = 0)
  size_t opens, list, copies, open_page, count, bytes;
};
static bool fork_plan(const swa_paged_fork_args* a, ForkPlan* w) {
  if (!pools_sizes_ok(a->pools) || a->B < 1 || a->B > 65535 || a->R < 1 || a->R > 65535) return false;
  if (a->page < 16 || a->page > 256 || (a->page & (a->page - 1))) return false;
  if (a->max_pages < 1 || a->max_pages > (1 << 30) / a->page) return false;
  if ((long long)a->B * a->max_pages >= (1LL << 31) || (long long)a->R * a->max_pages >= (1LL << 31)) return false;
  *w = ForkPlan{};
  w->one = a->pools.num_pages <= kOnePages && a->B <= kOneSeqs && a->R <= kOneSeqs && ((long long)a->B + a->R) * a->max_pages <= kOneEntries;
  if (w->one) return true;
  w->opens = up256s((size_t)a->B * 4);
  w->list = w->opens + up256s((size_t)a->pools.num_pages * 8);
  w->copies = w->list + up256s((size_t)a->pools.num_pages * 4);
  w->open_page = w->copies + up256s((size_t)a->R * 8);
  w->count = w->open_page + up256s((size_t)a->R * 4);
  w->bytes = w->count + 256;
  return true;
}
struct CompactPlan {
  bool one;
  size_t copies, count, bytes;
};
static bool compact_plan(const swa_paged_compact_args* a, CompactPlan* w) {
  if (!pools_sizes_ok(a->pools) || a->B < 1 || a->B > 65535) return false;
  if (a->max_pages < 1 || a->max_pages > (1 << 26) || (long long)a->B * a->max_pages >= (1LL << 31)) return false;
  *w = CompactPlan{};
  w->one = a->pools.num_pages <= kOnePages && (long long)a->B * a->max_pages <= kOneEntries;
  if (w->one) return true;
  w->copies = up256s((size_t)a->pools.num_pages * 4);
  w->count = w->copies + up256s((size_t)a->pools.num_pages * 8);
  w->bytes = w->count + 256;
  return true;
}

}  // namespace swa

using namespace swa;

extern "C" {

size_t swa_paged_fork_workspace_size(const swa_paged_fork_args* a) {
  ForkPlan w;
  return a && fork_plan(a, &w) ? (w.bytes ? w.bytes : 1) : 0;
}

int swa_paged_fork(const swa_paged_fork_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  if (!a->table || !a->lens || !a->parent || !a->refs || !a->table_out || !a->lens_out || !a->refs_out || !a->left)
    return SWA_E_NULL;
  ForkPlan w;
  if (!fork_plan(a, &w)) return SWA_E_SHAPE;
  const size_t pages = (size_t)a->pools.num_pages * 4;
  const Span words[9] = {{a->table_out, (size_t)a->R * a->max_pages * 4}, {a->lens_out, (size_t)a->R * 4}, {a->refs_out, pages},
                         {a->left, 4}, {a->refs, pages}, {a->table, (size_t)a->B * a->max_pages * 4}, {a->lens, (size_t)a->B * 4},
                         {a->parent, (size_t)a->R * 4}, {a->room, a->room ? (size_t)a->R * 4 : 0}};
  Span s[10 + SWA_MAX_POOLS];
  int n = 0;
  const int rc = pools_status(a->pools, s, &n);
  if (rc != SWA_OK) return rc;
  if (!words_aligned(words, 9) || (reinterpret_cast<uintptr_t>(a->workspace) & 255u)) return SWA_E_ALIGN;
  if (w.bytes && (!a->workspace || a->workspace_bytes < w.bytes)) return SWA_E_WORKSPACE;
  if (w.bytes) s[n++] = {a->workspace, w.bytes};
  for (int i = 0; i < 4; ++i) s[n++] = words[i];
  const int written = n;
  for (int i = 4; i < 9; ++i)
    if (words[i].bytes && !(i == 4 && a->refs == a->refs_out)) s[n++] = words[i];
  if (!spans_apart(s, n, written)) return SWA_E_SHAPE;
  ForkParams p{};
  p.B = a->B; p.R = a->R; p.num_pages = a->pools.num_pages; p.max_pages = a->max_pages;
  while ((1 << p.page_shift) < a->page) ++p.page_shift;
  p.cap = a->max_pages << p.page_shift;
  p.width_inv = a->max_pages > 1 ? ~0ull / a->max_pages + 1 : 0;
  p.table = a->table; p.lens = a->lens; p.parent = a->parent; p.room = a->room; p.refs = a->refs;
  p.table_out = a->table_out; p.lens_out = a->lens_out; p.refs_out = a->refs_out; p.left = a->left;
  p.err = a->err;
  p.pages = copies_of(a->pools);
  if (w.one)
    return launch_one<paged_fork_kernel<true>>((size_t)p.num_pages * 16 + (size_t)p.R * 24 + (size_t)p.B * 8,
                                               kOnePages * 16 + kOneSeqs * 32, p, a->refs == a->refs_out, a->left, stream);
  char* ws = static_cast<char*>(a->workspace);
  p.children = reinterpret_cast<int*>(ws);
  p.opens = reinterpret_cast<int2*>(ws + w.opens);
  p.free_list = reinterpret_cast<int*>(ws + w.list);
  p.copies = reinterpret_cast<int2*>(ws + w.copies);
  p.open_page = reinterpret_cast<int*>(ws + w.open_page);
  p.count = reinterpret_cast<int*>(ws + w.count);
  return launch_many<paged_fork_kernel<false>>(p, a->R, stream);
}

size_t swa_paged_compact_workspace_size(const swa_paged_compact_args* a) {
  CompactPlan w;
  return a && compact_plan(a, &w) ? (w.bytes ? w.bytes : 1) : 0;
}

int swa_paged_compact(const swa_paged_compact_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  if (!a->table || !a->refs || !a->table_out || !a->refs_out || !a->moved || !a->used) return SWA_E_NULL;
  CompactPlan w;
  if (!compact_plan(a, &w)) return SWA_E_SHAPE;
  const size_t pages = (size_t)a->pools.num_pages * 4, entries = (size_t)a->B * a->max_pages;
  const Span words[6] = {{a->table_out, entries * 4}, {a->refs_out, pages}, {a->moved, pages}, {a->used, 4}, {a->table, entries * 4}, {a->refs, pages}};
  Span s[7 + SWA_MAX_POOLS];
  int n = 0;
  const int rc = pools_status(a->pools, s, &n);
  if (rc != SWA_OK) return rc;
  if (!words_aligned(words, 6) || (reinterpret_cast<uintptr_t>(a->workspace) & 255u)) return SWA_E_ALIGN;
  if (w.bytes && (!a->workspace || a->workspace_bytes < w.bytes)) return SWA_E_WORKSPACE;
  if (w.bytes) s[n++] = {a->workspace, w.bytes};
  for (int i = 0; i < 4; ++i) s[n++] = words[i];
  const int written = n;
  if (a->table != a->table_out) s[n++] = words[4];
  if (a->refs != a->refs_out) s[n++] = words[5];
  if (!spans_apart(s, n, written)) return SWA_E_SHAPE;
  CompactParams p{};
  p.num_pages = a->pools.num_pages;
  p.entries = (long long)entries;
  p.table = a->table; p.refs = a->refs;
  p.table_out = a->table_out; p.refs_out = a->refs_out; p.moved = a->moved; p.used = a->used;
  p.err = a->err;
  p.pages = copies_of(a->pools);
  if (w.one)
    return launch_one<paged_compact_kernel<true>>((size_t)p.num_pages * 8 + (size_t)((p.num_pages + 1) / 2) * 12, kOnePages * 14, p,
                                                  a->refs == a->refs_out, a->used, stream);
  char* ws = static_cast<char*>(a->workspace);
  p.refs_moved = reinterpret_cast<int*>(ws);
  p.copies = reinterpret_cast<int2*>(ws + w.copies);
  p.count = reinterpret_cast<int*>(ws + w.count);
  return launch_many<paged_compact_kernel<false>>(p, (p.num_pages + 1) / 2, stream);
}

}  // extern "C"
