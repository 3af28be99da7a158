// Pages that sequences share: swa_paged_fork (the next batch's tables, counts of holders,
// copies of pages about to be written) and swa_paged_compact (pages in use to the front).
//
// Both are integer work over the tables and the counts, a few passes with sums in between,
// and then copies of whole pages. The passes are bound by latency, not by what they read: one
// cluster of 8 CTAs does them all in one launch, with the cluster's barrier (which orders global
// memory among its CTAs) between them. The copies are bound by memory: a second launch
// over all SMs takes them from the list that the first one leaves in the workspace.
// Sums are of whole numbers and every list is in ascending order: the result does not
// depend on timing.
#include <cooperative_groups.h>

#include "swa_paged.cuh"

namespace swa {
namespace cg = cooperative_groups;

constexpr int kPCtas = 8, kPThreads = 512, kPWarps = kPThreads / 32;
constexpr int kCopyThreads = 256, kCopyUnit = kCopyThreads * 4 * 16;   // bytes that a CTA copies at a time

struct PageCopies {
  int pools;
  char* base[SWA_MAX_POOLS];
  long long bytes[SWA_MAX_POOLS];      // of a page
  long long units[SWA_MAX_POOLS];      // of a page, up to and with this pool
  const int2* list;                    // (from, to)
  const int* count;
};

struct ForkParams {
  int B, R, num_pages, page_shift, max_pages, cap;
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
  int2* copies;                        // [R]
  int* count;
  uint32_t* err;
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
  uint32_t* err;
};

// Exclusive sums over the CTA's threads, and the totals (in every thread). s: kPWarps entries.
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
  int2 before = make_int2(incl.x - v.x, incl.y - v.y);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kPWarps; ++w) {
    const int2 t = s[w];
    if (w < warp) {
      before.x += t.x;
      before.y += t.y;
    }
    total.x += t.x;
    total.y += t.y;
  }
  return before;
}

// Sums of the CTAs before this one and of all, from a pair that each CTA has put into s_mine.
__device__ __forceinline__ int2 cluster_base(cg::cluster_group& cl, int2* s_mine, int2& total) {
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

__global__ void __cluster_dims__(kPCtas, 1, 1) __launch_bounds__(kPThreads) paged_fork_kernel(const ForkParams p) {
  __shared__ int2 s_scan[kPWarps];
  __shared__ int2 s_need, s_free;      // this CTA's sums: (pages, copies) its sequences need, (free pages, 0)
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), tid = threadIdx.x, all = kPCtas * kPThreads, me = rank * kPThreads + tid;
  const int page = 1 << p.page_shift;
  uint32_t bits = 0;
  auto ok = [&](int e) { return (unsigned)e < (unsigned)p.num_pages; };
  auto keys = [&](int b) {             // of old sequence b
    const int n = p.lens[b];
    if (n < 0 || n > p.cap) bits |= SWA_DERR_META;
    return n < 0 ? 0 : min(n, p.cap);
  };
  auto pages_of = [&](int n) { return (n >> p.page_shift) + ((n & (page - 1)) != 0); };   // n + page - 1 may pass 31 bits
  auto parent_of = [&](int r) {
    const int q = p.parent[r];
    if (q < -1 || q >= p.B) bits |= SWA_DERR_META;
    return q < -1 || q >= p.B ? -1 : q;
  };
  pdl_wait();
  pdl_trigger();

  for (int b = me; b < p.B; b += all) p.children[b] = 0;
  if (p.refs_out != p.refs)
    for (int i = me; i < p.num_pages; i += all) p.refs_out[i] = p.refs[i];
  cl.sync();

  for (int r = me; r < p.R; r += all) {
    const int q = parent_of(r), n = q < 0 ? 0 : keys(q);
    p.lens_out[r] = n;
    if (q >= 0) atomicAdd(&p.children[q], 1);
  }
  cl.sync();

  // the old rows let go, the new ones hold: a page changes by (children that keep it) - 1
  const unsigned width = p.max_pages, old_entries = p.B * width, new_entries = p.R * width;   // below 2^31
  for (unsigned x = me; x < old_entries; x += all) {
    const int e = p.table[x];
    if (!ok(e)) continue;
    const int b = x / width, i = x % width;
    const int d = (i < pages_of(keys(b)) ? p.children[b] : 0) - 1;
    if (d) atomicAdd(&p.refs_out[e], d);
  }
  for (unsigned x = me; x < new_entries; x += all) {
    const int r = x / width, i = x % width, n = p.lens_out[r];
    int e = -1;
    if (i < pages_of(n)) {
      e = p.table[(long long)parent_of(r) * p.max_pages + i];
      if (!ok(e)) {
        bits |= SWA_DERR_PAGE;
        e = -1;
      } else if (i == n >> p.page_shift) {
        p.opens[e] = make_int2(0, p.R);   // the page of slot n, begun: every writer of it sets the same
      }
    }
    p.table_out[x] = e;
  }
  cl.sync();

  // the page that sequence r writes next, if it has begun
  auto open_page = [&](int r) {
    const int n = p.lens_out[r];
    return n & (page - 1) ? p.table_out[(long long)r * p.max_pages + (n >> p.page_shift)] : -1;
  };
  for (int r = me; r < p.R; r += all) {
    const int e = open_page(r);
    if (e < 0) continue;
    atomicAdd(&p.opens[e].x, 1);
    atomicMin(&p.opens[e].y, r);
  }
  cl.sync();

  // what each sequence needs (CTAs and threads take consecutive ones), and the free pages
  auto copied = [&](int r) {           // the counts are those of step 2 until the barriers below
    const int e = open_page(r);
    if (e < 0 || p.refs_out[e] < 2) return false;
    const int2 o = p.opens[e];
    return !(o.x == p.refs_out[e] && o.y == r);
  };
  auto grows = [&](int r) {
    const int n = p.lens_out[r];
    int room = p.room ? p.room[r] : 0;
    if (room > p.cap - n) bits |= SWA_DERR_META;
    room = room < 0 ? 0 : min(room, p.cap - n);
    return pages_of(n + room) - pages_of(n);
  };
  const int r_share = (p.R + all - 1) / all, r0 = min(p.R, me * r_share), r1 = min(p.R, r0 + r_share);
  uint32_t copies = 0;                 // bit j: sequence r0 + j (16 a thread at most) gets a copy
  int2 need = make_int2(0, 0), need_cta;
  for (int r = r0; r < r1; ++r) {
    const bool c = copied(r);
    copies |= (uint32_t)c << (r - r0);
    need.x += grows(r) + c;
    need.y += c;
  }
  int2 at = block_scan(need, s_scan, need_cta);
  // pages: a CTA takes a run of them
  const int run = ((p.num_pages + kPCtas - 1) / kPCtas + 3) & ~3, p0 = min(p.num_pages, rank * run), p1 = min(p.num_pages, p0 + run);
  int2 free = make_int2(0, 0), free_cta;
  for (int i = p0 + tid; i < p1; i += kPThreads) {
    const int c = p.refs_out[i];
    if (c < 0) bits |= SWA_DERR_META;
    free.x += c == 0;
  }
  block_scan(free, s_scan, free_cta);
  if (tid == 0) {
    s_need = need_cta;
    s_free = free_cta;
  }
  cl.sync();
  int2 need_all, free_all;
  const int2 need_before = cluster_base(cl, &s_need, need_all);
  int k = cluster_base(cl, &s_free, free_all).x;     // free pages before this CTA's run
  for (int i0 = p0; i0 < p1 && k < need_all.x; i0 += 4 * kPThreads) {
    const int i = i0 + 4 * tid;
    bool c[4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = i + j < p1 && p.refs_out[i + j] == 0;
      n += c[j];
    }
    int2 sum;
    int to = k + block_scan(make_int2(n, 0), s_scan, sum).x;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c[j]) p.free_list[to++] = i + j;
    k += sum.x;
  }
  cl.sync();                           // and the sums of the other CTAs are read

  at.x += need_before.x;
  at.y += need_before.y;
  auto take = [&]() {
    const int e = at.x < free_all.x ? p.free_list[at.x] : -1;
    ++at.x;
    if (e < 0)
      bits |= SWA_DERR_FULL;
    else
      p.refs_out[e] = 1;
    return e;
  };
  for (int r = r0; r < r1; ++r) {
    const int n = p.lens_out[r], g = grows(r), first = pages_of(n);
    int32_t* row = p.table_out + (long long)r * p.max_pages;
    if (copies >> (r - r0) & 1) {
      const int from = row[first - 1], to = take();
      p.copies[at.y++] = make_int2(from, to);
      atomicSub(&p.refs_out[from], 1);
      row[first - 1] = to;
    }
    for (int i = 0; i < g; ++i) row[first + i] = take();
  }
  if (me == 0) {
    *p.left = free_all.x - need_all.x;
    *p.count = need_all.y;
  }
  if (bits) set_err(p.err, bits);
}

__global__ void __cluster_dims__(kPCtas, 1, 1) __launch_bounds__(kPThreads) paged_compact_kernel(const CompactParams p) {
  __shared__ int2 s_scan[kPWarps];
  __shared__ int2 s_used, s_lists;     // this CTA's sums: (pages in use, 0), (free ones below n, ones that move)
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), tid = threadIdx.x, all = kPCtas * kPThreads, me = rank * kPThreads + tid;
  const int run = ((p.num_pages + kPCtas - 1) / kPCtas + 3) & ~3, p0 = min(p.num_pages, rank * run), p1 = min(p.num_pages, p0 + run);
  uint32_t bits = 0;
  pdl_wait();
  pdl_trigger();

  int2 used = make_int2(0, 0), used_cta, used_all;
  for (int i = p0 + tid; i < p1; i += kPThreads) {
    const int c = p.refs[i];
    if (c < 0) bits |= SWA_DERR_META;
    used.x += c != 0;
  }
  block_scan(used, s_scan, used_cta);
  if (tid == 0) s_used = used_cta;
  cl.sync();
  cluster_base(cl, &s_used, used_all);
  const int n = used_all.x;
  auto kind = [&](int i, int c) { return make_int2(c == 0 && i < n, c != 0 && i >= n); };

  int2 lists = make_int2(0, 0), lists_cta, lists_all;
  for (int i = p0 + tid; i < p1; i += kPThreads) {
    const int2 w = kind(i, p.refs[i]);
    lists.x += w.x;
    lists.y += w.y;
  }
  block_scan(lists, s_scan, lists_cta);
  if (tid == 0) s_lists = lists_cta;
  cl.sync();
  int2 k = cluster_base(cl, &s_lists, lists_all);
  for (int i0 = p0; i0 < p1; i0 += 4 * kPThreads) {
    const int i = i0 + 4 * tid;
    int c[4];
    int2 w[4], sum = make_int2(0, 0), step;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = i + j < p1 ? p.refs[i + j] : 0;
      w[j] = i + j < p1 ? kind(i + j, c[j]) : make_int2(0, 0);
      sum.x += w[j].x;
      sum.y += w[j].y;
    }
    int2 to = block_scan(sum, s_scan, step);
    to.x += k.x;
    to.y += k.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j >= p1) continue;
      if (w[j].y) {                    // its count and new place: below
        p.copies[to.y].x = i + j;
        p.refs_moved[to.y++] = c[j];
        continue;
      }
      p.moved[i + j] = c[j] ? i + j : -1;
      if (w[j].x)
        p.copies[to.x++].y = i + j;
      else
        p.refs_out[i + j] = c[j];
    }
    k.x += step.x;
    k.y += step.y;
  }
  cl.sync();
  for (int x = me; x < lists_all.y; x += all) {
    const int2 c = p.copies[x];
    p.moved[c.x] = c.y;
    p.refs_out[c.y] = p.refs_moved[x];
    p.refs_out[c.x] = 0;
  }
  cl.sync();
  for (long long x = me; x < p.entries; x += all) {
    int e = p.table[x];
    if ((unsigned)e < (unsigned)p.num_pages) {
      e = p.moved[e];
      if (e < 0) bits |= SWA_DERR_PAGE;
    }
    p.table_out[x] = e;
  }
  if (me == 0) {
    *p.used = n;
    *p.count = lists_all.y;
  }
  if (bits) set_err(p.err, bits);
}

// The listed pages, kCopyUnit bytes at a time, over all pools.
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const __grid_constant__ PageCopies p) {
  pdl_wait();
  pdl_trigger();
  const long long per = p.units[p.pools - 1], total = per * *p.count;
  for (long long u = blockIdx.x; u < total; u += gridDim.x) {
    const int2 c = p.list[u / per];
    if (c.y < 0) continue;             // there was no page for it
    const long long v = u % per;
    int i = 0;
    while (v >= p.units[i]) ++i;
    const long long at = (v - (i ? p.units[i - 1] : 0)) * kCopyUnit + threadIdx.x * 16;
    const char* from = p.base[i] + c.x * p.bytes[i] + at;
    char* to = p.base[i] + c.y * p.bytes[i] + at;
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j * kCopyThreads * 16 < p.bytes[i]) x[j] = *reinterpret_cast<const uint4*>(from + j * kCopyThreads * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j * kCopyThreads * 16 < p.bytes[i]) *reinterpret_cast<uint4*>(to + j * kCopyThreads * 16) = x[j];
  }
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

static int launch_copies(const swa_page_pools& c, const int2* list, const int* count, long long most, cudaStream_t s) {
  if (!c.pools) return SWA_OK;
  PageCopies p{};
  p.pools = c.pools;
  long long units = 0;
  for (int i = 0; i < c.pools; ++i) {
    p.base[i] = static_cast<char*>(c.base[i]);
    p.bytes[i] = c.page_bytes[i];
    p.units[i] = units += (c.page_bytes[i] + kCopyUnit - 1) / kCopyUnit;
  }
  p.list = list;
  p.count = count;
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  const long long grid = units * most < 8 * sms ? units * most : 8 * sms;   // 8 CTAs an SM: 128 KB of loads under way
  return finish_launch(launch_pdl(paged_copy_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, s, p));
}

// offsets of the fork's parts of the workspace, from the front; .. + total
struct ForkPlan {
  size_t opens, list, copies, count, bytes;
};
static bool fork_plan(const swa_paged_fork_args* a, ForkPlan* w) {
  if (!pools_sizes_ok(a->pools) || a->B < 1 || a->B > 65535 || a->R < 1 || a->R > 65535) return false;
  if (a->page < 16 || a->page > 256 || (a->page & (a->page - 1))) return false;
  if (a->max_pages < 1 || a->max_pages > (1 << 30) / a->page) return false;
  if ((long long)a->B * a->max_pages >= (1LL << 31) || (long long)a->R * a->max_pages >= (1LL << 31)) return false;
  w->opens = up256s((size_t)a->B * 4);
  w->list = w->opens + up256s((size_t)a->pools.num_pages * 8);
  w->copies = w->list + up256s((size_t)a->pools.num_pages * 4);
  w->count = w->copies + up256s((size_t)a->R * 8);
  w->bytes = w->count + 256;
  return true;
}
struct CompactPlan {
  size_t copies, count, bytes;
};
static bool compact_plan(const swa_paged_compact_args* a, CompactPlan* w) {
  if (!pools_sizes_ok(a->pools) || a->B < 1 || a->B > 65535) return false;
  if (a->max_pages < 1 || a->max_pages > (1 << 26) || (long long)a->B * a->max_pages >= (1LL << 31)) return false;
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
  return a && fork_plan(a, &w) ? w.bytes : 0;
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
  if (!a->workspace || a->workspace_bytes < w.bytes) return SWA_E_WORKSPACE;
  s[n++] = {a->workspace, w.bytes};
  for (int i = 0; i < 4; ++i) s[n++] = words[i];
  const int written = n;
  for (int i = 4; i < 9; ++i)
    if (words[i].bytes && !(i == 4 && a->refs == a->refs_out)) s[n++] = words[i];
  if (!spans_apart(s, n, written)) return SWA_E_SHAPE;
  ForkParams p{};
  p.B = a->B; p.R = a->R; p.num_pages = a->pools.num_pages; p.max_pages = a->max_pages;
  while ((1 << p.page_shift) < a->page) ++p.page_shift;
  p.cap = a->max_pages << p.page_shift;
  p.table = a->table; p.lens = a->lens; p.parent = a->parent; p.room = a->room; p.refs = a->refs;
  p.table_out = a->table_out; p.lens_out = a->lens_out; p.refs_out = a->refs_out; p.left = a->left;
  char* ws = static_cast<char*>(a->workspace);
  p.children = reinterpret_cast<int*>(ws);
  p.opens = reinterpret_cast<int2*>(ws + w.opens);
  p.free_list = reinterpret_cast<int*>(ws + w.list);
  p.copies = reinterpret_cast<int2*>(ws + w.copies);
  p.count = reinterpret_cast<int*>(ws + w.count);
  p.err = a->err;
  const int st = finish_launch(launch_pdl(paged_fork_kernel, dim3(kPCtas), dim3(kPThreads), 0, stream, p));
  return st != SWA_OK ? st : launch_copies(a->pools, p.copies, p.count, a->R, stream);
}

size_t swa_paged_compact_workspace_size(const swa_paged_compact_args* a) {
  CompactPlan w;
  return a && compact_plan(a, &w) ? w.bytes : 0;
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
  if (!a->workspace || a->workspace_bytes < w.bytes) return SWA_E_WORKSPACE;
  s[n++] = {a->workspace, w.bytes};
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
  char* ws = static_cast<char*>(a->workspace);
  p.refs_moved = reinterpret_cast<int*>(ws);
  p.copies = reinterpret_cast<int2*>(ws + w.copies);
  p.count = reinterpret_cast<int*>(ws + w.count);
  p.err = a->err;
  const int st = finish_launch(launch_pdl(paged_compact_kernel, dim3(kPCtas), dim3(kPThreads), 0, stream, p));
  return st != SWA_OK ? st : launch_copies(a->pools, p.copies, p.count, (p.num_pages + 1) / 2, stream);
}

}  // extern "C"
