// The attention weight each cached key received from a chunk's rows (swa_paged_weigh).
//
// w_j += sum over query vectors i of 2^(qmul <q_i, k_j> - lse_i log2 e): with lse known
// every weight stands alone, so this is one matrix product with an exponential and a row
// sum as its epilogue, S^T = K Q^T: 128 keys (M, A operand) by up to QN query vectors (N, B
// operand). A thread then owns a key: the sum over its row of S^T needs no exchange.
// Bytes: K once (few rows: bound by that); operations: 2 hd and one exponential a pair, at
// hd 128 both 512 clk an SM for 128 x 128 pairs (8192 operations and 32 exponentials a clk).
//
// One CTA an SM. The units (sequence, KV head, 256 keys), each with its cost (tile_cost), are
// laid end to end and cut evenly. Roles: warp 8 streams K tiles of 128
// keys from the pages by TMA; warp 11 brings the query tiles (whole ones by TMA, else cp.async
// into the same swizzled layout, with each vector's lse and limit; the summing warps a pair
// that stays); warps 9 and 10 issue the products, two
// S buffers in TMEM for each half of a unit; a warpgroup (warps 0-3, 4-7) sums each half, so
// that a query tile serves 256 keys and nothing is exchanged. A sequence of at most two
// query tiles keeps them in shared memory for all its keys, else they are streamed per
// unit. The sums run in a fixed order: no atomics.
// Measured: one token of 64 sequences of 2048 to 4160 keys, 16 query heads on 4, hd 128: 37 us,
// 5.5 TB/s of K and weights. The last 32 to 64 rows of four prompts of 16384 to 32768 keys, 32
// heads on 8: 46.7 us (4.0 TB/s, 705 TFLOP/s). Of a CTA's 80 thousand clk, stamped: 13.7 until its
// first S (4.5 its share, 1.6 to the first K asked for, 7.6 that K and the pair of query tiles), then
// 36 tiles: 48.3 the sums (1700 for 128 columns, both warpgroups at once, 1024 of them exponentials
// at the special functions' rate), 5.2 the waits for S, 12.7 the turns between (weights stored, the
// next unit found); K is hardly waited for (2.8, under the sums). ncu: special functions and tensor
// pipe 28 % each, issue 37 %. Of one token's 65 thousand clk 28.8 wait for K. Tried: four warpgroups
// of sums (54 us when this took 51), K called into L2 ahead (54 for 51), the next 32 columns of S
// loaded while 32 are summed (53 for 51: S is freed later), 128 columns in registers (61: spills), a
// key of each half a thread over half of the columns, with one lse for both (51 for 46). All rows of
// prompts of 2048 rows over 4096 to 8192 keys, four of them, 32 heads on 8, hd 128: 327 us, 848
// TFLOP/s; 8 of 512 rows, 32 heads on 4, hd 64: 180 us, 445 TFLOP/s.
#include <cmath>

#include "swa_paged_tc.cuh"

namespace swa {

template <int D>
struct WeighCfg {
  static constexpr int QN = D == 256 ? 64 : 128;       // most query vectors of a tile (tile_vecs)
  // K slots of 128 keys, half of them for each half of a unit: a wait sees only the parity
  // of a barrier's phase, so whoever waits on a slot has to wait for each of its uses
  static constexpr int NS = D == 64 ? 8 : D == 128 ? 4 : 2, NSH = NS / 2;
  static constexpr int KB = 128 * D * 2;               // bytes of a K tile
  static constexpr int QB = QN * D * 2;
  static constexpr int SMEM = NS * KB + 2 * QB + 1024;
};
constexpr int kWeighThreads = 384;
constexpr int kUnit = 256;     // keys of a unit
// Cost of a unit in the time of 32 query columns (about 250 clk): two query tiles' worth of
// fixed work at least, and a query tile costs its columns and one more. kUnitCost covers the
// columns that the last query tile may lack, so that every unit costs something.
constexpr int kUnitCost = 5;
constexpr int kNote = 4;       // query tiles whose lse and limits are in shared memory

// x / d for 0 <= x < 2^31: shift = 31 + l with 2^l >= d and mul = ceil(2^shift / d) <= 2^32: the
// product's excess is below x * 2^l < 2^shift, so the quotient is exact.
struct Quot {
  uint32_t mul, shift;
  explicit Quot(int d = 2) : mul(0), shift(31) {
    while ((1 << (shift - 31)) < d) ++shift;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int x) const { return (int)((unsigned long long)(unsigned)x * mul >> shift); }
};

struct PagedWeighParams {
  PagedMap map;
  int T, nh, hpg, max_rows;
  Quot by_hpg, by_rows;        // vec / hpg: a vector's row; row / tile_rows: a row's tile
  // A query tile is as many whole rows as fit in QN vectors: tile_rows rows of hpg vectors
  int tile_rows, tile_vecs;
  float qmul;
  const void* q;
  long long q_row;
  int bulk_q;                  // map_q brings whole query tiles
  const float* lse;
  const float* weight;
  float* out;
  uint32_t* err;
};

__device__ __forceinline__ int row_of(const PagedWeighParams& p, int vec) { return p.by_hpg(vec); }

// A sequence's units of a KV head ("tiles" of kUnit keys) and the query tiles that see them.
struct WeighSeq {
  PagedSeq s;
  int nv, nqt, n_tiles, n_full;   // query vectors, query tiles, key tiles, key tiles seen by every query tile
  int base;                       // cost of a unit besides its query tiles
};
template <int QN>
__device__ __forceinline__ WeighSeq weigh_seq(const PagedWeighParams& p, int b, uint32_t& bits) {
  WeighSeq w;
  w.s = paged_seq(p.map, b, p.T, p.max_rows, bits);
  w.nv = w.s.t * p.hpg;
  w.nqt = w.s.t > 0 ? p.by_rows(w.s.t - 1) + 1 : 0;
  w.n_tiles = (w.s.len + kUnit - 1) / kUnit;
  w.n_full = w.nqt <= 1 ? w.n_tiles : w.s.len >= w.s.t ? min(w.n_tiles, (w.s.len - w.s.t) / kUnit + 1) : 0;
  w.base = kUnitCost - (w.nqt > 0 ? (w.nqt * p.tile_vecs - w.nv) / 32 : 0);   // the last query tile's missing columns
  return w;
}
// First query tile that sees keys of tile `tile`: its last row has a limit above the tile's
// first key, rows from (first key - (len - t)) on.
template <int QN>
__device__ __forceinline__ int first_qt(const PagedWeighParams& p, const WeighSeq& w, int tile) {
  const long long row = (long long)tile * kUnit - (w.s.len - w.s.t);
  return row <= 0 ? 0 : row < w.s.t ? p.by_rows((int)row) : w.nqt;
}
template <int QN>
__device__ __forceinline__ int tile_cost(const PagedWeighParams& p, const WeighSeq& w, int tile) {
  return w.base + (w.nqt - first_qt<QN>(p, w, tile)) * (QN / 32 + 1);
}
template <int QN>
__device__ __forceinline__ long long head_cost(const PagedWeighParams& p, const WeighSeq& w) {
  long long c = (long long)w.n_full * (w.base + w.nqt * (QN / 32 + 1));
  for (int i = w.n_full; i < w.n_tiles; ++i) c += tile_cost<QN>(p, w, i);
  return c;
}

// Walks this CTA's units; every role keeps its own.
template <int QN>
struct WeighIter {
  const PagedWeighParams& p;
  WeighSeq w;
  int b, g, tile;
  long long left;              // cost still to take
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ int qt0() const { return first_qt<QN>(p, w, tile); }
  __device__ __forceinline__ bool resident() const { return w.nqt <= 2; }
  __device__ __forceinline__ int halves() const { return tile * kUnit + 128 < w.s.len ? 2 : 1; }
  // the next unit; true when it belongs to another (sequence, KV head) (or there is none)
  __device__ __forceinline__ bool next() {
    left -= tile_cost<QN>(p, w, tile);
    if (++tile < w.n_tiles) return left <= 0;
    tile = 0;
    if (left <= 0) return true;
    if (++g == p.map.nk) {
      g = 0;
      uint32_t ignore = 0;
      do w = weigh_seq<QN>(p, ++b, ignore);
      while (w.n_tiles == 0);
    }
    return true;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWeighThreads, 1)
    paged_weigh_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ PagedWeighParams p) {
  using C = WeighCfg<D>;
  constexpr int QN = C::QN, NS = C::NS, NSH = C::NSH, CH = D / 8;
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char sm_raw[];
  // tests/test_paged_barriers_cpu.py runs the roles below on a model of these barriers: what waits
  // or arrives here has to be changed there too
  __shared__ __align__(8) uint64_t b_kfull[NS], b_kempty[NS], b_qfull[2], b_qempty[2], b_s[4], b_sfree[4], b_fin[2];
  // lse and limits have a ring of their own: a query tile's slot is free once its products are
  // done, while they are needed until its sums are
  __shared__ __align__(8) uint64_t b_nfull[kNote], b_nempty[kNote], b_pair;
  __shared__ __align__(16) float s_nlse[kNote][QN];             // -lse log2 e
  __shared__ __align__(16) int s_lim[kNote][QN];
  __shared__ long long s_scan[kWeighThreads / 32];
  __shared__ long long s_left;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_b, s_g, s_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  unsigned char* const sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* const sm_q = sm + NS * C::KB;
  // what needs no global memory, before the wait for the kernel in front
  if (warp == 8 && lane == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&b_kfull[i], 1);
      mbar_init(&b_kempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b_qfull[i], 1);
      mbar_init(&b_qempty[i], 2);
      mbar_init(&b_fin[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b_s[i], 1);
      mbar_init(&b_sfree[i], 4);
    }
    for (int i = 0; i < kNote; ++i) {
      mbar_init(&b_nfull[i], 1);
      mbar_init(&b_nempty[i], 8);
    }
    mbar_init(&b_pair, 1);
    mbar_fence_init();
    s_b = -1;
    s_abort = 0;
  }
  // rows of the query slots behind tile_vecs are read and never brought: zeros
  for (int i = tid; i < 2 * (QN - p.tile_vecs) * CH; i += kWeighThreads) {
    const int c = i % CH, r = p.tile_vecs + i / CH % (QN - p.tile_vecs), slot = i / CH / (QN - p.tile_vecs);
    *reinterpret_cast<uint4*>(sm_q + slot * C::QB + (c >> 3) * (QN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  pdl_wait();
  pdl_trigger();
  // Not before the wait: a CTA that held TMEM while it waits for the kernel in front could keep
  // it from that kernel's CTA on the same SM, which may still have its own to allocate.
  if (warp == 9) tc_alloc(&s_tmem, 512);

  // --- this CTA's share: units whose start lies in [u0, u1) of the summed costs
  {
    uint32_t bits = 0;
    const int E = (p.map.B + kWeighThreads - 1) / kWeighThreads;
    long long mine = 0;
    for (int e = 0; e < E; ++e) {
      const int b = tid * E + e;
      if (b < p.map.B) mine += p.map.nk * head_cost<QN>(p, weigh_seq<QN>(p, b, bits));
    }
    if (bits && blockIdx.x == 0) set_err(p.err, bits);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < kWeighThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long u0 = per * blockIdx.x, u1 = min(total, u0 + per);
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
      // the first unit that starts at or after u0
      long long at = before;
      uint32_t ignore = 0;
      int found = 0;
      for (int e = 0; e < E && !found; ++e) {
        const int b = tid * E + e;
        if (b >= p.map.B) break;
        const WeighSeq w = weigh_seq<QN>(p, b, ignore);
        const long long hc = head_cost<QN>(p, w);
        if (hc == 0 || at + hc * p.map.nk <= u0) {
          at += hc * p.map.nk;
          continue;
        }
        int g = at >= u0 ? 0 : (int)((u0 - at) / hc);
        at += hc * g;
        const int full = w.base + w.nqt * (QN / 32 + 1);
        int tile = at >= u0 ? 0 : (int)min((long long)w.n_full, (u0 - at + full - 1) / full);
        at += (long long)tile * full;
        while (tile < w.n_tiles && at < u0) at += tile_cost<QN>(p, w, tile++);
        if (tile == w.n_tiles) {            // the head's units all start before u0: the next head's first
          tile = 0;
          if (++g == p.map.nk) continue;    // or the next sequence's (at stands at its start)
        }
        found = 1;
        if (at < u1) {
          s_b = b;
          s_g = g;
          s_tile = tile;
          s_left = u1 - at;
        }
      }
      if (!found && at < u1) {
        // the next sequence with keys belongs to a later thread's share
        for (int b = tid * E + E; b < p.map.B; ++b) {
          if (weigh_seq<QN>(p, b, ignore).n_tiles > 0) {
            s_b = b;
            s_g = 0;
            s_tile = 0;
            s_left = u1 - at;
            break;
          }
        }
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  if (s_b < 0) {
    if (warp == 9) {
      tc_fence_after();
      tc_dealloc(s_tmem, 512);
    }
    return;
  }
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  auto give_up = [&]() {
    s_abort = 1;
    __threadfence_block();
    set_err(p.err, SWA_DERR_TIMEOUT);
  };
  // every wait is made by whole warps and has one outcome for the warp
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    return __all_sync(0xffffffffu, tc_wait(bar, (uint32_t)(phase & 1), &s_abort));
  };
  uint32_t ignore = 0;
  WeighIter<QN> it{p, weigh_seq<QN>(p, s_b, ignore), s_b, s_g, s_tile, s_left};
  bool ok = true;
  // Columns of query tile qt's product: its vectors, up to a multiple of 32
  auto columns_of = [&](int qt) {
    return min(QN, (min(p.tile_vecs, it.w.nv - qt * p.tile_vecs) + 31) & ~31);   // QN: known to the compiler
  };
  // Query tile qt's copy into a slot, by NTH threads: 16-byte chunks, CH a row, swizzled; zeros
  // behind its vectors. The row and head of a vector run along (a division a chunk: 270 instead
  // of 192 us, when this copied all tiles, for four prompts of 512 rows over 4096 to 8192 keys, 24 heads on 8, hd 128).
  auto copy_q = [&](int qt, int slot, int th, auto threads) {
    constexpr int STEP = decltype(threads)::value / CH;
    const int n = columns_of(qt), c = th % CH, end = min(it.w.nv, (qt + 1) * p.tile_vecs);
    const uint32_t dst = smem_u32(sm_q + slot * C::QB) + (c >> 3) * (QN * 128);
    const int di = STEP / p.hpg, dh = STEP - di * p.hpg;
    int vec = qt * p.tile_vecs + th / CH, h = vec - row_of(p, vec) * p.hpg;
    const long long ds = di * p.q_row + dh * D, dw = p.q_row - p.hpg * D;
    const T* src = static_cast<const T*>(p.q) + (size_t)(it.w.s.r0 + row_of(p, vec)) * p.q_row + (size_t)(it.g * p.hpg + h) * D + c * 8;
#pragma unroll 4
    for (int r = th / CH; r < n; r += STEP) {
      const bool in = vec < end;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   :: "r"(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)), "l"(in ? src : static_cast<const T*>(p.q)), "r"(in ? 16 : 0)
                   : "memory");
      vec += STEP;
      h += dh;
      src += ds;
      if (h >= p.hpg) {
        h -= p.hpg;
        src += dw;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // lse of vector v of query tile qt (infinite, for a weight of 0, where there is none); its limit
  auto vec_of = [&](int qt, int v) { return v < p.tile_vecs ? qt * p.tile_vecs + v : 0x7fffffff; };
  auto lse_of = [&](int vec) {
    if (vec >= it.w.nv) return INFINITY;
    const int i = row_of(p, vec);
    return p.lse[(size_t)(it.w.s.r0 + i) * p.nh + it.g * p.hpg + vec - i * p.hpg];
  };
  auto note_q = [&](int slot, int v, int vec, float lse) {
    s_nlse[slot][v] = lse * -1.4426950408889634f;
    s_lim[slot][v] = vec < it.w.nv ? min(it.w.s.len, it.w.s.len - it.w.s.t + row_of(p, vec) + 1) : 0;
  };

  // A pair of query tiles that a head keeps is brought by the summing warps: it needs both slots,
  // so it cannot come ahead of its use, and one warp takes 5 us for it (50.6 instead of 45.7 us
  // for the prompts above). Others come ahead, by warp 11.
  auto pair = [&]() { return it.resident() && it.w.nqt - it.qt0() == 2; };

  if (warp < 8) {
    // ------------------------------------------------------------ sums: thread = key
    const int h = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h * 2 * QN;
    const uint64_t mul2 = pack64(__float_as_uint(p.qmul), __float_as_uint(p.qmul));
    int jc = 0, qc = 0, q_base = it.qt0(), q_seen = 0;      // q_seen: query tiles known to be there
    int pairs = 0;
    auto fill = [&]() {                     // once warp 11 has seen that the slots are free
      if (!pair()) return;
      const int q0 = it.qt0();
      const int mt = tid / QN, mv = tid % QN, vec = vec_of(q0 + mt, mv);
      const float lse = mt < 2 ? lse_of(vec) : 0.f;
      ok &= tc_wait(&b_pair, (uint32_t)(pairs++ & 1), &s_abort);
      for (int k = 0; k < 2; ++k) copy_q(q0 + k, (qc + k) & 1, tid, Int<256>{});
      if (mt < 2) note_q((qc + mt) % kNote, mv, vec, lse);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      named_barrier(1, 256);
      if (tid == 0)
        for (int k = 0; k < 2; ++k) {
          mbar_arrive(&b_qfull[(qc + k) & 1]);
          mbar_arrive(&b_nfull[(qc + k) % kNote]);
        }
    };
    fill();
    while (!it.done()) {
      const int nqt = it.w.nqt, key = it.tile * kUnit + h * 128 + r;
      const bool res = it.resident(), here = h < it.halves();
      const size_t at = ((size_t)it.b * p.map.nk + it.g) * p.map.cap + key;
      const bool mine = key < it.w.s.len;
      const float w0 = mine && p.weight ? p.weight[at] : 0.f;   // under way during the products
      uint64_t sum[4] = {0, 0, 0, 0};
      for (int qt = it.qt0(); qt < nqt; ++qt) {
        const int qi = res ? qc + qt - q_base : qc, buf = jc & 1, slot = qi % kNote;
        // lse and limits; a thread whose wait gave up goes on (its warp stays together) and
        // writes nothing
        if (qi >= q_seen) {
          ok &= tc_wait(&b_nfull[slot], (uint32_t)((qi / kNote) & 1), &s_abort);
          q_seen = qi + 1;
        }
        if (here) {
          ok &= tc_wait(&b_s[2 * h + buf], (uint32_t)((jc >> 1) & 1), &s_abort);
          tc_fence_after();
          const int n = columns_of(qt);
          // columns [c, c + W): weights into the sums
          auto columns = [&](int c, auto width, auto masked) {
            constexpr int W = decltype(width)::value;
            uint32_t x[W / 32][32];
#pragma unroll
            for (int i = 0; i < W / 32; ++i) tc_ld32(lanes + buf * QN + c + i * 32, x[i]);
            wait_ld(x);
            if (c + W >= n) {               // S is in registers: the buffer is free
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&b_sfree[2 * h + buf]);
            }
            // 16 columns at a time: first their scaled scores, then their exponentials
#pragma unroll
            for (int k = 0; k < W; k += 16) {
              float e[16];
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const ulonglong2 l2 = *reinterpret_cast<const ulonglong2*>(&s_nlse[slot][c + k + i]);
                const uint32_t* y = &x[(k + i) >> 5][(k + i) & 31];
                unpack64(fma2(pack64(y[0], y[1]), mul2, l2.x), e[i], e[i + 1]);
                unpack64(fma2(pack64(y[2], y[3]), mul2, l2.y), e[i + 2], e[i + 3]);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) e[i] = ex2(e[i]);
              if constexpr (decltype(masked)::value) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                  const int4 lm = *reinterpret_cast<const int4*>(&s_lim[slot][c + k + i]);
                  e[i] = key < lm.x ? e[i] : 0.f;
                  e[i + 1] = key < lm.y ? e[i + 1] : 0.f;
                  e[i + 2] = key < lm.z ? e[i + 2] : 0.f;
                  e[i + 3] = key < lm.w ? e[i + 3] : 0.f;
                }
              }
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], pack64(__float_as_uint(e[i]), __float_as_uint(e[i + 1])));
            }
          };
          // some row of the tile does not see all keys of this half
          const bool mask =
              it.tile * kUnit + h * 128 + 128 >
              it.w.s.len - it.w.s.t + qt * p.tile_rows + 1;
          for (int c = 0; c < n; c += 64) {
            if (mask) {
              columns(c, Int<32>{}, std::true_type{});
              if (c + 32 < n) columns(c + 32, Int<32>{}, std::true_type{});
            } else if (c + 32 < n) {
              columns(c, Int<64>{}, std::false_type{});
            } else {
              columns(c, Int<32>{}, std::false_type{});
            }
          }
          ++jc;
        }
        if (!res) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_nempty[slot]);
          ++qc;
        }
      }
      float a0, a1;
      unpack64(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a0, a1);
      if (mine && ok) p.out[at] = w0 + (a0 + a1);
      const bool moved = it.next();
      if (moved && res) {
        __syncwarp();
        if (lane == 0)
          for (int i = q_base; i < nqt; ++i) mbar_arrive(&b_nempty[(qc + i - q_base) % kNote]);
        qc += nqt - q_base;
      }
      if (moved && !it.done()) {
        q_base = it.qt0();
        fill();
      }
    }
    if (!ok) give_up();
  } else if (warp == 8) {
    // ------------------------------------------------------------ K tiles
    const int page = 1 << p.map.page_shift, rows = min(page, 128), per_half = 128 / rows;
    const int oob = p.map.num_pages * p.map.nk << p.map.page_shift;       // rows of the pool: reads zeros
    int kc[2] = {0, 0};                     // tiles started of each half
    for (; ok && !it.done(); it.next()) {
      if (it.qt0() >= it.w.nqt) continue;
      const int32_t* table = p.map.table + (size_t)it.b * p.map.max_pages;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!ok || h >= it.halves()) continue;
        const int slot = h * NSH + kc[h] % NSH, use = kc[h] / NSH;
        // lane bx looks up box bx of each half of the features (8 at most), before the wait
        const int key = it.tile * kUnit + h * 128 + lane * rows;
        int y = oob;
        if (lane < per_half && key < it.w.s.len) {
          const int id = table[key >> p.map.page_shift];
          if (page_ok(p.map, id))
            y = ((id * p.map.nk + it.g) << p.map.page_shift) + (key & (page - 1));
          else
            set_err(p.err, SWA_DERR_PAGE);
        }
        ok = use == 0 || wait(&b_kempty[slot], use - 1);
        if (!ok) continue;
        if (lane == 0) mbar_arrive_expect_tx(&b_kfull[slot], C::KB);
        __syncwarp();
        if (lane < per_half)
#pragma unroll
          for (int half = 0; half < D / 64; ++half)
            tma_2d(smem_u32(sm + slot * C::KB + half * (128 * 128) + lane * rows * 128), &map_k, half * 64, y, &b_kfull[slot]);
        ++kc[h];
      }
    }
    // commits arrive at their barriers on their own time: the last ones must have done so
    // before the CTA (and its shared memory) goes
    for (int h = 0; h < 2; ++h)
      for (int u = max(0, kc[h] - NSH); ok && u < kc[h]; ++u) ok = wait(&b_kempty[h * NSH + u % NSH], u / NSH);
    if (!ok) {
      give_up();
      // copies in flight land before the CTA exits (bounded)
      for (int h = 0; h < 2; ++h)
        for (int u = max(0, kc[h] - NSH); u < kc[h]; ++u)
          mbar_wait_bounded(&b_kfull[h * NSH + u % NSH], (uint32_t)((u / NSH) & 1), kWaitLimitNs);
    }
  } else if (warp <= 10) {
    // ------------------------------------------------------------ products, a warp a half
    // Waits, issue and commits take a warp about as long as the sums take a warpgroup.
    // A wait that gave up leaves ok false and the role goes on to its end (no votes): what
    // follows only touches this CTA's own shared memory and TMEM, and nothing is written.
    const int h = warp - 9;
    const bool leader = elect_one();
    const uint64_t k_desc = sw128_desc(smem_u32(sm), 16), q_desc = sw128_desc(smem_u32(sm_q), 16);
    auto until = [&](uint64_t* bar, int phase) { ok &= tc_wait(bar, (uint32_t)(phase & 1), &s_abort); };
    int kc = 0, jc = 0, qc = 0, q_seen = 0; // this half's K tiles and products, query tiles loaded, known to be there
    int q_base = it.qt0();                  // first query tile kept of a resident head
    while (!it.done()) {
      const int nqt = it.w.nqt, nh = it.halves(), q_first = it.qt0();
      const bool res = it.resident();
      for (int qt = q_first; qt < nqt; ++qt) {
        const int qi = res ? qc + qt - q_base : qc;
        if (qi >= q_seen) {
          until(&b_qfull[qi & 1], qi >> 1);
          q_seen = qi + 1;
        }
        if (h < nh) {
          const int slot = h * NSH + kc % NSH, buf = 2 * h + (jc & 1);
          if (qt == q_first) until(&b_kfull[slot], kc / NSH);
          if (jc >= 2) until(&b_sfree[buf], (jc >> 1) - 1);
          tc_fence_after();
          if (leader) {
            const int n = columns_of(qt);
            const uint32_t id = tc_idesc_16(BF, false, n);
            const uint64_t kd = k_desc + (uint64_t)((slot * C::KB) >> 4), qd = q_desc + (uint64_t)(((qi & 1) * C::QB) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tmem + buf * QN, kd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                     qd + (((k >> 2) * (QN * 128) + (k & 3) * 32) >> 4), id, k > 0);
            tc_commit(&b_s[buf]);
            if (qt == nqt - 1) tc_commit(&b_kempty[slot]);
          }
          __syncwarp();
          ++jc;
        }
        if (!res) {
          if (leader) tc_commit(&b_qempty[qi & 1]);
          __syncwarp();
          ++qc;
        }
      }
      if (q_first < nqt && h < nh) ++kc;
      const bool moved = it.next();
      if (moved && res) {
        if (leader)
          for (int i = q_base; i < nqt; ++i) tc_commit(&b_qempty[(qc + i - q_base) & 1]);
        __syncwarp();
        qc += nqt - q_base;
      }
      if (moved && !it.done()) q_base = it.qt0();
    }
    // what was issued, commits among it, finishes before TMEM and shared memory go (bounded)
    if (leader) tc_commit(&b_fin[h]);
    ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&b_fin[h], 0, kWaitLimitNs));
    if (!ok) give_up();
  } else if (warp == 11) {
    // ------------------------------------------------------------ query tiles
    int qc = 0, pending = -1;               // tiles started, the one whose arrival is still to be told
    auto tell = [&](bool all) {
      if (pending < 0) return;
      if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
      else asm volatile("cp.async.wait_group 1;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_qfull[pending & 1]);
      pending = -1;
    };
    // phase `use - 1` of a slot's empty barrier; a tile under way is told before a long wait
    auto until_free = [&](uint64_t* bar, int use) {
      if (use == 0 || __all_sync(0xffffffffu, mbar_try_wait(bar, (uint32_t)((use - 1) & 1)))) return true;
      tell(true);
      return wait(bar, use - 1);
    };
    auto load = [&](int qt) {
      const int slot = qc & 1, note = qc % kNote;
      constexpr int LR = QN / 32;
      float lse[LR];
#pragma unroll
      for (int k = 0; k < LR; ++k) lse[k] = lse_of(vec_of(qt, lane + k * 32));   // on its way during the waits
      // whole tiles come by TMA: boxes of 64 features, hpg heads and tile_rows rows (1258 instead
      // of 375 us for four prompts of 2048 rows over 4096 to 8192 keys, when a warp copied them)
      const bool bulk = p.bulk_q && (qt + 1) * p.tile_rows <= it.w.s.t;
      if (!until_free(&b_qempty[slot], qc >> 1)) return false;
      if (bulk) {
        tell(true);
        if (lane == 0) mbar_arrive_expect_tx(&b_qfull[slot], p.tile_vecs * D * 2);
        __syncwarp();
        if (lane < D / 64)
          tma_3d(smem_u32(sm_q + slot * C::QB + lane * (QN * 128)), &map_q, lane * 64, it.g * p.hpg,
                 it.w.s.r0 + qt * p.tile_rows, &b_qfull[slot]);
      } else {
        copy_q(qt, slot, lane, Int<32>{});
        tell(false);
        pending = qc;
      }
      const int q = qc++;
      if (!until_free(&b_nempty[note], q / kNote)) return false;
#pragma unroll
      for (int k = 0; k < LR; ++k) note_q(note, lane + k * 32, vec_of(qt, lane + k * 32), lse[k]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_nfull[note]);
      return true;
    };
    // both slots of a pair are free: told to the summing warps
    auto give_pair = [&]() {
      tell(true);
      for (int q = qc; q < qc + 2; ++q)
        if (!until_free(&b_qempty[q & 1], q >> 1) || !until_free(&b_nempty[q % kNote], q / kNote)) return false;
      if (lane == 0) mbar_arrive(&b_pair);
      __syncwarp();
      qc += 2;
      return true;
    };
    bool fresh = true;
    while (ok && !it.done()) {
      if (it.resident()) {
        // the head's later key tiles need no query tile that its first one here does not
        if (fresh && pair()) {
          ok = give_pair();
        } else if (fresh) {
          for (int qt = it.qt0(); ok && qt < it.w.nqt; ++qt) ok = load(qt);
          tell(true);                       // the next load may be far away
        }
      } else {
        for (int qt = it.qt0(); ok && qt < it.w.nqt; ++qt) ok = load(qt);
      }
      if (ok) fresh = it.next();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    tell(true);
    for (int q = max(0, qc - 2); ok && q < qc; ++q) ok = wait(&b_qempty[q & 1], q >> 1);   // as for K above
    if (!ok) {
      give_up();
      for (int q = max(0, qc - 2); q < qc; ++q) mbar_wait_bounded(&b_qfull[q & 1], (uint32_t)((q >> 1) & 1), kWaitLimitNs);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

template <typename T, int D>
static int launch_weigh(const swa_paged_weigh_args* a, const PagedWeighParams& params, cudaStream_t s) {
  CUtensorMap mk, mq;
  int rc = pool_map(a->cache, a->cache.k, 128, &mk);
  constexpr int QN = WeighCfg<D>::QN;
  PagedWeighParams p = params;
  p.tile_rows = QN / p.hpg;
  p.tile_vecs = p.tile_rows * p.hpg;
  p.by_hpg = Quot(p.hpg);
  p.by_rows = Quot(p.tile_rows);
  p.bulk_q = p.max_rows >= p.tile_rows && a->q_row < (1LL << 39);   // no such tile; strides below 2^40 bytes
  if (rc == SWA_OK && p.bulk_q) rc = rows_map(a->cache, a->q, a->T, a->nh, a->q_row, p.hpg, p.tile_rows, &mq);
  else mq = mk;
  if (rc != SWA_OK) return rc;
  const cudaError_t e = allow_smem<paged_weigh_kernel<T, D>>(WeighCfg<D>::SMEM);
  if (e != cudaSuccess) return cuda_status(e);
  return finish_launch(launch_pdl(paged_weigh_kernel<T, D>, dim3(num_sms() > 0 ? num_sms() : 148), dim3(kWeighThreads),
                                  WeighCfg<D>::SMEM, s, mk, mq, p));
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
  if ((long long)a->T * a->nh >= (1LL << 31) - 256) return SWA_E_SHAPE;   // query vectors and their tiles in 32 bits
  if (!(a->scale >= 0.f) || std::isinf(a->scale)) return SWA_E_SHAPE;
  const long long qn = a->T > 0 ? rows_span(a->T, (long long)a->nh * c.hd, a->q_row) : 0;
  if (qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->q) || (a->T > 0 && (a->q_row & 7)) || (reinterpret_cast<uintptr_t>(a->lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->weight) & 3u) || (reinterpret_cast<uintptr_t>(a->out) & 3u))
    return SWA_E_ALIGN;
  PagedWeighParams p{};
  p.map = paged_map(&c);
  const size_t bytes = (size_t)c.B * c.nk * p.map.cap * 4;
  if (a->weight && a->weight != a->out && bytes_overlap(a->weight, bytes, a->out, bytes)) return SWA_E_SHAPE;
  if (a->T > 0 && (bytes_overlap(a->q, (size_t)qn * 2, a->out, bytes) ||
                   bytes_overlap(a->lse, (size_t)a->T * a->nh * 4, a->out, bytes)))
    return SWA_E_SHAPE;
  p.T = a->T; p.nh = a->nh; p.hpg = a->nh / c.nk; p.max_rows = a->max_rows < a->T ? a->max_rows : a->T;
  p.qmul = a->scale * 1.4426950408889634f;
  p.q = a->q; p.q_row = a->q_row;
  p.lse = a->lse; p.weight = a->weight; p.out = a->out; p.err = a->err;
  if (c.dtype == SWA_BF16)
    return c.hd == 64 ? launch_weigh<__nv_bfloat16, 64>(a, p, stream)
                      : c.hd == 128 ? launch_weigh<__nv_bfloat16, 128>(a, p, stream) : launch_weigh<__nv_bfloat16, 256>(a, p, stream);
  return c.hd == 64 ? launch_weigh<__half, 64>(a, p, stream)
                    : c.hd == 128 ? launch_weigh<__half, 128>(a, p, stream) : launch_weigh<__half, 256>(a, p, stream);
}

}  // extern "C"
