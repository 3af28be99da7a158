// Attention of chunks with many query vectors per KV head over the paged cache, on the
// tensor cores (tcgen05, accumulators in TMEM, pages copied by TMA).
//
// Work item: NT tiles of 128 query vectors (rows x heads of one KV head) of one
// sequence. S = Q K^T and O += P V per tile of KT keys are both matrix products with
// 128 rows; between them stand 128 x KT exponentials. At hd 128 the two products take an SM's
// tensor core 4 * 128 * 128 * 128 / 8192 = 1024 clk, and the exponentials, at 32 a clk, half of
// that. One tile's chain of S, softmax and P V would leave the tensor core idle for as long as the
// softmax takes, so something else has to run under it:
//   - hd 64 and 128: two tiles (NT = 2), each with its own softmax warpgroup and its
//     own issuing warp, share every K and V tile; while one tile is in its softmax the
//     tensor core works for the other. TMEM: S 2 x 128 and O 2 x hd columns.
//   - hd 256: O of two tiles would fill TMEM, so there is one tile, and S has two
//     buffers: the product of the next keys runs during this softmax (KT = 64, so that
//     Q and five slots of K / V fit in shared memory).
// P overwrites its S columns as 16-bit pairs and is read from TMEM as the A operand.
// One thread owns one row of S: maxima and sums need no exchange. The running maximum
// is raised only when a row's scores pass it by 2^kLazy (weights then stay below
// 2^kLazy times the scale), so that O is seldom rescaled.
// V of keys behind the sequence's last one is zeroed in shared memory (0 * NaN).
// Few items are split over the keys: grid.y shares of an item's tiles leave records
// that chunk_merge_kernel joins.
// Measured: four sequences of 2048 rows behind 6144 keys, 32 query heads on 8, hd 128, bf16:
// 646 us, 1490 TFLOP/s; ragged ones of 1024 to 2048 rows over 2048 to 16384 keys: 523 us,
// 1410 TFLOP/s (ncu: tensor pipe 64 %, special functions 32 %, issue 37 %). What is left is the chain
// S -> softmax -> P V -> S of a tile: about 330 clk from the last product issued to the
// barrier seen, twice a step, and P V before the S that overwrites P. Four of 1024 to 2048 rows over
// 8192 keys: hd 64 880 TFLOP/s, the same chain for half the products; hd 256 1180, every 128 query
// vectors read K and V.
// The weights are rounded to T once, which with T's own rounding of the result makes it 1.35 times as
// inexact as 32-bit weights would (bf16: 0.0023 and 0.0017 of its norm). What the rounding leaves
// would take a second P V, half as many products again.
#include <cmath>

#include "swa_paged_tc.cuh"

namespace swa {

template <int D>
struct ChunkCfg {
  static constexpr int NT = D == 256 ? 1 : 2;          // query tiles of an item
  static constexpr int SB = D == 256 ? 2 : 1;          // S buffers of a tile
  static constexpr int KT = D == 256 ? 64 : 128;       // keys of a tile
  static constexpr int NS = D == 64 ? 8 : 5;           // K / V slots
  static constexpr int SLOT = KT * D * 2;
  static constexpr int QB = 128 * D * 2;               // bytes of a query tile
  static constexpr int THREADS = NT * 128 + 128;       // softmax warpgroups; loader, issuers, idle warps
  static constexpr int SMEM = NT * QB + NS * SLOT + 1024;   // + alignment
  // Registers a thread: at launch, and after they moved over to the softmax threads (two tiles).
  // They move inside what the CTA was launched with: shares that are more than that wait for ever.
  static constexpr int REGS = NT == 2 ? 168 : 0, R_SOFT = 216, R_REST = 72;
  static_assert(NT == 1 || NT * 128 * R_SOFT + 128 * R_REST <= THREADS * REGS, "registers of a CTA");
  static constexpr int C_O = NT * SB * KT;             // first O column
};
constexpr int kSortSeqs = 64;            // sequences of a call up to which they are taken longest first
template <typename T>
struct LazyMax {                                       // log2 of what a weight may exceed its scale by
  static constexpr float kLazy = 8.f, kLog2 = 0.f;
};
template <>
struct LazyMax<__half> {   // 2^(4 + 11) = 2^15 < 65504; a weight loses 2^-25 / 2^11 of the largest at most; see PScale
  static constexpr float kLazy = 4.f, kLog2 = 11.f;
};

struct ChunkParams {
  PagedAttendParams a;
  int small;                   // sequences with at most this many query vectors are not ours
  int tile_tok;                // chunk rows of a query tile (128 / hpg)
  int splits;
  float* rec_acc;              // [item][split][NT * 128][D]
  float2* rec_ml;              // [item][split][NT * 128]
  int4* rec_desc;              // [item]: (b, g, first row of the item, 0), b < 0: no such item
};

// First K / V slot position of tile j's K and V in the order they are consumed.
template <int SB>
__device__ __forceinline__ int pos_k(int j) { return SB == 1 ? 2 * j : (j == 0 ? 0 : 2 * j - 1); }
template <int SB>
__device__ __forceinline__ int pos_v(int j, int n) { return SB == 1 ? 2 * j + 1 : (j < n - 1 ? 2 * j + 2 : 2 * n - 1); }

__device__ __forceinline__ int chunk_items(const PagedSeq& s, const ChunkParams& p, int item_tok) {
  return (long long)s.t * p.a.hpg > p.small ? (s.t + item_tok - 1) / item_tok * p.a.map.nk : 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(ChunkCfg<D>::THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const ChunkParams p) {
  using C = ChunkCfg<D>;
  constexpr int NT = C::NT, SB = C::SB, KT = C::KT, NS = C::NS;
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char sm_raw[];
  // tests/test_paged_barriers_cpu.py runs the roles below on a model of these barriers: what waits
  // or arrives here has to be changed there too
  __shared__ __align__(8) uint64_t b_full[NS], b_empty[NS], b_q[NT], b_s[NT * SB], b_p[NT * SB][2], b_pv[NT], b_fin[NT], b_turn[NT], b_tail;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_b, s_idx;
  __shared__ int s_scan[32];
  __shared__ int2 s_seq[kSortSeqs];        // (keys, items) of each sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  constexpr int W_LOAD = NT * 4, W_MMA = NT * 4 + 1;
  unsigned char* const sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* const sm_kv = sm + NT * C::QB;
  const PagedAttendParams& a = p.a;
  // what needs no global memory, before the wait for the kernel in front
  if (warp == W_LOAD) {
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&b_full[i], 1);
        mbar_init(&b_empty[i], NT);
      }
      for (int t = 0; t < NT; ++t) {
        mbar_init(&b_q[t], 128);
        mbar_init(&b_pv[t], 1);
        mbar_init(&b_fin[t], 1);
        mbar_init(&b_turn[t], 1);
      }
      for (int i = 0; i < NT * SB; ++i) {
        mbar_init(&b_s[i], 1);
        mbar_init(&b_p[i][0], 128);
        mbar_init(&b_p[i][1], 128);
      }
      mbar_init(&b_tail, 1);
      mbar_fence_init();
    }
  }
  if (tid == 0) {
    s_b = -1;
    s_abort = 0;
  }
  pdl_wait();
  pdl_trigger();
  // Not before the wait: a CTA that held TMEM while it waits for the kernel in front could keep
  // it from that kernel's CTA on the same SM, which may still have its own to allocate.
  if (warp == W_MMA) tc_alloc(&s_tmem, 512);

  // --- which item. CTAs start in the order of their numbers, so the longest sequences'
  // items come first and the SMs end together (the ragged prompts above: 579 us in the order
  // of the batch when this took 550). Every thread adds up the items in front of
  // its sequence's, which is quick for few sequences; many are taken as they come, by a scan.
  const int item_tok = NT * p.tile_tok;
  if (a.map.B <= kSortSeqs) {
    if (tid < a.map.B) {
      uint32_t bits = 0;
      const PagedSeq q = paged_seq(a.map, tid, a.T, a.max_rows, bits);
      if (bits && blockIdx.x == 0 && blockIdx.y == 0) set_err(a.err, bits);
      s_seq[tid] = make_int2(q.len, chunk_items(q, p, item_tok));
    }
    __syncthreads();
    if (tid < a.map.B) {
      const int2 mine = s_seq[tid];
      int before = 0;
      for (int b = 0; b < a.map.B; ++b) {
        const int2 o = s_seq[b];
        if (o.x > mine.x || (o.x == mine.x && b < tid)) before += o.y;
      }
      const int want = blockIdx.x;
      if (want >= before && want < before + mine.y) {
        s_b = tid;
        s_idx = want - before;
      }
    }
    tc_fence_before();
    __syncthreads();
  } else {
    uint32_t bits = 0;
    const int E = (a.map.B + C::THREADS - 1) / C::THREADS;
    int mine = 0;
    for (int e = 0; e < E; ++e) {
      const int b = tid * E + e;
      if (b < a.map.B) mine += chunk_items(paged_seq(a.map, b, a.T, a.max_rows, bits), p, item_tok);
    }
    if (bits && blockIdx.x == 0 && blockIdx.y == 0) set_err(a.err, bits);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int w = 0; w < warp; ++w) before += s_scan[w];
    const int want = blockIdx.x;
    if (want >= before && want < before + mine) {
      int off = want - before;
      for (int e = 0; e < E; ++e) {
        uint32_t ignore = 0;
        const int n = chunk_items(paged_seq(a.map, tid * E + e, a.T, a.max_rows, ignore), p, item_tok);
        if (off < n) {
          s_b = tid * E + e;
          s_idx = off;
          break;
        }
        off -= n;
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  if (s_b < 0) {
    if (p.splits > 1 && blockIdx.y == 0 && tid == 0) p.rec_desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (warp == W_MMA) {
      tc_fence_after();
      tc_dealloc(s_tmem, 512);
    }
    return;
  }
  uint32_t ignore = 0;
  const int b = s_b, g = s_idx % a.map.nk;
  const PagedSeq s = paged_seq(a.map, b, a.T, a.max_rows, ignore);
  // the item with the most keys first
  const int n_qt = (s.t + item_tok - 1) / item_tok;
  const int tok0 = (n_qt - 1 - s_idx / a.map.nk) * item_tok;
  if (p.splits > 1 && blockIdx.y == 0 && tid == 0) p.rec_desc[blockIdx.x] = make_int4(b, g, tok0, 0);

  // key tiles of each query tile, and this CTA's share [j0, j1) of the item's
  int n_tile[NT], n_all = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int first = tok0 + t * p.tile_tok, last = min(first + p.tile_tok, s.t) - 1;
    const int lim = last >= first ? min(s.len, s.len - s.t + last + 1) : 0;
    n_tile[t] = lim > 0 ? (lim + KT - 1) / KT : 0;
    n_all = max(n_all, n_tile[t]);
  }
  const int j0 = (int)((long long)n_all * blockIdx.y / p.splits), j1 = (int)((long long)n_all * (blockIdx.y + 1) / p.splits);
  const int n = j1 - j0;                                   // tiles of this CTA

  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  auto give_up = [&]() {
    s_abort = 1;
    __threadfence_block();
    set_err(a.err, SWA_DERR_TIMEOUT);
  };
  // a wait made by a whole warp, with one outcome for the warp
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    return __all_sync(0xffffffffu, tc_wait(bar, (uint32_t)(phase & 1), &s_abort));
  };

  // The softmax threads hold a row of S: registers move over to them.
  if (warp >= W_LOAD) {
  if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::R_REST));
  if (warp == W_LOAD) {
    // ------------------------------------------------------------ loader
    // a slot is boxes of `rows` keys x 64 features
    const int page = 1 << a.map.page_shift, rows = min(page, KT), per_half = KT / rows;
    constexpr int HALVES = D / 64;
    const int32_t* table = a.map.table + (size_t)b * a.map.max_pages;
    const int oob = a.map.num_pages * a.map.nk << a.map.page_shift;       // rows of the pool: reads zeros
    bool ok = true;
    int issued = 0;
    auto load = [&](int j, bool is_v, int pos) {
      const int slot = pos % NS, use = pos / NS, key0 = (j0 + j) * KT;
      // lane bx looks up box bx of each half of the features (8 at most), before the wait
      const int key = key0 + lane * rows;
      int y = oob;
      if (lane < per_half && key < s.len) {
        const int id = table[key >> a.map.page_shift];
        if (page_ok(a.map, id))
          y = ((id * a.map.nk + g) << a.map.page_shift) + (key & (page - 1));
        else
          set_err(a.err, SWA_DERR_PAGE);
      }
      if (use > 0 && !wait(&b_empty[slot], use - 1)) return false;
      const bool tail = is_v && key0 + KT > s.len;
      uint64_t* bar = tail ? &b_tail : &b_full[slot];
      if (lane == 0) mbar_arrive_expect_tx(bar, C::SLOT);
      __syncwarp();
      unsigned char* dst = sm_kv + slot * C::SLOT;
      if (lane < per_half)
#pragma unroll
        for (int half = 0; half < HALVES; ++half)
          tma_2d(smem_u32(dst + half * (KT * 128) + lane * rows * 128), is_v ? &map_v : &map_k, half * 64, y, bar);
      issued = pos + 1;
      if (tail) {
        // at most one tile of a sequence: its V rows from the last key on become zeros
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&b_tail, 0, kWaitLimitNs))) return false;
        const int first = s.len - key0;
        for (int i = lane; i < (KT - first) * 8 * HALVES; i += 32) {
          const int c = i & 7, r = first + (i >> 3) % (KT - first), half = (i >> 3) / (KT - first);
          *reinterpret_cast<uint4*>(dst + half * (KT * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_full[slot]);
      }
      return true;
    };
    for (int x = 0; ok && x < n; ++x) {
      if (SB == 1) {
        ok = load(x, false, pos_k<SB>(x)) && load(x, true, pos_v<SB>(x, n));
      } else {
        if (x == 0) ok = load(0, false, 0);
        if (ok && x + 1 < n) ok = load(x + 1, false, pos_k<SB>(x + 1));
        if (ok) ok = load(x, true, pos_v<SB>(x, n));
      }
    }
    if (!ok) {
      give_up();
      // copies in flight land before the CTA exits (bounded)
      for (int q = max(0, issued - NS); q < issued; ++q) mbar_wait_bounded(&b_full[q % NS], (uint32_t)((q / NS) & 1), kWaitLimitNs);
    }
  } else if (warp < W_MMA + NT && n > 0) {
    // ------------------------------------------------------------ issuers, one per query tile
    // Products run in the order P V of tile 0, its next S, P V of tile 1, its next S: each
    // tile's softmax lies under the other's products. (Left alone, the two tiles fall into
    // step, wait together for the tensor core and leave it idle together: 888 instead of
    // 738 us at hd 128, four times 2048 rows over 8192 keys.) A warp waits, issues and commits for its
    // tile alone and passes the turn on through b_turn, so that these latencies (about 100
    // clk a wait, 250 a commit) overlap with the other tile's. The warp stays converged and
    // one elected lane issues.
    constexpr uint32_t ID_S = tc_idesc_16(BF, false, KT), ID_O = tc_idesc_16(BF, true, D);
    const int t = warp - W_MMA;
    const bool leader = elect_one();
    const int mine = max(0, min(n_tile[NT == 2 ? t : 0] - j0, n));   // tiles that this query tile sees
    const uint32_t c_s = tmem + t * SB * KT, c_o = tmem + C::C_O + t * D;
    // descriptors are a base plus (byte offset >> 4): the addresses stay below 2^18, so the
    // address field never carries
    const uint64_t q_desc = sw128_desc(smem_u32(sm + t * C::QB), 16), k_desc = sw128_desc(smem_u32(sm_kv), 16);
    const uint64_t v_desc = sw128_desc(smem_u32(sm_kv), KT * 128);
    bool ok = true;
    const int other = NT == 2 ? max(0, min(n_tile[NT - 1 - t] - j0, n)) : 0;
    auto pass_turn = [&]() {
      if (NT == 2) mbar_arrive(&b_turn[1 - t]);
    };
    // before this tile's j-th P V: after tile 0's j-th (tile 1), after tile 1's j-1st (tile 0)
    // A wait that gave up leaves ok false and the role goes on to its end (its warp stays
    // together without votes, which cost 4 % here): what follows only touches this CTA's own
    // shared memory and TMEM, and nothing of it is written.
    auto until = [&](uint64_t* bar, int phase) { ok &= tc_wait(bar, (uint32_t)(phase & 1), &s_abort); };
    auto my_turn = [&](int j) {
      if (NT == 1) return;
      if (t == 0) {
        if (j > 0 && other > 0) until(&b_turn[0], j - 1);
      } else if (j < other) {
        until(&b_turn[1], j);
      }
    };
    auto s_mma = [&](int j) {                               // S of tile j
      const int slot = pos_k<SB>(j) % NS;
      until(&b_full[slot], pos_k<SB>(j) / NS);
      tc_fence_after();
      if (leader) {
        const uint64_t kd = k_desc + (uint64_t)((slot * C::SLOT) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(c_s + (j % SB) * KT, q_desc + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                 kd + (((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4), ID_S, k > 0);
        if (j > 0) pass_turn();
        tc_commit(&b_s[t * SB + j % SB]);
      }
      __syncwarp();
    };
    auto pv_mma = [&](int j) {                              // O += P V of tile j
      const int pos = pos_v<SB>(j, n), slot = pos % NS;
      const uint64_t vd = v_desc + (uint64_t)((slot * C::SLOT) >> 4);
      until(&b_full[slot], pos / NS);
      my_turn(j);
#pragma unroll
      for (int h = 0; h < 2; ++h) {                         // P arrives in halves
        until(&b_p[t * SB + j % SB][h], j / SB);
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = h * (KT / 32); k < (h + 1) * (KT / 32); ++k)
            tc_mma_f16(c_o, c_s + (j % SB) * KT + k * 8, vd + (uint64_t)((k * 2048) >> 4), ID_O, j > 0 || k > 0);
          if (h == 1 && j + 1 == mine) pass_turn();
          if (h == 1) tc_commit(&b_pv[t]);
          // P came out of S, so K of this tile is done with
          if (h == 0) mbar_arrive(&b_empty[pos_k<SB>(j) % NS]);
        }
        __syncwarp();
      }
    };
    // O of tile j is there: its V is done with
    auto pv_done = [&](int j) {
      until(&b_pv[t], j);
      if (leader) mbar_arrive(&b_empty[pos_v<SB>(j, n) % NS]);
      __syncwarp();
    };
    if (mine > 0) {
      until(&b_q[t], 0);
      s_mma(0);
    }
    for (int j = 0; j < mine; ++j) {
      // with two S buffers the other one holds P of tile j - 1, with one S overwrites P of tile j
      if (SB == 2 && j > 0) pv_done(j - 1);
      if (SB == 2 && j + 1 < mine) s_mma(j + 1);
      pv_mma(j);
      if (SB == 1) pv_done(j);
      if (SB == 1 && j + 1 < mine) s_mma(j + 1);
    }
    for (int j = mine; j < n; ++j) {                        // the other tile's keys: hand the slots on
      const int pk = pos_k<SB>(j), pv = pos_v<SB>(j, n);
      until(&b_full[pk % NS], pk / NS);
      if (leader) mbar_arrive(&b_empty[pk % NS]);
      until(&b_full[pv % NS], pv / NS);
      if (leader) mbar_arrive(&b_empty[pv % NS]);
      __syncwarp();
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      give_up();
      // what was issued finishes before TMEM goes (bounded)
      if (leader) tc_commit(&b_fin[t]);
      mbar_wait_bounded(&b_fin[t], 0, kWaitLimitNs);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax: thread = row
    if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::R_SOFT));
    const int t = warp >> 2, r = tid & 127, hpg = a.hpg;
    const int first = tok0 + t * p.tile_tok;
    const int ntok = max(0, min(p.tile_tok, s.t - first)), nvec = ntok * hpg;
    const int mine = max(0, min(n_tile[t] - j0, n));
    const bool valid = r < nvec;
    const int tok = valid ? first + r / hpg : 0, head = g * hpg + (valid ? r % hpg : 0);
    // rows of no query vector (Q = 0) stay unmasked: nothing of them is written
    const int lim = valid ? min(s.len, s.len - s.t + tok + 1) : 0x7fffffff;
    const int lim_min = s.len - s.t + first + 1;           // keys below it need no mask
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (mine > 0) {
      // Q into shared memory: 16-byte chunks, rows of 128 bytes, swizzled, zeros behind its
      // vectors; all copies under way together, the row's address running along (loads through
      // registers, one after the other, took 6700 clk instead of 2800 at hd 64: 146 instead of 99 us
      // for 16 sequences of up to 512 rows over 1024 keys, 32 heads on 8, hd 128)
      constexpr int CH = D / 8, STEP = 128 / CH;
      const int c = r % CH, di = STEP / hpg, dh = STEP - di * hpg, t0 = r / CH / hpg;
      int h = r / CH - t0 * hpg;
      const T* src = static_cast<const T*>(a.q) + (size_t)(s.r0 + first + t0) * a.q_row + (size_t)(g * hpg + h) * D + c * 8;
      const long long ds = di * a.q_row + dh * D, dw = a.q_row - hpg * D;
      const uint32_t qs = smem_u32(sm + t * C::QB) + (c >> 3) * (128 * 128);
#pragma unroll 8
      for (int row = r / CH; row < 128; row += STEP) {
        const bool in = row < nvec;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(qs + row * 128 + (((c & 7) ^ (row & 7)) << 4)), "l"(in ? src : static_cast<const T*>(a.q)), "r"(in ? 16 : 0)
                     : "memory");
        h += dh;
        src += ds;
        if (h >= hpg) {
          h -= hpg;
          src += dw;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(&b_q[t]);
    }
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t c_o = lanes + C::C_O + t * D;
    for (int j = 0; j < mine; ++j) {
      const uint32_t c_s = lanes + (t * SB + j % SB) * KT;
      // a thread whose wait gave up goes on (its warp stays together) and writes nothing
      ok &= tc_wait(&b_s[t * SB + j % SB], (uint32_t)((j / SB) & 1), &s_abort);
      tc_fence_after();
      uint32_t x[KT / 32][32];
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) tc_ld32(c_s + i * 32, x[i]);
      wait_ld(x);
      const int key0 = (j0 + j) * KT;
      if (key0 + KT > lim_min) {
#pragma unroll
        for (int i = 0; i < KT / 32; ++i)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (key0 + i * 32 + k >= lim) x[i][k] = 0xff800000u;
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < KT / 32; ++i)
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          mx4[(k >> 1) & 3] = max3(mx4[(k >> 1) & 3], __uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1]));
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.qmul;
      const bool raise = mx > m + LazyMax<T>::kLazy;        // m starts at -inf
      if (__any_sync(0xffffffffu, raise) && j > 0) {
        const float f = raise ? ex2(m - mx) : 1.f;
        // with one S buffer S of this tile came after P V of the last one
        if (SB == 2) ok &= tc_wait(&b_pv[t], (uint32_t)((j - 1) & 1), &s_abort);
        if (SB == 2) tc_fence_after();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tc_ld32(c_o + i * 32, o);
          wait_ld(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tc_st32(c_o + i * 32, o);
        }
        l *= f;
      }
      if (raise) m = mx;
      const float off = LazyMax<T>::kLog2 - (m == -INFINITY ? 0.f : m);
      const uint64_t mul2 = pack64(__float_as_uint(a.qmul), __float_as_uint(a.qmul)),
                     off2 = pack64(__float_as_uint(off), __float_as_uint(off));
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {                         // each half of P goes to P V on its own
        uint32_t w[KT / 4];
#pragma unroll
        for (int k = 0; k < KT / 4; ++k) {
          const int e = h * (KT / 2) + 2 * k;
          float e0, e1;
          unpack64(fma2(pack64(x[e >> 5][e & 31], x[e >> 5][(e & 31) + 1]), mul2, off2), e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum[k & 1] = add2(sum[k & 1], pack64(__float_as_uint(e0), __float_as_uint(e1)));
          w[k] = pack2(e0, e1, (const T*)nullptr);
        }
        if constexpr (KT == 128) tc_st32(c_s + h * (KT / 4), w);
        else tc_st16(c_s + h * (KT / 4), w);
        tc_wait_st();
        tc_fence_before();
        // A wait sees only the parity of a phase: when this thread waits for the last P V, the
        // one before must be known complete, and a wait for that one must not come after the
        // last. With one S buffer the last S came after it; with two it is waited for here,
        // while the last P V still lacks this half.
        if (SB == 2 && h == 1 && j > 0 && j == mine - 1) ok &= tc_wait(&b_pv[t], (uint32_t)((j - 1) & 1), &s_abort);
        mbar_arrive(&b_p[t * SB + j % SB][h]);
      }
      float l0, l1;
      unpack64(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
    }
    if (mine > 0) ok &= tc_wait(&b_pv[t], (uint32_t)((mine - 1) & 1), &s_abort);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const size_t rec = (((size_t)blockIdx.x * p.splits + blockIdx.y) * NT + t) * 128 + r;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (mine > 0) {
          tc_ld32(c_o + i * 32, o);
          wait_ld(o);
        }
        if (!valid) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = mine > 0 ? __uint_as_float(o[k * 8 + e]) : 0.f;
          if (p.splits > 1)
            store8(p.rec_acc + rec * D + i * 32 + k * 8, y);
          else
            paged_store_row<T>(a, s.r0 + tok, head, D, i * 32 + k * 8, m, l, LazyMax<T>::kLog2, y, i == 0 && k == 0);
        }
      }
      if (p.splits > 1 && valid) p.rec_ml[rec] = make_float2(m, l);
    } else {
      give_up();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

// Joins the records of split items: a block per (item, row of the item), threads over
// groups of 8 features.
template <typename T, int D>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkParams p) {
  constexpr int L = D / 8, RW = 128 / L;                   // threads a row, rows a block
  constexpr int NT = ChunkCfg<D>::NT;
  pdl_wait();
  pdl_trigger();
  const int4 d = p.rec_desc[blockIdx.x];
  if (d.x < 0) return;
  uint32_t ignore = 0;
  const PagedAttendParams& a = p.a;
  const PagedSeq s = paged_seq(a.map, d.x, a.T, a.max_rows, ignore);
  const int row = blockIdx.y * RW + threadIdx.x / L, c = threadIdx.x % L;
  const int t = row >> 7, r = row & 127;
  const int tok = d.z + t * p.tile_tok + r / a.hpg;
  if (r >= p.tile_tok * a.hpg || tok >= s.t) return;
  const size_t rec0 = ((size_t)blockIdx.x * p.splits * NT + t) * 128 + r;
  float m = -INFINITY, l = 0.f, acc[8] = {};
  for (int i = 0; i < p.splits; ++i) m = fmaxf(m, p.rec_ml[rec0 + (size_t)i * NT * 128].x);
  for (int i = 0; i < p.splits; ++i) {
    const size_t rec = rec0 + (size_t)i * NT * 128;
    const float2 ml = p.rec_ml[rec];
    if (ml.x == -INFINITY) continue;
    const float f = ex2(ml.x - m);
    float y[8];
    load8(p.rec_acc + rec * D + c * 8, y);
    l += f * ml.y;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += f * y[k];
  }
  paged_store_row<T>(a, s.r0 + tok, d.y * a.hpg + r % a.hpg, D, c * 8, m, l, LazyMax<T>::kLog2, acc, c == 0);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
ChunkPlan chunk_plan(const swa_paged_attend_args* a, int max_rows) {
  const swa_paged_cache& c = a->cache;
  const int hpg = a->nh / c.nk, nt = c.hd == 256 ? 1 : 2, kt = c.hd == 256 ? 64 : 128;
  ChunkPlan pl{};
  pl.tile_tok = 128 / hpg;
  const long long item_tok = (long long)nt * pl.tile_tok;
  pl.items = ((long long)a->T / item_tok + c.B) * c.nk;
  // one sequence of max_rows rows has no more items than its rows need
  const long long most = (max_rows + item_tok - 1) / item_tok * c.B * c.nk;
  if (most < pl.items) pl.items = most;
  // Fewer items than SMs: cut the keys, at least four tiles a share of a sequence as long as the
  // table is wide (with twice as many shares, for even ends: 80 instead of 50 us for 256 rows over
  // 32768 keys, 8 heads on 2, hd 128). The lengths and the rows of each sequence are the device's, so
  // what is counted here are bounds: a short sequence in a wide table is cut finer than pays (256 rows
  // over 512 keys, 8 heads on 2: 18.4 us in a table of 512, 25 in one of 32768), and single tokens in
  // the same call count as items (256 rows and 31 tokens over 16384 keys: 229 us, 43 and 107 apart).
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  const long long tiles = ((long long)c.max_pages * c.page + kt - 1) / kt;
  long long sp = sms / pl.items;
  if (sp > (tiles + 3) / 4) sp = (tiles + 3) / 4;
  pl.splits = (int)(sp < 1 ? 1 : sp);
  if (pl.splits > 1) {
    const size_t recs = (size_t)pl.items * pl.splits * nt * 128;
    pl.off_ml = up256s(recs * c.hd * sizeof(float));
    pl.off_desc = pl.off_ml + up256s(recs * sizeof(float2));
    pl.bytes = pl.off_desc + up256s((size_t)pl.items * sizeof(int4));
  }
  return pl;
}

template <typename T, int D>
static int launch(const swa_paged_attend_args* a, const PagedAttendParams& ap, const ChunkPlan& pl, int small, char* ws,
                  cudaStream_t s) {
  CUtensorMap mk, mv;
  int rc = pool_map(a->cache, a->cache.k, ChunkCfg<D>::KT, &mk);
  if (rc == SWA_OK) rc = pool_map(a->cache, a->cache.v, ChunkCfg<D>::KT, &mv);
  if (rc != SWA_OK) return rc;
  ChunkParams p{};
  p.a = ap;
  p.a.qmul = fmaxf(ap.qmul, 0x1p-100f);                    // masked scores stay -inf when scale is 0
  p.small = small;
  p.tile_tok = pl.tile_tok;
  p.splits = pl.splits;
  p.rec_acc = reinterpret_cast<float*>(ws);
  p.rec_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  p.rec_desc = reinterpret_cast<int4*>(ws + pl.off_desc);
  const cudaError_t e = allow_smem<paged_chunk_kernel<T, D>>(ChunkCfg<D>::SMEM, ChunkCfg<D>::REGS);
  if (e != cudaSuccess) return cuda_status(e);
  rc = finish_launch(launch_pdl(paged_chunk_kernel<T, D>, dim3((unsigned)pl.items, pl.splits), dim3(ChunkCfg<D>::THREADS),
                                ChunkCfg<D>::SMEM, s, mk, mv, p));
  if (rc != SWA_OK || pl.splits == 1) return rc;
  constexpr int RW = 128 / (D / 8);
  return finish_launch(launch_pdl(chunk_merge_kernel<T, D>, dim3((unsigned)pl.items, ChunkCfg<D>::NT * 128 / RW), dim3(128), 0, s, p));
}

int launch_paged_chunk(const swa_paged_attend_args* a, const PagedAttendParams& p, const ChunkPlan& pl, int small, char* ws,
                       cudaStream_t s) {
  const int d = a->cache.hd;
  if (a->cache.dtype == SWA_BF16)
    return d == 64 ? launch<__nv_bfloat16, 64>(a, p, pl, small, ws, s)
                   : d == 128 ? launch<__nv_bfloat16, 128>(a, p, pl, small, ws, s) : launch<__nv_bfloat16, 256>(a, p, pl, small, ws, s);
  return d == 64 ? launch<__half, 64>(a, p, pl, small, ws, s)
                 : d == 128 ? launch<__half, 128>(a, p, pl, small, ws, s) : launch<__half, 256>(a, p, pl, small, ws, s);
}

}  // namespace swa
