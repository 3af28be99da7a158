// Attention of chunks with many query vectors per KV head over the 4-bit paged cache, on the
// tensor cores. Part of swa_paged_chunk.cu, whose 16-bit kernel explains the plan: tiles of 128
// query vectors, S and O in TMEM, a softmax warpgroup and an issuing warp a tile, and
// two tiles (hd 64, 128) or two S buffers (hd 256) so that products run under the softmax.
// What differs:
//   - a warp copies codes and scales as they are (4.5 bits a feature) into rings of their own. They
//     become f16 operands, in the swizzled layout that the products read, once for the item's 256 query
//     vectors: with two tiles by the softmax warps, each between its weights and its next scores, V by those of
//     the first tile and K by those of the second, who then find the slot free; at hd 256 by two warpgroups of
//     their own, whose registers partly go to the softmax threads (38 sequences of 21 rows, 16 heads on 4, over 3729 .. 12025
//     keys: 202 us; with one 227, and with a ring of codes for K and one for V 247; without conversions 184). (Four more
//     warps that did only this at hd 128 left the softmax threads 184 registers of the 220 that a row of S takes, and took
//     their issue slots: 654 us where this takes 562; both warpgroups with half a tile each waited for one another: 638.)
//   - all products are f16: codes * scale is exact there, q is scaled by a power of two a row.
//   - tiles of keys that no row sees (between the sinks and the first row's window) are left
//     out; a row's own limits are masks.
// 4 chunks of up to 2048 rows over 2048 .. 16384 keys, 32 heads on 8, hd 128: 562 us, 1115 TFLOP/s (451 us without the
// conversions). The tensor pipe is busy for 49 % of it (both operands of Q K^T come from shared memory), the issue slots for 50 %;
// a tile's chain of scores, softmax and values has no second S buffer to hide in, and at hd 64 and 128 the softmax threads spill (48
// and 60 bytes stored, 232 and 344 loaded). (Two softmax warpgroups a query tile, half
// a row each: 594. An eighth or a quarter of the exponentials as polynomials: 587, 617.)
#pragma once
#include "swa_paged4_attend.cuh"

namespace swa {

template <int D>
struct Chunk4Cfg {
  static constexpr int NT = ChunkCfg<D>::NT, SB = ChunkCfg<D>::SB, KT = ChunkCfg<D>::KT;
  static constexpr bool OWN = NT == 2;                 // the softmax warps convert
  static constexpr int RK = 2, RV = D == 64 ? 2 : 1;   // slots of K's and of V's codes and scales
  static constexpr int SLOT = KT * D * 2, CODES = KT * D / 2, RAW = CODES + KT * D / 16;   // operands: two slots for K, two for V
  static constexpr int QB = 128 * D * 2;
  static constexpr int CW = OWN ? 4 : 8;                // warps that convert a tile
  static constexpr int THREADS = NT * 128 + 128 + (OWN ? 0 : 32 * CW);   // softmax; loader, issuers, idle warps; conversion
  static constexpr int SMEM = NT * QB + 4 * SLOT + (RK + RV) * RAW + 1024;   // + alignment
  // Registers a thread at launch and after they moved to the softmax threads
  static constexpr int REGS = NT == 2 ? 168 : 128, R_SOFT = NT == 2 ? 216 : 200, R_REST = NT == 2 ? 72 : 104;
  static_assert(NT * 128 * R_SOFT + (THREADS - NT * 128) * R_REST <= THREADS * REGS, "registers of a CTA");
  static constexpr int C_O = NT * SB * KT;             // first O column
};

struct Chunk4Params {
  Attend4Params q;
  ChunkParams c;               // its a: the same as q.a
};

// The tiles that rows [first, first + rows) of a sequence see, as list positions below `lim`'s
__device__ __forceinline__ int tiles_below(const Tiles4& tl, int lim, int kt) {
  const int end = lim > 0 ? (lim + kt - 1) / kt : 0;
  return end > tl.first ? tl.sink + end - tl.first : min(tl.sink, end);
}

template <int D>
__global__ void __launch_bounds__(Chunk4Cfg<D>::THREADS, 1) paged4_chunk_kernel(const __grid_constant__ Chunk4Params p) {
  using C = Chunk4Cfg<D>;
  constexpr int NT = C::NT, SB = C::SB, KT = C::KT, RK = C::RK, RV = C::RV;
  extern __shared__ unsigned char sm_raw[];
  // tests/test_paged4_barriers_cpu.py runs the roles below on a model of these barriers: what waits
  // or arrives here has to be changed there too
  __shared__ __align__(8) uint64_t b_raw[RK + RV], b_free[RK + RV], b_full[4], b_empty[4], b_q[NT], b_s[NT * SB], b_p[NT * SB][2], b_pv[NT], b_fin[NT], b_turn[NT];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_b, s_idx;
  __shared__ int s_scan[32];
  __shared__ int2 s_seq[kSortSeqs];        // (keys, items) of each sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  constexpr int W_LOAD = NT * 4, W_MMA = NT * 4 + 1, W_CONV = NT * 4 + 4;
  unsigned char* const sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* const sm_kv = sm + NT * C::QB;
  unsigned char* const sm_codes = sm_kv + 4 * C::SLOT;
  const PagedAttendParams& a = p.q.a;
  // what needs no global memory, before the wait for the kernel in front
  if (warp == W_LOAD) {
    if (lane == 0) {
      for (int i = 0; i < RK + RV; ++i) {
        mbar_init(&b_raw[i], 1);
        mbar_init(&b_free[i], C::CW);
      }
      for (int i = 0; i < 4; ++i) {        // K tiles 0 and 1 modulo 2, V tiles
        mbar_init(&b_full[i], C::CW);
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

  // --- which item (as in the 16-bit kernel: the longest sequences' first)
  const int item_tok = NT * p.c.tile_tok;
  if (a.map.B <= kSortSeqs) {
    if (tid < a.map.B) {
      uint32_t bits = 0;
      const PagedSeq q = paged_seq(a.map, tid, a.T, a.max_rows, bits);
      if (bits && blockIdx.x == 0 && blockIdx.y == 0) set_err(a.err, bits);
      s_seq[tid] = make_int2(q.len, chunk_items(q, p.c, item_tok));
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
      if (b < a.map.B) mine += chunk_items(paged_seq(a.map, b, a.T, a.max_rows, bits), p.c, item_tok);
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
        const int n = chunk_items(paged_seq(a.map, tid * E + e, a.T, a.max_rows, ignore), p.c, item_tok);
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
    if (p.c.splits > 1 && blockIdx.y == 0 && tid == 0) p.c.rec_desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
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
  if (p.c.splits > 1 && blockIdx.y == 0 && tid == 0) p.c.rec_desc[blockIdx.x] = make_int4(b, g, tok0, 0);

  // the item's tiles of keys, how many of them each query tile's rows reach, and this CTA's share [j0, j1)
  const int window = p.q.window, sinks = p.q.sinks;
  const int lo_min = first_key(s.len - s.t + tok0 + 1, window);   // the item's first row's
  Tiles4 tl;
  tl.first = lo_min / KT;
  tl.sink = min((min(sinks, s.len) + KT - 1) / KT, tl.first);
  int n_tile[NT], n_all = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int first = tok0 + t * p.c.tile_tok, last = min(first + p.c.tile_tok, s.t) - 1;
    const int lim = last >= first ? min(s.len, s.len - s.t + last + 1) : 0;
    n_tile[t] = tiles_below(tl, lim, KT);
    n_all = max(n_all, n_tile[t]);
  }
  const int j0 = (int)((long long)n_all * blockIdx.y / p.c.splits), j1 = (int)((long long)n_all * (blockIdx.y + 1) / p.c.splits);
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
  // K and V tiles in the order in which they are copied and converted, V x + 1 and K x + 2 after the scores of x: K 0,
  // V 0, K 1, V 1, ..; f(tile, is V)
  auto in_order = [&](auto f) {
    bool ok = true;
    for (int x = -2; ok && x < n; ++x) {
      if (x >= -1 && x + 1 < n) ok = f(x + 1, true);
      if (ok && x + 2 < n) ok = f(x + 2, false);
    }
    return ok;
  };
  // tile x's slot of codes and the use of it: K's and V's own where different warps convert them, else all in their order
  auto raw_slot = [&](int x, bool is_v) { return !C::OWN ? (2 * x + is_v) % (RK + RV) : is_v ? RK + x % RV : x % RK; };
  auto raw_use = [&](int x, bool is_v) { return !C::OWN ? (2 * x + is_v) / (RK + RV) : is_v ? x / RV : x / RK; };

  // Codes to operands: tile x by one or two warpgroups whose thread is wt, 32 features a thread at a time
  constexpr int LR = D / 32, RP = 32 * C::CW / LR;        // lanes of a key, keys of a pass
  auto convert = [&](int wt, int x, bool is_v) {
    const int q = wt % LR, r0 = wt / LR, raw = raw_slot(x, is_v), slot = (is_v ? 2 : 0) + (x & 1), key0 = tl.at(j0 + x) * KT;
    // 16-byte chunk i of these 32 features goes to chunk 4 (q & 1) + i of its 64-feature half; lanes of
    // other halves take their chunks in another order, so that eight lanes store to eight bank groups
    const int turn = D == 256 ? q >> 1 : D == 128 ? 2 * (q >> 1) : 0;
    static_assert(RP % 8 == 0, "a thread's keys are the same modulo 8");
    if (!wait(&b_raw[raw], raw_use(x, is_v))) return false;
    if (x >= 2 && !wait(&b_empty[slot], (x >> 1) - 1)) return false;
    const uint32_t src = smem_u32(sm_codes) + raw * C::RAW + q * 16, scales = smem_u32(sm_codes) + raw * C::RAW + C::CODES + q * 2;
    const uint32_t dst = smem_u32(sm_kv) + slot * C::SLOT + (q >> 1) * (KT * 128);
    // what no row sees may be NaN in V: zeros, by its scale
    const bool part = is_v && (key0 + KT > s.len || key0 < lo_min);
#pragma unroll 2
    for (int r = r0; r < KT; r += RP) {
      uint32_t w[4];
      lds_words<4>(w, src + r * (D / 2));
      uint32_t u = lds_u16(scales + r * (D / 16));
      if (part && (key0 + r >= s.len || (key0 + r < lo_min && key0 + r >= sinks))) u = 0;
      uint32_t sc = e4m3x2_f16x2(u);
      if (D >= 128 && (turn & 2)) {
        const uint32_t y = w[0], z = w[1];
        w[0] = w[2];
        w[1] = w[3];
        w[2] = y;
        w[3] = z;
        sc = __byte_perm(sc, sc, 0x1032);
      }
      if (D == 256 && (turn & 1)) {
        const uint32_t y = w[0], z = w[2];
        w[0] = w[1];
        w[1] = y;
        w[2] = w[3];
        w[3] = z;
      }
      const uint32_t s0 = __byte_perm(sc, sc, 0x1010), s1 = __byte_perm(sc, sc, 0x3232);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = i < 2 ? s0 : s1;
        sts_words(dst + r * 128 + (((4 * (q & 1) + (i ^ turn)) ^ (r0 & 7)) << 4), hmul2(e2m1x2_f16x2<0>(w[i]), m),
                  hmul2(e2m1x2_f16x2<1>(w[i]), m), hmul2(e2m1x2_f16x2<2>(w[i]), m), hmul2(e2m1x2_f16x2<3>(w[i]), m));
      }
    }
    fence_proxy_async_smem();             // before the products read it
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&b_free[raw]);
      mbar_arrive(&b_full[slot]);
    }
    return true;
  };

  // The softmax threads hold a row of S: registers move over to them.
  if (warp >= W_LOAD) {
  regs_give<C::R_REST>();
  if (warp == W_LOAD) {
    // ------------------------------------------------------------ loader: a run of codes or of scales a lane
    const int page = 1 << a.map.page_shift, rows = min(page, KT), runs = KT / rows;   // 2 * runs <= 16
    const bool codes = lane < runs, mine = lane < 2 * runs;
    const int run = codes ? lane : lane - runs, row = codes ? D / 2 : D / 16;
    const int32_t* table = a.map.table + (size_t)b * a.map.max_pages;
    int last[RK + RV];                    // the last use of each slot that was copied to
#pragma unroll
    for (int i = 0; i < RK + RV; ++i) last[i] = -1;
    const bool ok = in_order([&](int x, bool is_v) {
      const int slot = raw_slot(x, is_v), use = raw_use(x, is_v), key = tl.at(j0 + x) * KT + run * rows;
      unsigned char* const dst = sm_codes + slot * C::RAW + (codes ? 0 : C::CODES) + run * rows * row;
      const uint8_t* from = nullptr;
      bool blank = false;
      if (mine && key < s.len) {          // looked up before the wait
        const int id = table[key >> a.map.page_shift];
        if (page_ok(a.map, id)) {
          from = (is_v ? (codes ? p.q.c.v : p.q.c.vs) : (codes ? p.q.c.k : p.q.c.ks)) +
                 ((((long long)id * a.map.nk + g) << a.map.page_shift) + (key & (page - 1))) * row;
        } else {
          set_err(a.err, SWA_DERR_PAGE);
          blank = !codes;                 // such keys read as zeros: by their scales
        }
      }
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, from ? rows * row : 0);
      if (use > 0 && !wait(&b_free[slot], use - 1)) return false;
      if (blank) {
        for (int i = 0; i < rows * row; i += 16) *reinterpret_cast<uint4*>(dst + i) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();         // before a later copy into this slot
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&b_raw[slot], bytes);
      __syncwarp();
      if (from) bulk_g2s(dst, from, rows * row, &b_raw[slot]);
      last[slot] = use;
      return true;
    });
    if (!ok) {
      give_up();
      // copies in flight land before the CTA exits (bounded)
#pragma unroll
      for (int i = 0; i < RK + RV; ++i)
        if (last[i] >= 0) mbar_wait_bounded(&b_raw[i], (uint32_t)(last[i] & 1), kWaitLimitNs);
    }
  } else if (!C::OWN && warp >= W_CONV) {
    // ------------------------------------------------------------ conversion
    if (!in_order([&](int x, bool is_v) { return convert(tid - W_CONV * 32, x, is_v); })) give_up();
  } else if (warp < W_MMA + NT && n > 0) {
    // ------------------------------------------------------------ issuers, one per query tile (as in the 16-bit kernel)
    constexpr uint32_t ID_S = tc_idesc_16(false, false, KT), ID_O = tc_idesc_16(false, true, D);
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
    // A wait that gave up leaves ok false and the role goes on to its end: what follows only touches
    // this CTA's own shared memory and TMEM, and nothing of it is written.
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
      const int slot = j & 1;
      until(&b_full[slot], j >> 1);
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
      const int slot = 2 + (j & 1);
      const uint64_t vd = v_desc + (uint64_t)((slot * C::SLOT) >> 4);
      until(&b_full[slot], j >> 1);
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
          if (h == 0) mbar_arrive(&b_empty[j & 1]);
        }
        __syncwarp();
      }
    };
    // O of tile j is there: its V is done with
    auto pv_done = [&](int j) {
      until(&b_pv[t], j);
      if (leader) mbar_arrive(&b_empty[2 + (j & 1)]);
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
      until(&b_full[j & 1], j >> 1);
      if (leader) mbar_arrive(&b_empty[j & 1]);
      until(&b_full[2 + (j & 1)], j >> 1);
      if (leader) mbar_arrive(&b_empty[2 + (j & 1)]);
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
    regs_take<C::R_SOFT>();
    const int t = warp >> 2, r = tid & 127, hpg = a.hpg;
    const int first = tok0 + t * p.c.tile_tok;
    const int ntok = max(0, min(p.c.tile_tok, s.t - first)), nvec = ntok * hpg;
    const int mine = max(0, min(n_tile[t] - j0, n));
    const bool valid = r < nvec;
    const int tok = valid ? first + r / hpg : 0, head = g * hpg + (valid ? r % hpg : 0);
    // rows of no query vector (Q = 0): nothing of them is written
    const int lim = valid ? max(0, min(s.len, s.len - s.t + tok + 1)) : 0x7fffffff;
    const int lim_min = s.len - s.t + first + 1;           // keys below it are before or at every row's own
    const int lo_max = first_key(min(s.len, s.len - s.t + first + max(ntok, 1)), window);   // the last row's first key
    float m = -INFINITY, l = 0.f, qmul = 1.f;
    bool ok = true;
    if (mine > 0) {
      // the thread's own row of Q, scaled and in f16, in shared memory: rows of 128 bytes, swizzled
      uint4 w[D / 8];
      const uint16_t* const src = static_cast<const uint16_t*>(a.q) + (size_t)(s.r0 + tok) * a.q_row + (size_t)head * D;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) w[c] = valid ? *reinterpret_cast<const uint4*>(src + c * 8) : make_uint4(0, 0, 0, 0);
      auto each = [&](uint4& v, auto f) {
        uint32_t* const y[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float e0, e1;
          if (p.q.bf) unpack2(*y[i], e0, e1, (const __nv_bfloat16*)nullptr);
          else unpack2(*y[i], e0, e1, (const __half*)nullptr);
          f(*y[i], e0, e1);
        }
      };
      float top = 0.f, inv;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) each(w[c], [&](uint32_t&, float e0, float e1) { top = max3(top, fabsf(e0), fabsf(e1)); });
      const float mul = query_scale(top, inv);
      // masked scores stay -inf, also where the scale is 0 or nearly
      qmul = fmaxf(a.qmul * inv, 0x1p-126f);
      unsigned char* const qs = sm + t * C::QB + r * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        each(w[c], [&](uint32_t& y, float e0, float e1) { y = pack2(e0 * mul, e1 * mul, (const __half*)nullptr); });
        *reinterpret_cast<uint4*>(qs + (c >> 3) * (128 * 128) + (((c & 7) ^ (r & 7)) << 4)) = w[c];
      }
      fence_proxy_async_smem();
      mbar_arrive(&b_q[t]);
    }
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t c_o = lanes + C::C_O + t * D;
    // After the scores of tile j a later one (own or not) is converted: V j + 1 by the first query tile's threads,
    // K j + 2 by the second's
    const int ahead = t == 0 ? 1 : 2;
    if (C::OWN) {
#pragma unroll 1
      for (int x = 0; x < min(ahead, n); ++x) ok &= convert(r, x, t == 0);
    }
    for (int j = 0; j < mine; ++j) {
      const uint32_t c_s = lanes + (t * SB + j % SB) * KT;
      // a thread whose wait gave up goes on (its warp stays together) and writes nothing
      ok &= tc_wait(&b_s[t * SB + j % SB], (uint32_t)((j / SB) & 1), &s_abort);
      tc_fence_after();
      uint32_t x[KT / 32][32];
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) tc_ld32(c_s + i * 32, x[i]);
      wait_ld(x);
      const int key0 = tl.at(j0 + j) * KT;
      if (key0 + KT > lim_min || key0 < lo_max) {
        const int end = lim - key0, lo = lim - window - key0, sk = sinks - key0;   // seen: below end, and from lo on or below sk
#pragma unroll
        for (int i = 0; i < KT / 32; ++i)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (i * 32 + k >= end || (i * 32 + k < lo && i * 32 + k >= sk)) x[i][k] = 0xff800000u;
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < KT / 32; ++i)
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          mx4[(k >> 1) & 3] = max3(mx4[(k >> 1) & 3], __uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1]));
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * qmul;
      const bool raise = mx > m + kLazy4;                   // m starts at -inf
      if (__any_sync(0xffffffffu, raise) && j > 0) {
        const float f = raise ? ex2(m - mx) : 1.f;
        // with one S buffer S of this tile came after P V of the last one
        if (SB == 2) ok &= tc_wait(&b_pv[t], (uint32_t)((j - 1) & 1), &s_abort);
        if (SB == 2) tc_fence_after();
#pragma unroll 1
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
      const float off = kLog24 - (m == -INFINITY ? 0.f : m);
      const uint64_t mul2 = pack64(__float_as_uint(qmul), __float_as_uint(qmul)),
                     off2 = pack64(__float_as_uint(off), __float_as_uint(off));
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {                         // each half of P goes to P V on its own
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          uint32_t w[KT / 8];
#pragma unroll
          for (int k = 0; k < KT / 8; ++k) {
            const int e = h * (KT / 2) + z * (KT / 4) + 2 * k;
            float e0, e1;
            unpack64(fma2(pack64(x[e >> 5][e & 31], x[e >> 5][(e & 31) + 1]), mul2, off2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            sum[k & 1] = add2(sum[k & 1], pack64(__float_as_uint(e0), __float_as_uint(e1)));
            w[k] = pack2(e0, e1, (const __half*)nullptr);
          }
          if constexpr (KT == 128) tc_st16(c_s + h * (KT / 4) + z * (KT / 8), w);
          else tc_st8(c_s + h * (KT / 4) + z * (KT / 8), w);
        }
        tc_wait_st();
        tc_fence_before();
        // A wait sees only the parity of a phase: the P V before the last must be known complete before the
        // last is waited for (see the 16-bit kernel)
        if (SB == 2 && h == 1 && j > 0 && j == mine - 1) ok &= tc_wait(&b_pv[t], (uint32_t)((j - 1) & 1), &s_abort);
        mbar_arrive(&b_p[t * SB + j % SB][h]);
      }
      float l0, l1;
      unpack64(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
      if (C::OWN && j + ahead < n) ok &= convert(r, j + ahead, t == 0);
    }
    if (C::OWN) {                                           // the other tile's keys
#pragma unroll 1
      for (int x = mine + ahead; x < n; ++x) ok &= convert(r, x, t == 0);
    }
    if (mine > 0) ok &= tc_wait(&b_pv[t], (uint32_t)((mine - 1) & 1), &s_abort);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const size_t rec = (((size_t)blockIdx.x * p.c.splits + blockIdx.y) * NT + t) * 128 + r;
      const float unit = p.c.splits > 1 && p.q.bf ? 0x1p-11f : 1.f;     // the merge's weights of bf16 rows carry no 2^kLog24
      const float v_mul = p.q.c.v_mul * unit;
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
          for (int e = 0; e < 8; ++e) y[e] = mine > 0 ? __uint_as_float(o[k * 8 + e]) * v_mul : 0.f;
          if (p.c.splits > 1)
            store8(p.c.rec_acc + rec * D + i * 32 + k * 8, y);
          else if (p.q.bf)
            paged_store_row<__nv_bfloat16>(a, s.r0 + tok, head, D, i * 32 + k * 8, m, l, kLog24, y, i == 0 && k == 0);
          else
            paged_store_row<__half>(a, s.r0 + tok, head, D, i * 32 + k * 8, m, l, kLog24, y, i == 0 && k == 0);
        }
      }
      if (p.c.splits > 1 && valid) p.c.rec_ml[rec] = make_float2(m, l * unit);
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

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
ChunkPlan chunk4_plan(const swa_paged4_attend_args* a, int max_rows) {
  const swa_paged4_cache& c = a->cache;
  const int hpg = a->nh / c.nk, nt = c.hd == 256 ? 1 : 2, kt = c.hd == 256 ? 64 : 128;
  ChunkPlan pl{};
  pl.tile_tok = 128 / hpg;
  const long long item_tok = (long long)nt * pl.tile_tok;
  pl.items = ((long long)a->T / item_tok + c.B) * c.nk;
  // one sequence of max_rows rows has no more items than its rows need
  const long long most = (max_rows + item_tok - 1) / item_tok * c.B * c.nk;
  if (most < pl.items) pl.items = most;
  // Fewer items than SMs: cut the keys, at least four tiles a share of what a row can see at most
  const long long sms = num_sms() > 0 ? num_sms() : 148;
  long long tiles = ((long long)c.max_pages * c.page + kt - 1) / kt;
  if (a->window) {
    const long long seen = ((long long)a->window + item_tok) / kt + a->sinks / kt + 3;
    if (seen < tiles) tiles = seen;
  }
  long long sp = sms / pl.items;
  if (sp > (tiles + 3) / 4) sp = (tiles + 3) / 4;
  // About as many items as SMs: the longest sequence's CTA, or a second round of a few, would decide. Shares of 2560 keys at
  // least, so that two of them fall to each SM. The host knows no lengths, so that this gains where a second round would be
  // a few items of full length, and loses where lengths differ and even that round out. 16 heads on 4, whole / cut, us:
  //   152 items (38 sequences; 21 rows at hd 256, 40 below)  3729 .. 12025 keys  hd 256 238 / 209, 128 185 / 171, 64 152 / 134
  //                                                          8000 keys each      hd 256 165 / 193, 128 132 / 156
  //   160 and 200 items   8000 keys each      hd 256 319 / 269, 322 / 278   128 256 / 225, 258 / 230   64 209 / 175, 211 / 179
  //                       3729 .. 12025 keys  hd 256 237 / 246, 253 / 292   128 190 / 206, 218 / 246   64 157 / 158, 180 / 194
  //   80 items            3729 .. 12025 keys  128 181 / 119 (in three), 64 149 / 93
  // (One sequence's items are about equal: only where SMs would be left over. Where the keys are cut anyway twice as many shares
  // cost more: 64 rows over 131072 keys, 8 items in 19, 138 us, in 38 177.)
  if (sp < 2 && pl.items * 3 <= sms * 4 && (c.B > 1 || pl.items * 4 < sms * 3)) {
    long long even = (2 * sms + pl.items - 1) / pl.items;
    if (even > tiles * kt / 2560) even = tiles * kt / 2560;
    if (sp < even) sp = even;
  }
  pl.splits = (int)(sp < 1 ? 1 : sp);
  if (pl.splits > 1) {
    const size_t recs = (size_t)pl.items * pl.splits * nt * 128;
    pl.off_ml = up256s(recs * c.hd * sizeof(float));
    pl.off_desc = pl.off_ml + up256s(recs * sizeof(float2));
    pl.bytes = pl.off_desc + up256s((size_t)pl.items * sizeof(int4));
  }
  return pl;
}

template <int D>
static int launch4(const Attend4Params& ap, const ChunkPlan& pl, int small, char* ws, cudaStream_t s) {
  Chunk4Params p{};
  p.q = ap;
  p.c.a = ap.a;
  p.c.small = small;
  p.c.tile_tok = pl.tile_tok;
  p.c.splits = pl.splits;
  p.c.rec_acc = reinterpret_cast<float*>(ws);
  p.c.rec_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  p.c.rec_desc = reinterpret_cast<int4*>(ws + pl.off_desc);
  const cudaError_t e = allow_smem<paged4_chunk_kernel<D>>(Chunk4Cfg<D>::SMEM, Chunk4Cfg<D>::REGS);
  if (e != cudaSuccess) return cuda_status(e);
  const int rc = finish_launch(launch_pdl(paged4_chunk_kernel<D>, dim3((unsigned)pl.items, pl.splits), dim3(Chunk4Cfg<D>::THREADS),
                                          Chunk4Cfg<D>::SMEM, s, p));
  if (rc != SWA_OK || pl.splits == 1) return rc;
  constexpr int RW = 128 / (D / 8);
  const dim3 grid((unsigned)pl.items, Chunk4Cfg<D>::NT * 128 / RW);
  return finish_launch(ap.bf ? launch_pdl(chunk_merge_kernel<__nv_bfloat16, D>, grid, dim3(128), 0, s, p.c)
                             : launch_pdl(chunk_merge_kernel<__half, D>, grid, dim3(128), 0, s, p.c));
}

int launch_paged4_chunk(int hd, const Attend4Params& p, const ChunkPlan& pl, int small, char* ws, cudaStream_t s) {
  return hd == 64 ? launch4<64>(p, pl, small, ws, s) : hd == 128 ? launch4<128>(p, pl, small, ws, s) : launch4<256>(p, pl, small, ws, s);
}

}  // namespace swa
