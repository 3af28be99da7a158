// Attention of a ragged chunk over the 4-bit paged cache: the kernel for few query vectors per
// KV head (decode tokens, verify chunks) and the host side of swa_paged4_attend.
//
// A key costs 4.5 bits a feature to read, and 16 bits at least to multiply: the codes have to become
// f16 on the way. At the memory's rate an SM has 98 clk for the 2304 bytes of 16 keys and values
// (hd 128); turning them into f16 takes 47 clk of its conversion unit (44 pairs of codes a clk,
// measured) and 31 of its f16 multipliers (the scales), if that happens once and in the registers of
// the product that reads them. So the keys are the rows of both products, whose operand A holds
// what a warp has just converted, and up to 32 query vectors are the columns:
//   S^T [16 keys x 8 vectors] = K [16 x hd] Q^T, in steps of 16 features. The sum over features may
//     run in any order: lane (g, t) takes 16 bytes of key g at a time, features 32 t .. 32 t + 31,
//     and Q^T is laid out alike.
//   O^T [hd x 8 vectors] += V^T [hd x 16 keys] P^T. A pair of an operand is now two keys of one feature:
//     the lower (upper) halves of two keys' bytes are put into one byte before the conversion.
//   P^T comes out of S^T by movmatrix: 8 x 8 transposed, in registers.
// A value code * scale is exact in f16. Weights enter the second product in f16, scaled by
// 2^(kLog24 + up to kLazy4) so that small ones keep their bits, with what that rounding leaves where the result shows it.
// Every CTA gets the same share of the whole call's tiles and items' starts, wherever the cuts fall; one warp copies
// them from the pages (plain bulk copies: a head's keys of a page are consecutive), the others take
// a quarter of a tile's keys each (or half, for half of the vectors or features), with a running maximum and
// sums of their own, joined at an item's end.
// Items that are cut leave a record (m, l, sum p v) per CTA, joined by paged_merge_kernel.
// 64 sequences of 1024 .. 8192 keys, 8 KV heads of hd 128, one token of 4 vectors a head (367 MB): 78 us, 4.7 TB/s.
// The copies alone take 65, the products with the conversions 73: some 300 instructions of a warp for 16 keys, at 0.6 a clk
// of each of the SM's four schedulers. (Where the call took 85 us, four CTAs an SM with 96 registers took 95, by what no
// longer fits; four CTAs without a warp that copies, the last to read a stage refilling it, 101.)
// 32 times 16 vectors (4 drafts) over a window of 4096 keys, 4 KV heads of hd 256 (153 MB): 62 us, 73 with the rest of f16 weights; copies alone 39, products 59.
#include <cmath>

#include "swa_paged4_attend.cuh"
#include "swa_paged_merge.cuh"

namespace swa {

constexpr int kWarps4 = 4;           // warps that compute
constexpr int kWeighed = 8;          // tiles a CTA from which on an item's start counts (below that the cuts matter more)
constexpr int kMinKeys4 = 128;       // a CTA takes at least this many keys (one sequence of 1024, 2 KV heads: 8.6 us, 9.6 with 256)

// A warp has NV tiles of 8 query vectors. VG groups of warps share a tile's keys and have other vectors; FS
// warps share keys and vectors and have other features: they add their parts of the scores up through shared
// memory (at hd 256, where a warp with all features would have room for 8 vectors only, or convert twice).
template <int D, int NV, int VG, int FS>
struct Split4Cfg {
  static constexpr int THREADS = kWarps4 * 32 + 32;         // and the warp that copies
  static constexpr int KT = D == 256 ? 64 : 128;            // keys of a tile
  // Tiles that take as long as an item's start and join (3.3 us, a tile 1.3, at hd 128 and 4 vectors; 5.3 and 1.6 for 16
  // vectors at hd 256). Shares count them: the last CTA of 64 x 1024 .. 8192 keys ended at 80 us with tiles alone, half of the
  // others before 68; the call takes 83 us without, 80 / 78 / 79 with 2 / 3 / 4.
  static constexpr int START = FS == 2 && NV == 2 ? 4 : 3;
  static constexpr int CODES = KT * D / 2, SCALES = KT * D / 16, STAGE = 2 * (CODES + SCALES);
  static constexpr int ROWS = 8 * NV * VG;                  // query vectors
  static constexpr int DW = D / FS;                         // features of a warp
  static constexpr bool QS = NV * DW > 128;                 // Q^T waits in shared memory, not in registers
  // CTAs an SM: 96 registers a thread for four, 128 for three, 168 for two. All forms spill a little within these (16 to 164 bytes a
  // thread stored, 28 to 304 loaded); NV = 2 with 128 features spills more with 128: 16 vectors over 32 x 6144 keys, 8 KV
  // heads, 93 us with three, 85 with two
  static constexpr int CTAS = DW == 64 ? 5 - NV : 4 - NV;
  static constexpr int G = 2;                               // groups of 16 keys that a warp takes at a time (one: 64 x 1024 .. 8192
                                                            // keys, 4 vectors, hd 128, 89 us; two: 85)
  // V is loaded before S is computed where 16 vectors of half the features wait for the other half's S (drafts of
  // 16 vectors at hd 256: 66 us, after it 67; one vector at hd 128: 54 before it, 51 after)
  static constexpr bool V_FIRST = FS == 2 && NV == 2;
  // The warps of a group join their O in shared memory, in two rounds where one would take the stages' room
  static constexpr int JR = NV * D > 128 ? 2 : 1, JT = DW / 16 / JR, JROW = 16 * JT + 4;   // a vector's floats, and 4 apart
  static constexpr int JOIN = kWarps4 * 8 * NV * JROW * 4;
  static constexpr int QB = QS ? ROWS * D * 2 : 0;
  static constexpr int XB = FS > 1 ? 2 * kWarps4 * G * NV * 512 : 0;   // parts of scores, two rounds
  static constexpr int FIT = (226 * 1024 / CTAS - 1024 - JOIN - QB - XB - 128 - 1024) / STAGE;
  static constexpr int ST = FIT < 8 ? FIT : 8;
  static constexpr int SMEM = ST * STAGE + JOIN + QB + XB + 128;   // + alignment
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// c += a b (ZERO: c = a b)
template <bool ZERO>
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (ZERO)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Each byte's lower half from a, its upper half from b's lower half; and the upper halves alike
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u); }
template <int I>
__device__ __forceinline__ uint32_t codes_pair(const uint32_t* w) { return e2m1x2_f16x2<(I & 3)>(w[I >> 2]); }

template <int I, int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
  if constexpr (I < N) {
    f(Int<I>{});
    unrolled<I + 1, N>(f);
  }
}

// Part `part` of FS of one vector's features as the B operands of lane lt's columns (pairs of f16), scaled by the
// whole vector's largest value; the inverse scale is returned. By a whole warp.
template <int D, int FS>
__device__ __forceinline__ float load_query4(const Attend4Params& p, long long at, bool in, int lt, int part, uint32_t (&q)[D / FS / 16][2]) {
  constexpr int DW = D / FS, N = DW / 32;                   // 16-byte loads of a lane
  const uint16_t* const src = static_cast<const uint16_t*>(p.a.q) + at + lt * (8 * N);
  float top = 0.f;
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 w = in ? *reinterpret_cast<const uint4*>(src + c * DW + i * 8) : make_uint4(0, 0, 0, 0);
      q[2 * i][0] = w.x;
      q[2 * i][1] = w.y;
      q[2 * i + 1][0] = w.z;
      q[2 * i + 1][1] = w.w;
    }
  };
  auto each = [&](auto f) {
#pragma unroll
    for (int s = 0; s < DW / 16; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x, y;
        if (p.bf) unpack2(q[s][i], x, y, (const __nv_bfloat16*)nullptr);
        else unpack2(q[s][i], x, y, (const __half*)nullptr);
        f(q[s][i], x, y);
      }
  };
#pragma unroll
  for (int c = FS - 1; c >= 0; --c) {                       // its own part last
    fetch((part + c) % FS);
    each([&](uint32_t&, float x, float y) { top = fmaxf(top, fmaxf(fabsf(x), fabsf(y))); });
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  float inv;
  const float mul = query_scale(top, inv);
  each([&](uint32_t& w, float x, float y) { w = pack2(x * mul, y * mul, (const __half*)nullptr); });
  return inv;
}

__device__ __forceinline__ void store_four4(const Attend4Params& p, long long at, float x, float y, float z, float w) {
  if (p.a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) = make_float4(x, y, z, w);
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at) =
      p.bf ? make_uint2(pack2(x, y, (const __nv_bfloat16*)nullptr), pack2(z, w, (const __nv_bfloat16*)nullptr))
           : make_uint2(pack2(x, y, (const __half*)nullptr), pack2(z, w, (const __half*)nullptr));
}

// Tiles of one (sequence, KV head): none where the sequence has no rows or more query
// vectors than this kernel takes.
__device__ __forceinline__ Tiles4 split4_tiles(const PagedSeq& s, const Attend4Params& p, int kt) {
  if (s.t == 0 || (long long)s.t * p.a.hpg > p.a.most) return {0, 0, 0};
  return key_tiles(s, p, kt);
}

// REST: what the weights' rounding to f16 leaves enters the value product too, and a weight is off by 2^-22, not 2^-11. For
// results in f16 and f32: with one rounding 64 tokens (32 drafts of 4 under a window) in f16 were 2.33e-4 (2.36e-4) of
// the norm from 64 bits, with the rest 2.07e-4 (2.09e-4), as with weights of 32 bits. A result in bf16 is itself rounded
// by 2^-8, and is 1.65e-3 away in all of these.
//   1: in a second product with the same V. 64 x 1024 .. 8192 keys, 32 heads on 8: 78.6 -> 88.3 us; drafts 62.9 -> 72.8
//   2: up to four vectors: in the columns 4 .. 7 of the product, whose scores are those of columns 0 .. 3. 78.6 -> 81.3 us
// Blocks of 32 vectors, and the chunk kernel, round once: a second product would cost them more than that.
template <int D, int NV, int VG, int FS, int REST>
__global__ void __launch_bounds__(Split4Cfg<D, NV, VG, FS>::THREADS, Split4Cfg<D, NV, VG, FS>::CTAS)
    paged4_split_kernel(const __grid_constant__ Attend4Params p) {
  using C = Split4Cfg<D, NV, VG, FS>;
  constexpr int DW = C::DW, ST = C::ST, KT = C::KT, KS = DW / 16, NW = C::THREADS / 32, KG = kWarps4 / (VG * FS), SUBS = KT / 16 / KG, G = C::G;
  constexpr bool QS = C::QS;
  static_assert(SUBS % G == 0, "a warp's keys of a tile in whole turns");
  extern __shared__ unsigned char sm_raw[];
  __shared__ __align__(8) uint64_t b_full[ST], b_empty[ST];
  __shared__ longlong2 s_scan[NW];
  __shared__ long long s_off;
  __shared__ int s_b, s_abort;
  __shared__ float2 s_ml[kWarps4][8 * NV];
  __shared__ float s_shift[C::ROWS], s_inv[C::ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* const sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 127) & ~(uintptr_t)127);
  const uint32_t smb = smem_u32(sm);
  float* const join = reinterpret_cast<float*>(sm + ST * C::STAGE);
  uint2* const s_q = reinterpret_cast<uint2*>(sm + ST * C::STAGE + C::JOIN);   // [8-vector tile][step][lane]
  const uint32_t q_base = smb + ST * C::STAGE + C::JOIN + lane * 8;
  const PagedAttendParams& a = p.a;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], kWarps4);
    }
    mbar_fence_init();
    s_abort = 0;
    s_b = -1;
  }
  pdl_wait();
  pdl_trigger();

  // --- this CTA's share of all tiles: a scan over the sequences, of their tiles and of the items that have some
  uint32_t bits = 0;
  int weight = 0;                           // what an item's start costs, in tiles
  long long total = 0, per = 0;
  if (a.whole) {
    if (tid == 0) {
      const int b = blockIdx.x / a.map.nk;
      const int n = split4_tiles(paged_seq(a.map, b, a.T, a.max_rows, bits), p, KT).n;
      if (bits) set_err(a.err, bits);
      if (n > 0) s_b = b;
      s_off = (long long)(blockIdx.x % a.map.nk) * n;
      s_scan[0] = make_longlong2(n, 1);
    }
    __syncthreads();
    total = per = s_scan[0].x;
  } else {
    const int E = (a.map.B + C::THREADS - 1) / C::THREADS;
    longlong2 mine = make_longlong2(0, 0);
    for (int e = 0; e < E; ++e) {
      const int b = tid * E + e;
      const int n = b < a.map.B ? split4_tiles(paged_seq(a.map, b, a.T, a.max_rows, bits), p, KT).n : 0;
      mine.x += (long long)a.map.nk * n;
      mine.y += n > 0 ? a.map.nk : 0;
    }
    if (bits && blockIdx.x == 0) set_err(a.err, bits);
    longlong2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x += x;
        incl.y += y;
      }
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    longlong2 before = make_longlong2(incl.x - mine.x, incl.y - mine.y), sum = make_longlong2(0, 0);
    for (int w = 0; w < NW; ++w) {
      if (w < warp) {
        before.x += s_scan[w].x;
        before.y += s_scan[w].y;
      }
      sum.x += s_scan[w].x;
      sum.y += s_scan[w].y;
    }
    if (sum.x >= (long long)kWeighed * gridDim.x) weight = C::START;
    total = sum.x + weight * sum.y;
    per = max((total + gridDim.x - 1) / gridDim.x, (long long)(kMinKeys4 / KT));
    const long long at = per * blockIdx.x - (before.x + weight * before.y);
    if (at >= 0 && at < mine.x + weight * mine.y) {
      long long off = at;
      for (int e = 0; e < E; ++e) {
        const int b = tid * E + e;
        uint32_t ignore = 0;
        const int tiles = split4_tiles(paged_seq(a.map, b, a.T, a.max_rows, ignore), p, KT).n;
        const long long n = tiles ? (long long)a.map.nk * (tiles + weight) : 0;
        if (off < n) {
          s_b = b;
          s_off = off;
          break;
        }
        off -= n;
      }
    }
    __syncthreads();
  }
  const long long u0 = a.whole ? 0 : per * blockIdx.x, u1 = min(u0 + per, total);
  if (tid == 0 && !a.whole) a.ws_desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (s_b < 0) return;
  // the items of this share, walked by the copying warp and by the others alike
  int b = s_b;
  uint32_t ignore = 0;
  PagedSeq s = paged_seq(a.map, b, a.T, a.max_rows, ignore);
  Tiles4 tl = split4_tiles(s, p, KT);
  int g = (int)(s_off / (tl.n + weight));
  long long item = u0 - s_off % (tl.n + weight);            // its first unit
  // the tiles of the share in it: [tile0, tile1), none where the share ends in front of its first
  int tile0, tile1;
  auto tiles_of_item = [&]() {
    tile0 = (int)max(0LL, u0 - item - weight);
    tile1 = (int)max(0LL, min(u1 - item - weight, (long long)tl.n));
    return tile0 < tile1;
  };
  auto next_item = [&]() {                  // false at the end
    item += tl.n + weight;
    if (item >= u1) return false;
    if (++g == a.map.nk) {
      g = 0;
      do {
        s = paged_seq(a.map, ++b, a.T, a.max_rows, ignore);
        tl = split4_tiles(s, p, KT);
      } while (tl.n == 0);
    }
    return tiles_of_item();
  };
  if (!tiles_of_item() && !next_item()) return;
  if (warp == kWarps4) {
    // ------------------------------------------------------------ copies: a run of keys of one array a lane
    const int page = 1 << a.map.page_shift, rows = min(page, KT), runs = KT / rows;   // 4 * runs <= 32
    const int arr = lane / runs, run = lane % runs;      // 0: K codes, 1: V codes, 2: K scales, 3: V scales
    const bool mine = arr < 4, codes = arr < 2;
    const uint8_t* const src = arr == 0 ? p.c.k : arr == 1 ? p.c.v : arr == 2 ? p.c.ks : p.c.vs;
    const int row = codes ? D / 2 : D / 16;
    const int dst = (codes ? arr * C::CODES : 2 * C::CODES + (arr - 2) * C::SCALES) + run * rows * row;
    bool ok = true;
    int it = 0;                             // tiles of this share so far: stage it % ST
    do {
      const int32_t* table = a.map.table + (size_t)b * a.map.max_pages;
      for (int x = tile0; ok && x < tile1; ++x, ++it) {
        const int key = tl.at(x) * KT + run * rows, st = it % ST;
        const uint8_t* from = nullptr;
        bool blank = false;
        if (mine && key < s.len) {          // looked up before the wait
          const int id = table[key >> a.map.page_shift];
          if (page_ok(a.map, id)) {
            from = src + ((((long long)id * a.map.nk + g) << a.map.page_shift) + (key & (page - 1))) * row;
          } else {
            set_err(a.err, SWA_DERR_PAGE);
            blank = !codes;                 // such keys read as zeros: by their scales
          }
        }
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, from ? rows * row : 0);
        if (it >= ST) ok = __all_sync(0xffffffffu, tc_wait(&b_empty[st], (uint32_t)((it / ST - 1) & 1), &s_abort));
        if (!ok) break;
        if (blank) {
          for (int i = 0; i < rows * row; i += 16) *reinterpret_cast<uint4*>(sm + st * C::STAGE + dst + i) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();         // before a later copy into this stage
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&b_full[st], bytes);
        __syncwarp();
        if (from) bulk_g2s(sm + st * C::STAGE + dst, from, rows * row, &b_full[st]);
      }
      if (!ok || !next_item()) break;
    } while (true);
    if (!ok) {
      set_err(a.err, SWA_DERR_TIMEOUT);
      // copies in flight land before the CTA exits (bounded)
      for (int i = max(0, it - ST); i < it; ++i) mbar_wait_bounded(&b_full[i % ST], (uint32_t)((i / ST) & 1), kWaitLimitNs);
    }
    return;
  }

  // ------------------------------------------------------------ products
  const int lg = lane >> 2, lt = lane & 3, hpg = a.hpg, hpg_inv = 65536 / hpg + 1, fs = warp / KG % FS, vg = warp / (KG * FS);
  auto row_of = [&](int x) { return x * hpg_inv >> 16; };   // x / hpg (x < 32: a vector)
  // the key of the group's 16 that is row i of the products: lanes that read at the same time
  // then find rows of both parities, and fewer of them in the same banks
  auto key_of = [](int i) { return i ^ ((i >> 1) & 1); };
  bool ok = true;                           // a thread whose wait gave up goes on and writes nothing
  // FS = 2: where this warp's parts of scores go, those of the other one, and which of two rounds it is
  const uint32_t x_base = smb + ST * C::STAGE + C::JOIN + C::QB + lane * 16;
  const uint32_t x_mine = x_base + warp * (G * NV * 512), x_other = x_base + (warp ^ KG) * (G * NV * 512);
  uint32_t turn = 0;
  int st = 0;                               // the next tile's stage, and the parity of its barrier's phase
  uint32_t phase = 0;
  do {
    const int nvec = s.t * hpg;
    // --- Q^T as B operands in f16, each vector scaled by a power of two; scores' factors, limits
    uint32_t qf[QS ? 1 : NV][KS][2];
    float qm[NV][2];
    int lim[NV][2];
    auto query = [&](int tile, int part, uint32_t (&q)[KS][2]) {      // of 8 vectors; the inverse scale of vector lg
      const int r = REST == 2 ? lg & 3 : tile * 8 + lg;
      const bool in = r < nvec;
      const int i = in ? row_of(r) : 0, h = in ? r - i * hpg : 0;
      return load_query4<D, FS>(p, (long long)(s.r0 + i) * a.q_row + (long long)(g * hpg + h) * D, in, lt, part, q);
    };
    if constexpr (QS) {
      for (int x = warp; x < C::ROWS / 8 * FS; x += kWarps4) {
        const int tile = x / FS;
        const float shift = query(tile, x % FS, qf[0]);
        if (lt == 0) s_shift[tile * 8 + lg] = shift;        // (the same from every part)
#pragma unroll
        for (int i = 0; i < KS; ++i) s_q[(x * KS + i) * 32 + lane] = make_uint2(qf[0][i][0], qf[0][i][1]);
      }
      named_barrier(1, kWarps4 * 32);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float shift = 0.f;
      if constexpr (!QS) shift = query(vg * NV + v, fs, qf[v]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = REST == 2 ? 2 * (lt & 1) + e : (vg * NV + v) * 8 + 2 * lt + e;
        if constexpr (QS) shift = s_shift[c];
        qm[v][e] = fmaxf(a.qmul * (QS ? shift : __shfl_sync(0xffffffffu, shift, (2 * lt + e) * 4)), 0x1p-126f);   // masked scores stay -inf
        lim[v][e] = c < nvec ? max(0, min(s.len, s.len - s.t + row_of(c) + 1)) : 0;
      }
    }
    auto q_at = [&](int v, int i) {
      if constexpr (QS) {
        uint32_t w[2];
        lds_words<2>(w, q_base + (((vg * NV + v) * FS + fs) * KS + i) * 256);
        return make_uint2(w[0], w[1]);
      } else {
        return make_uint2(qf[v][i][0], qf[v][i][1]);
      }
    };
    const int lim_min = s.len - s.t + 1;                    // keys below it are before or at every row's own
    const int lo_min = first_key(lim_min, p.window), lo_max = first_key(s.len, p.window);   // the first and the last row's first key

    // off: kLog24 less the running maximum, once a key was seen; bar: the products above which it is raised
    float o[NV][KS][4], l[NV][2], off[NV][2], bar[NV][2];
    int seen[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[v][j][e] = 0.f;
      off[v][0] = off[v][1] = kLog24;
      bar[v][0] = bar[v][1] = -INFINITY;
      seen[v] = 0;
      l[v][0] = l[v][1] = 0.f;
    }

    // this lane's keys of 16 in S (ka and ka + 8) and in P V (k1, k2 and these + 8), and its places in a stage
    const int ka = key_of(lg), k1 = key_of(2 * lt), k2 = key_of(2 * lt + 1);
    constexpr int W = DW == 64 ? 2 : 4;                              // words of a key in S
    constexpr int VW = DW / 64;                                      // .. and in P V
    const uint32_t group0 = smb + (warp % KG) * SUBS * 16 * (D / 2) + fs * (DW / 2);
    const uint32_t scale0 = smb + 2 * C::CODES + (warp % KG) * SUBS * 16 * (D / 16) + fs * (DW / 16);
    const uint32_t at_k = group0 + ka * (D / 2) + lt * (W * 4), at_ks = scale0 + ka * (D / 16) + (DW == 64 ? lt : lt * 2);
    const uint32_t at_v1 = group0 + C::CODES + k1 * (D / 2) + lg * (VW * 4), at_v2 = at_v1 + (k2 - k1) * (D / 2);
    const uint32_t at_vs1 = scale0 + C::SCALES + k1 * (D / 16) + (DW == 64 ? lg >> 1 : lg);
    const uint32_t at_vs2 = at_vs1 + (k2 - k1) * (D / 16);
#pragma unroll 1
    for (int x = tile0; x < tile1; ++x) {
      ok &= tc_wait(&b_full[st], phase, &s_abort);
      __syncwarp();
#pragma unroll 1
      for (int sub = 0; sub < SUBS; sub += G) {             // this warp's keys, 16 G at a time
        const int k0 = tl.at(x) * KT + (warp % KG) * (SUBS * 16) + sub * 16;
        if (k0 >= s.len || (k0 + 16 * G <= lo_min && k0 >= p.sinks)) continue;
        const uint32_t codes = st * C::STAGE + sub * 16 * (D / 2), scales = st * C::STAGE + sub * 16 * (D / 16);
        const bool mask = __any_sync(0xffffffffu, k0 + 16 * G > lim_min || k0 < lo_max);   // a branch, not selects
        // V^T: keys 2 lt, 2 lt + 1 (+ 8) of the products' rows, features (hd / 8) lg ..; loaded and regrouped before
        // the weights are known
        uint32_t lo[G][2][VW], hi[G][2][VW], u1[G][2], u2[G][2];
        auto load_v = [&]() {
#pragma unroll
          for (int y = 0; y < G; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w1[VW], w2[VW];
              lds_words<VW>(w1, at_v1 + codes + (y * 16 + h * 8) * (D / 2));
              lds_words<VW>(w2, at_v2 + codes + (y * 16 + h * 8) * (D / 2));
#pragma unroll
              for (int w = 0; w < VW; ++w) {
                lo[y][h][w] = low_halves(w1[w], w2[w]);
                hi[y][h][w] = high_halves(w1[w], w2[w]);
              }
              u1[y][h] = lds_u8(at_vs1 + scales + (y * 16 + h * 8) * (D / 16));
              u2[y][h] = lds_u8(at_vs2 + scales + (y * 16 + h * 8) * (D / 16));
            }
        };
        if constexpr (C::V_FIRST) load_v();
        float sc[G][NV][4];
        // 4 features a step; the groups in turn, since a step's products wait for the step's before
        uint32_t wa[G][W], wc[G][W], sa[G][2], sb[G][2];   // codes of the two keys; a block's scale in both halves
#pragma unroll
        for (int y = 0; y < G; ++y) {
          lds_words<W>(wa[y], at_k + codes + y * 16 * (D / 2));
          lds_words<W>(wc[y], at_k + codes + (y * 16 + 8) * (D / 2));
          const uint32_t at = at_ks + scales + y * 16 * (D / 16);
          if constexpr (DW == 64) {
            sa[y][0] = e4m3x2_f16x2(lds_u8(at) * 0x0101u);
            sb[y][0] = e4m3x2_f16x2(lds_u8(at + 8 * (D / 16)) * 0x0101u);
          } else {
            const uint32_t ua = e4m3x2_f16x2(lds_u16(at)), uc = e4m3x2_f16x2(lds_u16(at + 8 * (D / 16)));
            sa[y][0] = __byte_perm(ua, ua, 0x1010);
            sa[y][1] = __byte_perm(ua, ua, 0x3232);
            sb[y][0] = __byte_perm(uc, uc, 0x1010);
            sb[y][1] = __byte_perm(uc, uc, 0x3232);
          }
        }
        unrolled<0, KS>([&](auto i) {
          constexpr int I = decltype(i)::value, B = DW == 64 ? 0 : I / 4;
#pragma unroll
          for (int y = 0; y < G; ++y) {
            const uint32_t f[4] = {hmul2(codes_pair<2 * I>(wa[y]), sa[y][B]), hmul2(codes_pair<2 * I>(wc[y]), sb[y][B]),
                                   hmul2(codes_pair<2 * I + 1>(wa[y]), sa[y][B]), hmul2(codes_pair<2 * I + 1>(wc[y]), sb[y][B])};
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const uint2 q = q_at(v, I);
              mma_f16<I == 0>(sc[y][v], f, q.x, q.y);
            }
          }
        });
        if constexpr (!C::V_FIRST) load_v();
        if constexpr (FS == 2) {            // the other features' part, added in the same order by both
#pragma unroll
          for (int y = 0; y < G; ++y)
#pragma unroll
            for (int v = 0; v < NV; ++v)
              sts_words(x_mine + turn + (y * NV + v) * 512, __float_as_uint(sc[y][v][0]), __float_as_uint(sc[y][v][1]),
                        __float_as_uint(sc[y][v][2]), __float_as_uint(sc[y][v][3]));
          named_barrier(2 + vg * KG + warp % KG, 64);
#pragma unroll
          for (int y = 0; y < G; ++y)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              uint32_t z[4];
              lds_words<4>(z, x_other + turn + (y * NV + v) * 512);
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[y][v][e] += __uint_as_float(z[e]);
            }
          turn ^= kWarps4 * G * NV * 512;
        }
        // masked scores: element e is (key row lg + 8 (e / 2), vector 2 lt + e % 2)
        if (mask) {
#pragma unroll
          for (int y = 0; y < G; ++y) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = k0 + y * 16 + ka + (e < 2 ? 0 : 8), top = lim[v][e & 1];
                if (key >= top || (key < top - p.window && key >= p.sinks)) sc[y][v][e] = -INFINITY;
              }
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // what no row sees may be NaN: zeros
              const int y1 = k0 + y * 16 + k1 + 8 * h, y2 = k0 + y * 16 + k2 + 8 * h;
              if (y1 >= s.len || (y1 < lo_min && y1 >= p.sinks)) u1[y][h] = 0;
              if (y2 >= s.len || (y2 < lo_min && y2 >= p.sinks)) u2[y][h] = 0;
            }
          }
        }
        auto top_of = [&](int v, int e) {
          float mx = fmaxf(sc[0][v][e], sc[0][v][e + 2]);
#pragma unroll
          for (int y = 1; y < G; ++y) mx = fmaxf(mx, fmaxf(sc[y][v][e], sc[y][v][e + 2]));
          return mx;
        };
        bool raise = false;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 2; ++e) raise |= top_of(v, e) > bar[v][e];
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = top_of(v, e);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              const float old = kLog24 - off[v][e], mn = fmaxf(seen[v] >> e & 1 ? old : -INFINITY, mx * qm[v][e]);
              if (mn == -INFINITY) continue;                // no key yet
              const float f = seen[v] >> e & 1 ? ex2(old - mn) : 0.f;
              seen[v] |= 1 << e;
              off[v][e] = kLog24 - mn;
              bar[v][e] = (mn + kLazy4) / qm[v][e];
              l[v][e] *= f;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                o[v][j][e] *= f;
                o[v][j][e + 2] *= f;
              }
            }
        }
        uint32_t pf[G][NV][2], pr[G][REST == 1 ? NV : 1][2], vs[G][2];
#pragma unroll
        for (int y = 0; y < G; ++y) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = ex2(fmaf(sc[y][v][i], qm[v][i & 1], off[v][i & 1]));
              l[v][i & 1] += e[i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w = pack2(e[2 * i], e[2 * i + 1], (const __half*)nullptr), rest = 0;
              if constexpr (REST > 0) {
                float h0, h1;
                unpack2(w, h0, h1, (const __half*)nullptr);
                rest = pack2(e[2 * i] - h0, e[2 * i + 1] - h1, (const __half*)nullptr);
              }
              if (REST == 2 && lt >= 2) w = rest;
              pf[y][v][i] = movmatrix(w);
              if constexpr (REST == 1) pr[y][v][i] = movmatrix(rest);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) vs[y][h] = e4m3x2_f16x2(__byte_perm(u1[y][h], u2[y][h], 0x0040));
        }
#pragma unroll
        for (int y = 0; y < G; ++y)
          unrolled<0, KS>([&](auto j) {
            constexpr int J = decltype(j)::value;
            const uint32_t f[4] = {hmul2(codes_pair<J>(lo[y][0]), vs[y][0]), hmul2(codes_pair<J>(hi[y][0]), vs[y][0]),
                                   hmul2(codes_pair<J>(lo[y][1]), vs[y][1]), hmul2(codes_pair<J>(hi[y][1]), vs[y][1])};
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              mma_f16<false>(o[v][J], f, pf[y][v][0], pf[y][v][1]);
              if constexpr (REST == 1) mma_f16<false>(o[v][J], f, pr[y][v][0], pr[y][v][1]);
            }
          });
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_empty[st]);
      if (++st == ST) {
        st = 0;
        phase ^= 1;
      }
    }

    // --- join the warps of a group: each scales its part to their maximum, then they are added up
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[v][e] += __shfl_xor_sync(0xffffffffu, l[v][e], d);
        if (lg == 0) s_ml[warp][v * 8 + 2 * lt + e] = make_float2(seen[v] >> e & 1 ? kLog24 - off[v][e] : -INFINITY, l[v][e]);
      }
    if constexpr (REST == 2) {              // the rest's columns join their vectors'
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][j][e] += __shfl_xor_sync(0xffffffffu, o[0][j][e], 2);
    }
    const bool whole = tile0 == 0 && tile1 == tl.n;
    // record of the item this CTA continues: slot 2c, of the one it starts: 2c + 1
    const size_t rec = ((size_t)blockIdx.x * 2 + (tile0 == 0 ? 1 : 0)) * p.rows;
    named_barrier(1, kWarps4 * 32);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = v * 8 + 2 * lt + e, pv = vg * (8 * NV) + c;
        float mt = -INFINITY, sum = 0.f, mine = 0.f;
#pragma unroll
        for (int w = 0; w < KG; ++w) mt = fmaxf(mt, s_ml[warp - warp % KG + w][c].x);
#pragma unroll
        for (int w = 0; w < KG; ++w) {
          const float2 ml = s_ml[warp - warp % KG + w][c];
          const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt + (p.rec_log2 - kLog24));
          sum += f * ml.y;
          if (w == warp % KG) mine = f * p.c.v_mul;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          o[v][j][e] *= mine;
          o[v][j][e + 2] *= mine;
        }
        if (lg > 0 || warp % (KG * FS)) continue;           // a lane for each vector
        s_inv[pv] = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // no key: zeros; NaN stays
        if (pv >= nvec || s_abort) continue;
        if (!whole) a.ws_ml[rec + pv] = make_float2(mt, sum);
        else if (a.lse)
          a.lse[(size_t)(s.r0 + row_of(pv)) * a.nh + g * hpg + pv - row_of(pv) * hpg] = sum == 0.f ? -INFINITY : (mt - p.rec_log2 + log2f(sum)) * 0.6931471805599453f;
      }
#pragma unroll
    for (int j0 = 0; j0 < KS; j0 += C::JT) {
      if (j0 > 0) named_barrier(1, kWarps4 * 32);           // the part before is read
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < C::JT; j += 2)
            *reinterpret_cast<float4*>(join + (warp * (8 * NV) + v * 8 + 2 * lt + e) * C::JROW + lg * (2 * C::JT) + 2 * j) =
                make_float4(o[v][j0 + j][e], o[v][j0 + j][e + 2], o[v][j0 + j + 1][e], o[v][j0 + j + 1][e + 2]);
      named_barrier(1, kWarps4 * 32);
      if (s_abort) continue;
      // four features of a vector at a time: in group y / .. , vector c of its own
      constexpr int QUADS = 4 * C::JT;
      for (int y = tid; y < C::ROWS * FS * QUADS; y += kWarps4 * 32) {
        const int quad = y % QUADS, c = y / QUADS % (8 * NV), gr = y / (QUADS * 8 * NV), pv = gr / FS * (8 * NV) + c;
        if (pv >= nvec) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KG; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(join + ((gr * KG + w) * (8 * NV) + c) * C::JROW + quad * 4);
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
        }
        const int f = gr % FS * DW + quad / (C::JT / 2) * (DW / 8) + 2 * j0 + quad % (C::JT / 2) * 4;
        if (whole) {
          const float inv = s_inv[pv];
          const bool none = inv == 0.f;
          store_four4(p, ((long long)(s.r0 + row_of(pv)) * a.nh + g * hpg + pv - row_of(pv) * hpg) * D + f, none ? 0.f : acc.x * inv, none ? 0.f : acc.y * inv,
                      none ? 0.f : acc.z * inv, none ? 0.f : acc.w * inv);
        } else {
          *reinterpret_cast<float4*>(a.ws_acc + (rec + pv) * D + f) = acc;
        }
      }
    }
    if (!whole && tile0 == 0 && tid == 0) a.ws_desc[blockIdx.x] = make_int4(s.r0, g, (int)((item + weight + tl.n - 1) / per), s.t);   // .. CTA that ends it
    if (!next_item()) break;
    named_barrier(1, kWarps4 * 32);         // s_ml and join are read
  } while (true);
  if (!ok) set_err(a.err, SWA_DERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// Keys that a row may see up to which a CTA takes a (sequence, KV head) whole: no scan over the
// sequences and no second kernel. By the table's width (or the window), since the lengths are the device's.
// Measured with one row of 8 vectors and one KV head, whole against cut, for 1, 16 and 64 sequences: 1024 keys at hd 128 9.6,
// 10.3, 10.4 us against 9.9, 10.6, 12.1; at hd 256 768 keys 14.7, 15.8, 15.7 against 11.7, 15.2, 17.3, 1024 keys 16.3, 18.8,
// 19.2 against 11.6, 15.2, 18.3. These are the GPU's times; called one by one from Python the cut form takes 19.
static long long whole_keys4(int hd) { return hd == 256 ? 768 : 1024; }

struct Split4Plan {
  int rows, vecs, whole, grid; // query vectors of a block (0: no sequence for this kernel), and those that sequences have at most
  size_t off_ml, off_desc, bytes;
};

template <int D, int NV, int VG, int FS>
static int split4_occupancy() {
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (!cache[dev]) {
    auto k = paged4_split_kernel<D, NV, VG, FS, 0>;   // (the other form has the same bounds)
    int n = 0;
    if (allow_smem<paged4_split_kernel<D, NV, VG, FS, 0>>(Split4Cfg<D, NV, VG, FS>::SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, Split4Cfg<D, NV, VG, FS>::THREADS, Split4Cfg<D, NV, VG, FS>::SMEM) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = 1;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

template <int D, int NV, int VG, int FS, int REST>
static int launch_split4(const Attend4Params& p, const Split4Plan& sp, cudaStream_t s) {
  const cudaError_t e = allow_smem<paged4_split_kernel<D, NV, VG, FS, REST>>(Split4Cfg<D, NV, VG, FS>::SMEM);
  if (e != cudaSuccess) return cuda_status(e);
  const int rc = finish_launch(launch_pdl(paged4_split_kernel<D, NV, VG, FS, REST>, dim3(sp.grid), dim3(Split4Cfg<D, NV, VG, FS>::THREADS),
                                          Split4Cfg<D, NV, VG, FS>::SMEM, s, p));
  if (rc != SWA_OK || p.a.whole) return rc;
  // a block a row up to 16, which then take rows in turn: most of sp.grid's columns are empty
  const long long vecs = (long long)p.a.max_rows * p.a.hpg;
  const dim3 grid(sp.grid, (unsigned)(vecs < 16 ? vecs : 16));
  return finish_launch(p.bf ? launch_pdl(paged_merge_kernel<__nv_bfloat16, D>, grid, dim3(kMergeThreads), 0, s, p.a, p.rows)
                            : launch_pdl(paged_merge_kernel<__half, D>, grid, dim3(kMergeThreads), 0, s, p.a, p.rows));
}

// rows: query vectors of a block, 8, 16 or 32 (hd 256: 8 or 16)
template <typename F>
static int by_size4(int hd, int rows, F f) {
  if (hd == 256) return rows == 8 ? f(Int<256>{}, Int<1>{}, Int<1>{}, Int<2>{}) : f(Int<256>{}, Int<2>{}, Int<1>{}, Int<2>{});
#define SWA_ROWS(D) \
  (rows == 8 ? f(Int<D>{}, Int<1>{}, Int<1>{}, Int<1>{}) : rows == 16 ? f(Int<D>{}, Int<2>{}, Int<1>{}, Int<1>{}) \
                                                                     : f(Int<D>{}, Int<2>{}, Int<2>{}, Int<1>{}))
  return hd == 64 ? SWA_ROWS(64) : SWA_ROWS(128);
#undef SWA_ROWS
}

// Query vectors of a (sequence, KV head) up to which the split kernel takes it: as many as its columns hold. (With
// that many over 32 x 4096 .. 8192 keys it takes 56 / 80 / 88 us at hd 64 / 128 / 256, the chunk kernel 131 / 164 / 261.)
static int split4_vecs(int hd) { return hd == 256 ? 16 : 32; }

static void split4_plan(const swa_paged4_attend_args* a, long long vecs, Split4Plan* sp) {
  const swa_paged4_cache& c = a->cache;
  *sp = Split4Plan{};
  sp->vecs = (int)vecs;
  sp->rows = vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
  long long keys = (long long)c.max_pages * c.page;
  if (a->window) {
    const long long w = (long long)a->window + a->sinks + a->max_rows + 256;
    keys = w < keys ? w : keys;
  }
  sp->whole = keys <= whole_keys4(c.hd);
  const int occ = sp->whole ? 0 : by_size4(c.hd, sp->rows, [](auto d, auto n, auto g, auto f) {
    return split4_occupancy<decltype(d)::value, decltype(n)::value, decltype(g)::value, decltype(f)::value>();
  });
  sp->grid = sp->whole ? c.B * c.nk : (num_sms() > 0 ? num_sms() : 148) * occ;
  if (!sp->whole) {
    const size_t recs = (size_t)sp->grid * 2 * sp->rows;
    sp->off_ml = up256s(recs * c.hd * sizeof(float));
    sp->off_desc = sp->off_ml + up256s(recs * sizeof(float2));
    sp->bytes = sp->off_desc + up256s((size_t)sp->grid * sizeof(int4));
  }
}

// Sizes alone (the workspace query); pointers are checked by the call.
static bool attend4_sizes_ok(const swa_paged4_attend_args* a) {
  const swa_paged4_cache& c = a->cache;
  if (c.B < 1 || c.B > 65535 || c.nk < 1 || c.nk > 65535 || (long long)c.B * c.nk > (1 << 24)) return false;
  if (c.hd != 64 && c.hd != 128 && c.hd != 256) return false;
  if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1))) return false;
  if (c.max_pages < 1 || c.max_pages > (1 << 30) / c.page) return false;
  if (a->T < 0 || a->max_rows < 1 || a->nh < 1 || a->nh % c.nk || a->nh / c.nk > 32) return false;
  if (a->window < 0 || a->sinks < 0 || (a->q_dtype != SWA_BF16 && a->q_dtype != SWA_F16)) return false;
  return (long long)a->T * a->nh < (1LL << 31) - 256;
}

// Which kernels a call runs. All sequences have at most max_rows rows (and T): when these fit
// the split kernel it runs alone. Otherwise the chunk kernel runs, and before it the split kernel if
// some sequence may be shorter (B * max_rows > T); if not, the chunk kernel takes every sequence.
struct Attend4Plan {
  Split4Plan split;
  ChunkPlan chunk;
  bool has_chunk;
  int most;                              // query vectors of a sequence up to which it is the split kernel's
  size_t off_chunk, bytes;
};

static void attend4_plan(const swa_paged4_attend_args* a, Attend4Plan* pl) {
  const int hpg = a->nh / a->cache.nk, max_rows = a->max_rows < a->T ? a->max_rows : a->T > 0 ? a->T : 1;
  const long long vecs = (long long)max_rows * hpg;
  *pl = Attend4Plan{};
  pl->has_chunk = vecs > split4_vecs(a->cache.hd);
  if (!pl->has_chunk || (long long)a->cache.B * max_rows > a->T) {
    pl->most = split4_vecs(a->cache.hd);
    split4_plan(a, vecs < pl->most ? vecs : pl->most, &pl->split);
  }
  pl->off_chunk = pl->bytes = pl->split.bytes;
  if (pl->has_chunk) {
    pl->chunk = chunk4_plan(a, max_rows);
    pl->bytes += pl->chunk.bytes;
  }
}

}  // namespace swa

using namespace swa;

extern "C" {

size_t swa_paged4_attend_workspace_size(const swa_paged4_attend_args* a) {
  if (!a || !attend4_sizes_ok(a)) return 0;
  Attend4Plan pl;
  attend4_plan(a, &pl);
  return pl.bytes ? pl.bytes : 1;
}

int swa_paged4_attend(const swa_paged4_attend_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged4_cache& c = a->cache;
  int rc = paged4_cache_status(&c);
  if (rc != SWA_OK) return rc;
  if (!attend4_sizes_ok(a) || !(a->scale >= 0.f) || std::isinf(a->scale)) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->q || !a->out) return SWA_E_NULL;
  const long long qn = rows_span(a->T, (long long)a->nh * c.hd, a->q_row);
  if (qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->q) || !aligned16p(a->out) || (a->q_row & 7) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
    return SWA_E_ALIGN;
  Attend4Plan pl;
  attend4_plan(a, &pl);
  if (pl.bytes && (!a->workspace || a->workspace_bytes < pl.bytes)) return SWA_E_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return SWA_E_ALIGN;
  const size_t rows = (size_t)a->T * a->nh, on = rows * c.hd * (a->out_f32 ? 4 : 2), ln = a->lse ? rows * 4 : 0;
  if (bytes_overlap(a->q, (size_t)qn * 2, a->out, on) ||
      (a->lse && (bytes_overlap(a->q, (size_t)qn * 2, a->lse, ln) || bytes_overlap(a->out, on, a->lse, ln))))
    return SWA_E_SHAPE;
  Attend4Params p{};
  PagedAttendParams& pa = p.a;
  pa.map = paged4_map(&c);
  pa.T = a->T; pa.nh = a->nh; pa.hpg = a->nh / c.nk; pa.max_rows = a->max_rows < a->T ? a->max_rows : a->T;
  pa.most = pl.most;
  p.c = paged4_pools(&c);
  pa.qmul = a->scale * 1.4426950408889634f * p.c.k_mul;
  pa.q = a->q; pa.q_row = a->q_row;
  pa.out = a->out; pa.out_f32 = a->out_f32 != 0; pa.lse = a->lse;
  pa.err = a->err;
  p.bf = a->q_dtype == SWA_BF16;
  constexpr int kAll = 1 << 30;                            // no sequence is longer
  p.window = a->window > 0 && a->window < kAll ? a->window : kAll;
  p.sinks = a->window == 0 ? 0 : a->sinks < kAll ? a->sinks : kAll;
  p.rec_log2 = p.bf ? PScale<__nv_bfloat16>::kLog2 : PScale<__half>::kLog2;
  char* ws = static_cast<char*>(a->workspace);
  cudaError_t e;
  if (a->ev_start && (e = cudaEventRecord(a->ev_start, stream)) != cudaSuccess) return cuda_status(e);
  if (pl.split.rows) {
    pa.whole = pl.split.whole;
    p.rows = pl.split.rows;
    pa.ws_acc = reinterpret_cast<float*>(ws);
    pa.ws_ml = reinterpret_cast<float2*>(ws + pl.split.off_ml);
    pa.ws_desc = reinterpret_cast<int4*>(ws + pl.split.off_desc);
    rc = by_size4(c.hd, pl.split.rows, [&](auto d, auto n, auto g, auto f) {
      constexpr int D = decltype(d)::value, NV = decltype(n)::value, VG = decltype(g)::value, FS = decltype(f)::value;
      if constexpr (NV * VG <= 2)
        if (!p.bf || pa.out_f32) {
          if constexpr (NV == 1)
            if (pl.split.vecs <= 4) return launch_split4<D, NV, VG, FS, 2>(p, pl.split, stream);
          return launch_split4<D, NV, VG, FS, 1>(p, pl.split, stream);
        }
      return launch_split4<D, NV, VG, FS, 0>(p, pl.split, stream);
    });
    if (rc != SWA_OK) return rc;
  }
  if (pl.has_chunk) {
    rc = launch_paged4_chunk(c.hd, p, pl.chunk, pl.split.rows ? pl.most : 0, ws + pl.off_chunk, stream);
    if (rc != SWA_OK) return rc;
  }
  if (a->ev_stop && (e = cudaEventRecord(a->ev_stop, stream)) != cudaSuccess) return cuda_status(e);
  return SWA_OK;
}

}  // extern "C"
