// Attention of a ragged chunk over the paged cache: the kernel for few query
// vectors per KV head (decode tokens, verify chunks), the merge of its partial
// records, and the host side of swa_paged_attend.
//
// A block of up to 64 query vectors (rows x heads of one KV head) needs 4 * 64 * hd
// operations for the 4 * hd bytes of a key: 64 a byte, far below the 280 a byte where
// the matrix peak meets the memory's. The kernel is bound by reading K and V once.
// So: every CTA gets the same number of 64-key tiles of the whole call (work of all
// sequences and KV heads laid end to end and cut evenly, wherever the cuts fall). One warp
// copies them from the pages by TMA, ahead across items; the others compute with warp-level
// mma.sync.m16n8k16: S = Q K^T with Q in registers, the online softmax on S's registers,
// and these registers again as the A operand of P V. A (sequence, KV head)
// that lies whole in one CTA is finished there; one that is cut leaves a
// record (m, l, sum p v) per CTA, joined by paged_merge_kernel.
// Measured, one token a sequence: 64 sequences of 1024 to 8192 keys, 16 query heads on 4,
// hd 128, bf16: 99 us, 6.0 TB/s; 16 of 32768 to 131072 keys, 8 heads on 2, hd 256, f16:
// 410 us, 7.0 TB/s (ncu: 89 % of the DRAM's peak, 1.001 times the bytes of K and V).
#include <cmath>

#include "swa_mma16.cuh"
#include "swa_paged_merge.cuh"
#include "swa_paged_tc.cuh"

namespace swa {

// ---------------------------------------------------------------------------
// Host checks shared by the paged calls
// ---------------------------------------------------------------------------
bool bytes_overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

int paged_cache_status(const swa_paged_cache* c, bool rows) {
  if (!c->k || !c->v || !c->table || !c->lens || (rows && !c->row_start)) return SWA_E_NULL;
  if (c->B < 1 || c->B > 65535 || c->nk < 1 || c->nk > 65535 || (long long)c->B * c->nk > (1 << 24)) return SWA_E_SHAPE;
  if (c->hd != 64 && c->hd != 128 && c->hd != 256) return SWA_E_SHAPE;
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return SWA_E_SHAPE;
  if (c->num_pages < 1 || (long long)c->num_pages * c->nk >= (1LL << 31) / c->page) return SWA_E_SHAPE;
  if (c->max_pages < 1 || c->max_pages > (1 << 30) / c->page) return SWA_E_SHAPE;
  if (c->dtype != SWA_BF16 && c->dtype != SWA_F16) return SWA_E_SHAPE;
  if (!aligned16p(c->k) || !aligned16p(c->v) || (reinterpret_cast<uintptr_t>(c->table) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->row_start) & 3u) || (reinterpret_cast<uintptr_t>(c->lens) & 3u))
    return SWA_E_ALIGN;
  return SWA_OK;
}

PagedMap paged_map(const swa_paged_cache* c) {
  PagedMap m{};
  m.B = c->B; m.nk = c->nk; m.num_pages = c->num_pages; m.max_pages = c->max_pages;
  while ((1 << m.page_shift) < c->page) ++m.page_shift;
  m.cap = c->max_pages << m.page_shift;
  m.table = c->table; m.row_start = c->row_start; m.lens = c->lens;
  return m;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of 16-bit elements, 128-byte swizzle, zeros out of range; dims, strides (in
// bytes, from the second dimension on) and box by rank.
static int tensor_map(int dtype, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                      const cuuint32_t* box, CUtensorMap* m) {
  static EncodeTiled encode = nullptr;
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult st;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st);
    if (e != cudaSuccess) return cuda_status(e);
    if (st != cudaDriverEntryPointSuccess || !f) return cuda_status(cudaErrorNotSupported);
    encode = reinterpret_cast<EncodeTiled>(f);
  }
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = encode(m, dtype == SWA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SWA_OK : cuda_status(cudaErrorInvalidValue);
}

// Tensor map of a pool: rows of hd elements, boxes of 64 features x min(page, KT) rows.
int pool_map(const swa_paged_cache& c, void* base, int kt, CUtensorMap* m) {
  const cuuint64_t dims[2] = {(cuuint64_t)c.hd, (cuuint64_t)c.num_pages * c.nk * c.page};
  const cuuint64_t strides[1] = {(cuuint64_t)c.hd * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)(c.page < kt ? c.page : kt)};
  return tensor_map(c.dtype, base, 2, dims, strides, box, m);
}

int rows_map(const swa_paged_cache& c, const void* q, int T, int nh, long long row, int heads, int rows, CUtensorMap* m) {
  const cuuint64_t dims[3] = {(cuuint64_t)c.hd, (cuuint64_t)nh, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)c.hd * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  return tensor_map(c.dtype, q, 3, dims, strides, box, m);
}

// ---------------------------------------------------------------------------
// The split kernel
// ---------------------------------------------------------------------------
constexpr int kKeys = 64;            // keys per tile
constexpr int kMinTiles = 2;         // a CTA takes at least this many tiles

template <int D>
struct SplitCfg {
  // Four warps share a tile's rows and keys. At hd 256 two warps split the value product
  // of each (and repeat its scores): with one warp a scheduler the chain of dependent
  // products bounds it (3.2 instead of 4.9 TB/s).
  static constexpr int DS = D == 256 ? 2 : 1;
  static constexpr int THREADS = 4 * DS * 32 + 32;          // and the warp that copies
  // stages of one K and one V tile: 96 KB (two CTAs an SM) at hd 128
  static constexpr int ST = D == 64 ? 4 : 3;
  static constexpr int TILE = kKeys * D * 2;
  static constexpr int CW = 32;                             // columns of O a warp joins at a time
  static constexpr int SMEM = ST * 2 * TILE + 4 * DS * 16 * CW * 4 + 1024;
};

// Tiles of one (sequence, KV head): none where the sequence has no rows or more query
// vectors than this kernel takes.
__device__ __forceinline__ int split_tiles(const PagedSeq& s, const PagedAttendParams& p) {
  if (s.t == 0 || (long long)s.t * p.hpg > p.most) return 0;
  return s.len > 0 ? (s.len + kKeys - 1) / kKeys : 1;      // a row without keys is still written
}

// ROWS: query vectors of a CTA's block (16, 32 or 64): ROWS / 16 groups of 16 rows,
// the other warps take the tile's keys in turn.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(SplitCfg<D>::THREADS)
    paged_split_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ PagedAttendParams p) {
  using C = SplitCfg<D>;
  constexpr int RG = ROWS / 16, KG = 4 / RG, KW = kKeys / KG;   // row groups, key groups, keys of a warp
  constexpr int DS = C::DS, DV = D / DS, ST = C::ST, CW = C::CW, NWARPS = C::THREADS / 32;
  // Weights are rounded to T for the value product. A block of 16 vectors adds what the rounding
  // leaves, in a second product with the same V registers: the weight is then off by 2^-16 (f16:
  // 2^-22) at most. It is bound by memory and pays 1 % (64 tokens as above: 98.6 and 99.8 us);
  // wider blocks, whose warps are busy, would pay more: 4 % with 32 vectors over 32768 keys, 10 %
  // with unequal rows and 20 % in a call that mixes 63 tokens with a prompt.
  constexpr bool REST = ROWS == 16;
  extern __shared__ unsigned char sm_raw[];
  __shared__ __align__(8) uint64_t b_full[ST], b_empty[ST];   // modelled in tests/test_paged_barriers_cpu.py
  __shared__ long long s_scan[NWARPS];
  __shared__ long long s_off, s_total;
  __shared__ int s_b, s_abort;
  __shared__ float2 s_ml[4][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* const sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  float* const ob = reinterpret_cast<float*>(sm + ST * 2 * C::TILE);   // [4 * DS warps][16][CW]
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 4 * DS);
    }
    mbar_fence_init();
    s_abort = 0;
    s_b = -1;
  }
  pdl_wait();
  pdl_trigger();

  // --- this CTA's share of all tiles: a scan over the sequences
  uint32_t bits = 0;
  if (p.whole) {
    if (tid == 0) {
      const int b = blockIdx.x / p.map.nk;
      const int n = split_tiles(paged_seq(p.map, b, p.T, p.max_rows, bits), p);
      if (bits) set_err(p.err, bits);
      if (n > 0) s_b = b;
      s_off = (long long)(blockIdx.x % p.map.nk) * n;
      s_total = n;
    }
    __syncthreads();
  } else {
    const int E = (p.map.B + C::THREADS - 1) / C::THREADS;
    long long mine = 0;
    for (int e = 0; e < E; ++e) {
      const int b = tid * E + e;
      if (b < p.map.B) mine += (long long)p.map.nk * split_tiles(paged_seq(p.map, b, p.T, p.max_rows, bits), p);
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
    for (int w = 0; w < NWARPS; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    long long per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinTiles) per = kMinTiles;
    const long long u0 = per * blockIdx.x;
    if (u0 >= before && u0 < before + mine) {
      long long off = u0 - before;
      for (int e = 0; e < E; ++e) {
        const int b = tid * E + e;
        uint32_t ignore = 0;
        const long long n = (long long)p.map.nk * split_tiles(paged_seq(p.map, b, p.T, p.max_rows, ignore), p);
        if (off < n) {
          s_b = b;
          s_off = off;
          break;
        }
        off -= n;
      }
    }
    if (tid == 0) s_total = total;
    __syncthreads();
  }
  const long long total = s_total;
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMinTiles) per = kMinTiles;
  if (p.whole) per = total;
  const long long u0 = p.whole ? 0 : per * blockIdx.x;
  if (tid == 0 && !p.whole) p.ws_desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (s_b < 0) return;
  // the items of this share, walked by the copying warp and by the others alike
  long long left = min(per, total - u0);
  int b = s_b;
  uint32_t ignore = 0;
  PagedSeq s = paged_seq(p.map, b, p.T, p.max_rows, ignore);
  int n_tiles = split_tiles(s, p);
  int tile0 = (int)(s_off % n_tiles), g = (int)(s_off / n_tiles);
  auto next_item = [&](int tile1) {         // false at the end
    left -= tile1 - tile0;
    tile0 = 0;
    if (left <= 0) return false;
    if (++g == p.map.nk) {
      g = 0;
      do {
        s = paged_seq(p.map, ++b, p.T, p.max_rows, ignore);
        n_tiles = split_tiles(s, p);
      } while (n_tiles == 0);
    }
    return true;
  };
  const uint32_t smb = smem_u32(sm);
  int it = 0;                               // tiles of this share so far: stage it % ST

  if (warp == NWARPS - 1) {
    // ------------------------------------------------------------ copies: a box a lane
    constexpr int HALVES = D / 64;
    const int page = 1 << p.map.page_shift, rows = min(page, kKeys), per_half = kKeys / rows;
    const int boxes = per_half * HALVES;    // of K, and as many of V: 32 at most together
    const int oob = p.map.num_pages * p.map.nk << p.map.page_shift;       // rows of the pool: reads zeros
    const bool mine = lane < 2 * boxes, is_v = lane >= boxes;
    const int box = is_v ? lane - boxes : lane, half = box / per_half, bx = box % per_half;
    bool ok = true;
    do {
      const int tile1 = (int)min((long long)n_tiles, tile0 + left);
      const int32_t* table = p.map.table + (size_t)b * p.map.max_pages;
      for (int tile = tile0; ok && tile < tile1; ++tile, ++it) {
        const int key = tile * kKeys + bx * rows, st = it % ST;
        int y = oob;
        if (mine && key < s.len) {          // looked up before the wait
          const int id = table[key >> p.map.page_shift];
          if (page_ok(p.map, id))
            y = ((id * p.map.nk + g) << p.map.page_shift) + (key & (page - 1));
          else
            set_err(p.err, SWA_DERR_PAGE);
        }
        if (it >= ST) ok = __all_sync(0xffffffffu, tc_wait(&b_empty[st], (uint32_t)((it / ST - 1) & 1), &s_abort));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&b_full[st], 2 * C::TILE);
        __syncwarp();
        if (mine)
          tma_2d(smb + (st * 2 + (is_v ? 1 : 0)) * C::TILE + half * (kKeys * 128) + bx * rows * 128, is_v ? &map_v : &map_k,
                 half * 64, y, &b_full[st]);
      }
      if (!ok || !next_item(tile1)) break;
    } while (true);
    if (!ok) {
      set_err(p.err, SWA_DERR_TIMEOUT);
      // copies in flight land before the CTA exits (bounded)
      for (int i = max(0, it - ST); i < it; ++i) mbar_wait_bounded(&b_full[i % ST], (uint32_t)((i / ST) & 1), kWaitLimitNs);
    }
    return;
  }

  // ------------------------------------------------------------ products
  const int ds = warp >> 2, rg = (warp & 3) / KG, kg = (warp & 3) % KG;
  const int hpg = p.hpg;
  const T* const qp = static_cast<const T*>(p.q);
  bool ok = true;                           // a thread whose wait gave up goes on and writes nothing
  // 16-byte chunk c of row r of a tile: halves of 64 features, rows of 128 bytes, swizzled
  auto at = [](int r, int c) { return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
  do {
    const int tile1 = (int)min((long long)n_tiles, tile0 + left);
    const int nvec = s.t * hpg;
    // --- Q of this warp's 16 rows as A operands; the rows' limits
    uint32_t qf[D / 16][4];
    int lim[2];
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int r = rg * 16 + hrow * 8 + (lane >> 2);
      const bool in = r < nvec;
      const int i = in ? r / hpg : 0, h = in ? r % hpg : 0;
      lim[hrow] = in ? min(s.len, s.len - s.t + i + 1) : 0;
      const T* src = qp + (size_t)(s.r0 + i) * p.q_row + (size_t)(g * hpg + h) * D + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][hrow] = in ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
        qf[k][hrow + 2] = in ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
      }
    }
    const int lim_min = s.len - s.t + 1;                    // keys below it are seen by every row

    float o[DV / 8][4];
#pragma unroll
    for (int i = 0; i < DV / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int tile = tile0; tile < tile1; ++tile, ++it) {
      const int st = it % ST;
      ok &= tc_wait(&b_full[st], (uint32_t)((it / ST) & 1), &s_abort);
      __syncwarp();
      const uint32_t kb = smb + (uint32_t)(st * 2 * C::TILE), vb = kb + C::TILE;
      const int k0 = tile * kKeys + kg * KW;
      const bool tail = tile * kKeys + kKeys > s.len;
      if (tail) {                           // V behind the last key: zeros (0 * NaN)
        const int first = max(0, s.len - k0);
        for (int x = lane; x < (KW - first) * (DV / 8); x += 32) {
          const int r = kg * KW + first + x / (DV / 8), c = ds * (DV / 8) + x % (DV / 8);
          *reinterpret_cast<uint4*>(sm + (st * 2 + 1) * C::TILE + at(r, c)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();           // before the copy that comes next into this stage
        __syncwarp();
      }

      float sc[KW / 8][4];
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int n = 0; n < KW / 16; ++n) {
          uint32_t f[4];
          ldsm4(f, kb + at(kg * KW + n * 16 + ((lane >> 4) << 3) + (lane & 7), k * 2 + ((lane >> 3) & 1)));
          mma16816<T>(sc[2 * n], qf[k], f[0], f[1]);
          mma16816<T>(sc[2 * n + 1], qf[k], f[2], f[3]);
        }
      }
      // scores in log2 units, masked
      const bool mask = tile * kKeys + kKeys > lim_min;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < KW / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = sc[n][j] * p.qmul;
          if (mask && k0 + n * 8 + (lane & 3) * 2 + (j & 1) >= lim[j >> 1]) x = -INFINITY;
          sc[n][j] = x;
          mx[j >> 1] = fmaxf(mx[j >> 1], x);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {   // else nothing to rescale
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = fmaxf(m[r], mx[r]);
          const float a = mn == -INFINITY ? 1.f : ex2(m[r] - mn);    // m = -inf: 0
          m[r] = mn;
          l[r] *= a;
#pragma unroll
          for (int i = 0; i < DV / 8; ++i) {
            o[i][2 * r] *= a;
            o[i][2 * r + 1] *= a;
          }
        }
      }
      float off[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) off[r] = PScale<T>::kLog2 - (m[r] == -INFINITY ? 0.f : m[r]);
#pragma unroll
      for (int n = 0; n < KW / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[n][j] = ex2(sc[n][j] + off[j >> 1]);
          l[j >> 1] += sc[n][j];
        }
#pragma unroll
      for (int n = 0; n < KW / 16; ++n) {
        uint32_t pa[4], pr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e0 = sc[2 * n + (j >> 1)][2 * (j & 1)], e1 = sc[2 * n + (j >> 1)][2 * (j & 1) + 1];
          pa[j] = pack2(e0, e1, (const T*)nullptr);
          if constexpr (REST) {
            float h0, h1;
            unpack2(pa[j], h0, h1, (const T*)nullptr);
            pr[j] = pack2(e0 - h0, e1 - h1, (const T*)nullptr);
          }
        }
#pragma unroll
        for (int dd = 0; dd < DV / 16; ++dd) {
          uint32_t f[4];
          ldsm4t(f, vb + at(kg * KW + n * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), ds * (DV / 8) + dd * 2 + (lane >> 4)));
          mma16816<T>(o[2 * dd], pa, f[0], f[1]);
          mma16816<T>(o[2 * dd + 1], pa, f[2], f[3]);
          if constexpr (REST) {
            mma16816<T>(o[2 * dd], pr, f[0], f[1]);
            mma16816<T>(o[2 * dd + 1], pr, f[2], f[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_empty[st]);
    }

    // --- join the key groups, CW columns of each warp's O at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (ds == 0 && (lane & 3) == 0) s_ml[warp][r * 8 + (lane >> 2)] = make_float2(m[r], l[r]);
    }
    const bool whole = tile0 == 0 && tile1 == n_tiles;
    // record of the item this CTA continues: slot 2c, of the one it starts: 2c + 1
    const size_t rec = ((size_t)blockIdx.x * 2 + (tile0 == 0 ? 1 : 0)) * ROWS;
#pragma unroll
    for (int c0 = 0; c0 < DV; c0 += CW) {
      if (c0 > 0) named_barrier(1, 4 * DS * 32);            // the columns before are read
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < CW / 8; ++i)
          *reinterpret_cast<float2*>(ob + (warp * 16 + r * 8 + (lane >> 2)) * CW + i * 8 + (lane & 3) * 2) =
              make_float2(o[c0 / 8 + i][2 * r], o[c0 / 8 + i][2 * r + 1]);
      named_barrier(1, 4 * DS * 32);
      if (s_abort) continue;
      for (int x = tid; x < nvec * DS * (CW / 8); x += 4 * DS * 32) {
        const int row = x / (DS * (CW / 8)), cc = x % (DS * (CW / 8)), d = cc / (CW / 8), c = cc % (CW / 8);
        const int w0 = (row >> 4) * KG, rr = row & 15, col = d * DV + c0 + c * 8;
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < KG; ++w) mt = fmaxf(mt, s_ml[w0 + w][rr].x);
        float lt = 0.f, acc[8] = {};
#pragma unroll
        for (int w = 0; w < KG; ++w) {
          const float2 ml = s_ml[w0 + w][rr];
          const float a = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt);
          float y[8];
          load8(ob + ((d * 4 + w0 + w) * 16 + rr) * CW + c * 8, y);
          lt += a * ml.y;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += a * y[j];
        }
        if (whole) {
          paged_store_row<T>(p, s.r0 + row / hpg, g * hpg + row % hpg, D, col, mt, lt, PScale<T>::kLog2, acc, col == 0);
        } else {
          store8(p.ws_acc + (rec + row) * D + col, acc);
          if (col == 0) p.ws_ml[rec + row] = make_float2(mt, lt);
        }
      }
    }
    if (!whole && tile0 == 0 && tid == 0) {
      // units of this item from here on / per CTA: the CTA that ends it
      const long long end = u0 + (min(per, total - u0) - left) + n_tiles - 1;
      p.ws_desc[blockIdx.x] = make_int4(s.r0, g, (int)(end / per), s.t);
    }
    if (!next_item(tile1)) break;
    named_barrier(1, 4 * DS * 32);          // s_ml and ob are read
  } while (true);
  if (!ok) set_err(p.err, SWA_DERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// Query vectors of a (sequence, KV head) up to which the split kernel takes it; more go
// to the tensor-core kernel (swa_paged_chunk.cu). 32 sequences of 2048 keys, 8 KV heads, split and
// tensor-core kernel: 32 vectors at hd 64 45 and 45 us, at hd 128 64 and 56, 48 vectors 59 and 45,
// 82 and 57; at hd 256 20 vectors 155 and 93 us. One sequence of 32768 keys, 32 vectors: hd 64 30
// and 32 us, hd 128 41 and 45; 8 ragged ones: 24 and 26, 29 and 30. So at hd 128 the rule costs a
// batch of 17 to 32 vectors an eighth and gains a single sequence a tenth: it does not look at the
// batch, because the lengths that would tell are the device's. Where sequences have unequal
// rows (B * max_rows > T) both kernels may have to run, one after the other, so up to 64 stay with
// one: 26 sequences of up to 22 rows over 18 to 4453 keys, 6 heads on 3, hd 128: 48 instead of 75 us
// (hd 256, 8 of up to 29 rows over 323 to 15713 keys: 99 instead of 56, so 16 there all the same).
// The block is then 64 vectors wide for single tokens too: 63 of them and a prompt of 512 rows, over
// 4096 keys each, 32 heads on 8, hd 128, take 286 us, apart 187 and 45.
static int split_vecs(const swa_paged_attend_args* a, int max_rows) {
  return a->cache.hd == 256 ? 16 : (long long)a->cache.B * max_rows > a->T ? 64 : 32;
}

// Keys of a sequence up to which a CTA takes a (sequence, KV head) whole: no scan over the
// sequences and no second kernel. By the table's width, since the lengths are the device's: one
// token over 133 keys takes 10.3 us in a table of 144 and 14.7 in one of 4608.
constexpr int kWholeKeys = 512;

struct SplitPlan {
  int rows, whole, grid;                 // query vectors of a block (16, 32 or 64; 0: no sequence for this kernel), CTAs
  size_t off_ml, off_desc, bytes;
};

template <typename T, int D, int ROWS>
static int split_occupancy() {
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (!cache[dev]) {
    auto k = paged_split_kernel<T, D, ROWS>;
    int n = 0;
    if (allow_smem<paged_split_kernel<T, D, ROWS>>(SplitCfg<D>::SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, SplitCfg<D>::THREADS, SplitCfg<D>::SMEM) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = 1;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

template <typename T, int D, int ROWS>
static int launch_split(const swa_paged_cache& c, const PagedAttendParams& p, const SplitPlan& sp, cudaStream_t s) {
  CUtensorMap mk, mv;
  int rc = pool_map(c, c.k, kKeys, &mk);
  if (rc == SWA_OK) rc = pool_map(c, c.v, kKeys, &mv);
  if (rc != SWA_OK) return rc;
  const cudaError_t e = allow_smem<paged_split_kernel<T, D, ROWS>>(SplitCfg<D>::SMEM);
  if (e != cudaSuccess) return cuda_status(e);
  rc = finish_launch(launch_pdl(paged_split_kernel<T, D, ROWS>, dim3(sp.grid), dim3(SplitCfg<D>::THREADS),
                                SplitCfg<D>::SMEM, s, mk, mv, p));
  if (rc != SWA_OK || p.whole) return rc;
  // a block a row up to 16, which then take rows in turn: most of sp.grid's columns are empty
  const long long vecs = (long long)p.max_rows * p.hpg;
  return finish_launch(launch_pdl(paged_merge_kernel<T, D>, dim3(sp.grid, (unsigned)(vecs < 16 ? vecs : 16)),
                                  dim3(kMergeThreads), 0, s, p, ROWS));
}

template <typename F>
static int by_type(int dtype, int hd, int rows, F f) {
#define SWA_ROWS(T, D) (rows == 16 ? f((T*)nullptr, Int<D>{}, Int<16>{}) : rows == 32 ? f((T*)nullptr, Int<D>{}, Int<32>{}) \
                                                                                    : f((T*)nullptr, Int<D>{}, Int<64>{}))
#define SWA_HD(T) (hd == 64 ? SWA_ROWS(T, 64) : hd == 128 ? SWA_ROWS(T, 128) : f((T*)nullptr, Int<256>{}, Int<16>{}))
  return dtype == SWA_BF16 ? SWA_HD(__nv_bfloat16) : SWA_HD(__half);
#undef SWA_HD
#undef SWA_ROWS
}

// Which kernels a call runs. All sequences have at most max_rows rows (and T): when these fit
// the split kernel it runs alone. Otherwise the tensor-core kernel runs, and before it
// the split kernel if some sequence may be shorter (B * max_rows > T); if not, the
// tensor-core kernel takes every sequence.
struct PagedPlan {
  SplitPlan split;
  ChunkPlan chunk;
  bool has_chunk;
  int most;                              // query vectors of a sequence up to which it is the split kernel's
  size_t off_chunk, bytes;
};

static void attend_plan(const swa_paged_attend_args* a, PagedPlan* pl) {
  const int hpg = a->nh / a->cache.nk, max_rows = a->max_rows < a->T ? a->max_rows : a->T > 0 ? a->T : 1;
  const long long vecs = (long long)max_rows * hpg;
  SplitPlan& sp = pl->split;
  sp = SplitPlan{};
  pl->most = split_vecs(a, max_rows);
  pl->has_chunk = vecs > pl->most;
  if (!pl->has_chunk || (long long)a->cache.B * max_rows > a->T) {
    const long long v = vecs < pl->most ? vecs : pl->most;
    sp.rows = v <= 16 ? 16 : v <= 32 ? 32 : 64;
    sp.whole = (long long)a->cache.max_pages * a->cache.page <= kWholeKeys;
    const int occ = sp.whole ? 0 : by_type(a->cache.dtype, a->cache.hd, sp.rows, [](auto* t, auto d, auto r) {
      return split_occupancy<std::remove_pointer_t<decltype(t)>, decltype(d)::value, decltype(r)::value>();
    });
    sp.grid = sp.whole ? a->cache.B * a->cache.nk : (num_sms() > 0 ? num_sms() : 148) * occ;
    if (!sp.whole) {
      const size_t recs = (size_t)sp.grid * 2 * sp.rows;
      sp.off_ml = up256s(recs * a->cache.hd * sizeof(float));
      sp.off_desc = sp.off_ml + up256s(recs * sizeof(float2));
      sp.bytes = sp.off_desc + up256s((size_t)sp.grid * sizeof(int4));
    }
  }
  pl->off_chunk = sp.bytes;
  pl->bytes = sp.bytes;
  if (pl->has_chunk) {
    pl->chunk = chunk_plan(a, max_rows);
    pl->bytes += pl->chunk.bytes;
  }
}

// Sizes alone (the workspace query); pointers are checked by the call.
static bool attend_sizes_ok(const swa_paged_attend_args* a) {
  const swa_paged_cache& c = a->cache;
  if (c.B < 1 || c.B > 65535 || c.nk < 1 || c.nk > 65535 || (long long)c.B * c.nk > (1 << 24)) return false;
  if ((c.hd != 64 && c.hd != 128 && c.hd != 256) || (c.dtype != SWA_BF16 && c.dtype != SWA_F16)) return false;
  if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1))) return false;
  if (c.max_pages < 1 || c.max_pages > (1 << 30) / c.page) return false;
  if (a->T < 0 || a->max_rows < 1 || a->nh < 1 || a->nh % c.nk || a->nh / c.nk > 32) return false;
  return (long long)a->T * a->nh < (1LL << 31) - 256;
}

}  // namespace swa

using namespace swa;

extern "C" {

size_t swa_paged_attend_workspace_size(const swa_paged_attend_args* a) {
  if (!a || !attend_sizes_ok(a)) return 0;
  PagedPlan pl;
  attend_plan(a, &pl);
  return pl.bytes ? pl.bytes : 1;
}

int swa_paged_attend(const swa_paged_attend_args* a, cudaStream_t stream) {
  if (!a) return SWA_E_NULL;
  const swa_paged_cache& c = a->cache;
  int rc = paged_cache_status(&c, true);
  if (rc != SWA_OK) return rc;
  if (!attend_sizes_ok(a) || !(a->scale >= 0.f) || std::isinf(a->scale)) return SWA_E_SHAPE;
  if (a->T == 0) return SWA_OK;
  if (!a->q || !a->out) return SWA_E_NULL;
  const long long qn = rows_span(a->T, (long long)a->nh * c.hd, a->q_row);
  if (qn < 0) return SWA_E_SHAPE;
  if (!aligned16p(a->q) || !aligned16p(a->out) || (a->q_row & 7) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
    return SWA_E_ALIGN;
  PagedPlan pl;
  attend_plan(a, &pl);
  if (pl.bytes && (!a->workspace || a->workspace_bytes < pl.bytes)) return SWA_E_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return SWA_E_ALIGN;
  const size_t rows = (size_t)a->T * a->nh, on = rows * c.hd * (a->out_f32 ? 4 : 2), ln = a->lse ? rows * 4 : 0;
  if (bytes_overlap(a->q, (size_t)qn * 2, a->out, on) ||
      (a->lse && (bytes_overlap(a->q, (size_t)qn * 2, a->lse, ln) || bytes_overlap(a->out, on, a->lse, ln))))
    return SWA_E_SHAPE;
  PagedAttendParams p{};
  p.map = paged_map(&c);
  p.T = a->T; p.nh = a->nh; p.hpg = a->nh / c.nk; p.max_rows = a->max_rows < a->T ? a->max_rows : a->T;
  p.most = pl.most;
  p.qmul = a->scale * 1.4426950408889634f;
  p.q = a->q; p.q_row = a->q_row;
  p.out = a->out; p.out_f32 = a->out_f32 != 0; p.lse = a->lse;
  p.err = a->err;
  char* ws = static_cast<char*>(a->workspace);
  cudaError_t e;
  if (a->ev_start && (e = cudaEventRecord(a->ev_start, stream)) != cudaSuccess) return cuda_status(e);
  if (pl.split.rows) {
    p.whole = pl.split.whole;
    p.ws_acc = reinterpret_cast<float*>(ws);
    p.ws_ml = reinterpret_cast<float2*>(ws + pl.split.off_ml);
    p.ws_desc = reinterpret_cast<int4*>(ws + pl.split.off_desc);
    rc = by_type(c.dtype, c.hd, pl.split.rows, [&](auto* t, auto d, auto r) {
      return launch_split<std::remove_pointer_t<decltype(t)>, decltype(d)::value, decltype(r)::value>(c, p, pl.split, stream);
    });
    if (rc != SWA_OK) return rc;
  }
  if (pl.has_chunk) {
    rc = launch_paged_chunk(a, p, pl.chunk, pl.split.rows ? p.most : 0, ws + pl.off_chunk, stream);
    if (rc != SWA_OK) return rc;
  }
  if (a->ev_stop && (e = cudaEventRecord(a->ev_stop, stream)) != cudaSuccess) return cuda_status(e);
  return SWA_OK;
}

}  // extern "C"
