// Paged attention over the 4-bit cache for many query rows per kv head (prompts and
// chunks of them), on the 5th-generation tensor cores.
//
// The formulas are those of lq_attn_q4.cu.  With hundreds of rows per code the
// matrix products bound the work (4 head_dim flops per row and position), so here
// a CTA takes 256 query rows of one kv head as two row tiles (one for head_dim 256)
// and walks the positions they see in tiles of 128 (64):
//     S = Q K^T       tcgen05.mma in fp16, both operands in shared memory, S in TMEM
//     W = 2^(x - max) by one thread per row, from TMEM and back: the fp16
//                     weights take the columns of the scores
//     O += W V        tcgen05.mma in fp16 with W from TMEM, O in TMEM
// One warp fetches codes, scales and bases by untiled bulk copies, up to three half
// tiles (K, V, K, ...) ahead; warps 0..3 turn them into fp16 values in two stages of shared
// memory; four warps per row tile hold its rows' maxima and sums, and one issues its
// products.  The values are what the cache stands for, exactly, so the softmax knows
// nothing of scales: a weight is one fma and one exponential.  A word of eight codes
// becomes pairs (0, 4), (1, 5), (2, 6), (3, 7) of dimensions, and is left in that order:
// queries are brought into it when they are read, outputs out of it when they are
// written.  bf16 queries are exact in fp16 after a power of two per row.
//
// The two row tiles run half a period apart, so that one's products run under the
// other's exponentials, and share every tile of values.  Scores are overwritten only
// after the products that read the weights there have completed.  The running maximum
// may lag by 2^7, so that a row's weights are made in one pass and O is rescaled only
// when the maximum really moves.  bf16 only: the tensor core's accumulator truncates,
// 6e-5 of the output after 30000 positions (measured), which fp32 outputs would show.
//
// What bounds it, head_dim 128 (prompt chunks of 1900 tokens over 2300 to 5400, 226 us):
// a step of 128 tokens takes 3350 clocks, in which the products of both row tiles run
// one after the other without a gap, 1650 clocks for the values and next scores of a
// tile where the tensor core's rate would be 1024.  Their operands come from shared
// memory at its 128 bytes a clock for the scores, and the conversions (2100 clocks a
// step, beside them) write there too: 296 KB a step, 2300 clocks.  A row's weights take
// 1000 clocks of that period, under the other tile's products.
//
// At head_dim 256 there is one row tile, two buffers of scores instead, and the queries
// lie in tensor memory.  A step of 64 tokens takes 2200 clocks: the 16 products of the
// scores are issued over 1000, then those of the values, and the next scores wait 950
// for these to complete (a third buffer does not fit); the conversions take 1900 beside
// them.  Before and after its tiles a CTA spends 9 us on the lengths, its queries and its
// outputs (24 requests of 500 to 12000 tokens, 24 to 40 rows each: 48.5 us of GPU time).
//
// Few row tiles, or requests much longer than others, would leave SMs idle: then several
// CTAs share a unit's positions (a pair of row tiles and a kv head), a range each, and a
// second kernel joins their outputs by row, in the order of the positions.  How many share
// a unit follows from the lengths, which only the device knows: no range is longer than P
// tiles, and every CTA finds the same P before it looks up its own range, as the one of
// some hundred that promises the earliest end.  (24 requests of 500 to 12000 tokens at
// head_dim 256: the same number of CTAs for every unit 80 us, by length 60.)
//
// Every wait is bounded (about a second of clock cycles); on expiry
// LQ_DEV_TIMEOUT is recorded and the CTA winds down.
#include "lq_attn_paged.cuh"
#include "lq_attn_q4.cuh"
#include "lq_attn_tiles.cuh"

namespace lq {
namespace q4 {

using namespace attn;

template <int D>
struct TileCfg : TileShape<D> {
  using TileShape<D>::T;
  using TileShape<D>::BN;
  using TileShape<D>::kSub;
  static constexpr int kQBytes = kTileRows * D * 2;         // of a row tile
  static constexpr int kValueBytes = BN * D * 2;            // a K or V tile as fp16
  static constexpr int kRawBytes = BN * D / 2;              // a K or V tile's codes
  static constexpr int kParamBytes = BN * (D / 32) * 4;     // and its scales and bases, at most
  // Half tiles as fetched, K and V in turn: from a slot's last read to the next data in it
  // 2200 clocks pass, which with one slot each for K and V the conversions waited for
  // (head_dim 256: 86 to 84 us with three; nine are no faster).
  static constexpr int kRaw = 3;
  static constexpr int kSmem = T * kQBytes + 4 * kValueBytes + kRaw * (kRawBytes + kParamBytes) + 1024;
  static constexpr uint32_t kCols = 512;
  // Columns for scores: one row tile has two buffers, so that the next tile's scores are
  // there when a tile's weights are done; with two row tiles each is the other's gap.
  static constexpr int kBufs = T == 1 ? 2 : 1;
  // and for its query rows, which the products would read again for every tile
  static constexpr bool kQueriesInTmem = T == 1;
  static_assert(T * (kBufs * BN + D) + (kQueriesInTmem ? D / 2 : 0) <= (int)kCols, "S, O and the queries fit TMEM");
  static constexpr int kMmaWarp = 4 + 4 * T;                // and the next, one per row tile
  static constexpr int kFetchWarp = kMmaWarp + T;
  static constexpr int kMoreWarp = kMmaWarp + 4;            // with one row tile, four more that convert
  static constexpr int kConvertWarps = T == 1 ? 8 : 4;
  static constexpr int kThreads = 512;                      // whole groups of four warps
  static_assert(kThreads == 32 * (4 + 4 * T + kConvertWarps), "four warps fetch and issue");
  // Registers per thread: the launch gives every warp 65536 / 512 = 128 (T = 2)
  // and the groups then divide those up, 80 + 2 x 184 + 64 = 4 x 128.
  static constexpr bool kSplitRegs = T == 2;
  static constexpr int kConvertRegs = 80, kSoftmaxRegs = 184, kIssueRegs = 64;
  static_assert(!kSplitRegs || kConvertRegs + 2 * kSoftmaxRegs + kIssueRegs <= 4 * 128, "the launch's registers");
  // tokens that the converting threads take in one pass (16 codes each), and passes per tile
  static constexpr int kPassRows = 32 * kConvertWarps * 16 / D;
  static constexpr int kPasses = BN / kPassRows;
};

struct TileArgs {
  CacheArgs ca;
  // Where CTAs may share a unit: the units of a kv head at most (0: they do not), and the
  // rows of a CTA's piece
  int items, stride, ctas, sms;
  int2* places;                  // of every query row: its first piece's row, and how many CTAs share it
};
// What a CTA costs beside its tiles, in tiles, and how many shares are tried.  (Measured at
// head_dim 256, 9 us in steps of 2200 clocks, and taken for the others too, whose steps of
// 3350 clocks make it 13 us.)
constexpr int kFixedTiles = 8, kMostShares = 128;

// A row's weights of one tile from its scores: packed fp16 weights and their sum;
// returns the largest weight's bits, or more (positive fp16 numbers are in the order of
// their bits, with infinity and NaN above, and take three-way integer maxima two at a
// time).  The exponent of a token is score * fac + base.
template <int BN>
__device__ __forceinline__ uint32_t row_weights(uint32_t tmem, float fac, float base, uint32_t (&w)[BN / 2], float& l) {
  uint32_t top = 0;
  uint32_t s[2][32];
  const float2 k2 = make_float2(fac, fac), d2 = make_float2(base, base);
  float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
  tmem_ld32_async(tmem, s[0]);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t (&x32)[32] = s[c & 1];
    tmem_wait_ld(x32);
    if (c + 1 < BN / 32) tmem_ld32_async(tmem + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float2 x = fma2(make_float2(__uint_as_float(x32[2 * e]), __uint_as_float(x32[2 * e + 1])), k2, d2);
      x = make_float2(ex2(x.x), ex2(x.y));
      if (e & 1) sum1 = add2(sum1, x);
      else sum0 = add2(sum0, x);
      w[16 * c + e] = pack_f16(x.x, x.y);
      if (e & 1) top = __vimax3_u16x2(top, w[16 * c + e - 1], w[16 * c + e]);
    }
  }
  sum0 = add2(sum0, sum1);
  l += sum0.x + sum0.y;
  return max(top >> 16, top & 0xFFFFu);
}

// The tiles that the above does not serve, few of a unit: tokens that a row does
// not see (beyond vis0, or in a block that is gone), rows whose maximum moves.  Two
// short loops, the largest exponent and then the weights: code that runs so seldom
// comes from far away.
template <int BN>
__device__ __forceinline__ float row_top(uint32_t tmem, float fac, uint32_t gone, int vis0) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t x32[32];
    tmem_ld32(tmem + 32 * c, x32);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int g = 2 * c + half, vis = (gone >> g & 1) ? -1 : vis0 - 16 * g;      // tokens 0 .. vis are seen
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, e > vis ? -INFINITY : __uint_as_float(x32[16 * half + e]) * fac);
    }
  }
  return top;
}
template <int BN>
__device__ __forceinline__ void store_weights(uint32_t tmem, float fac, float base, uint32_t gone, int vis0, float& l) {
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t x32[32], w[16];
    tmem_ld32(tmem + 32 * c, x32);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int g = 2 * c + half, vis = (gone >> g & 1) ? -1 : vis0 - 16 * g;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = ex2(2 * e > vis ? -INFINITY : fmaf(__uint_as_float(x32[16 * half + 2 * e]), fac, base));
        const float x1 = ex2(2 * e + 1 > vis ? -INFINITY : fmaf(__uint_as_float(x32[16 * half + 2 * e + 1]), fac, base));
        sum0 += x0;
        sum1 += x1;
        w[8 * half + e] = pack_f16(x0, x1);
      }
      l += sum0 + sum1;
    }
    tmem_st16(tmem + 16 * c, w);                            // over scores read before
  }
}

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1) tiles_kernel(const __grid_constant__ TileArgs ta) {
  using C = TileCfg<D>;
  constexpr int BN = C::BN, T = C::T;
  const Args& a = ta.ca.a;
  extern __shared__ uint8_t q4_tiles_smem_raw[];
  uint8_t* smem = q4_tiles_smem_raw + ((0u - smem_addr(q4_tiles_smem_raw)) & 1023u);
  uint8_t* sq = smem;                                       // the query rows
  uint8_t* sk = sq + T * C::kQBytes;                        // two stages each
  uint8_t* sv = sk + 2 * C::kValueBytes;
  uint8_t* raw = sv + 2 * C::kValueBytes;                   // codes as fetched
  uint8_t* params = raw + C::kRaw * C::kRawBytes;           // and their (scale, base) pairs
  __shared__ uint64_t k_full[2], k_free[2], v_full[2], v_free[2];   // per stage
  __shared__ uint64_t raw_full[C::kRaw], raw_free[C::kRaw];
  constexpr int B = C::kBufs;
  __shared__ uint64_t s_full[T][B], p_full[T][B], o_done[T][B], q_full[T], turn[T][2], drain;
  __shared__ uint32_t tmem_base;
  __shared__ int timeout_flag, found[5];                    // request, row tile, kv head; share, shares
  __shared__ int wsum[C::kThreads / 32];
  __shared__ unsigned long long best[C::kThreads / 32];
  volatile int* timeout = &timeout_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = D >> ta.ca.log2_group;

  pdl_wait();
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init1(&raw_full[i], 1);
      mbar_init1(&raw_free[i], C::kConvertWarps);           // one arrival per converting warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init1(&k_full[i], C::kConvertWarps);
      mbar_init1(&v_full[i], C::kConvertWarps);
      mbar_init1(&k_free[i], T);                            // the row tiles' products that read the stage are done
      mbar_init1(&v_free[i], T);
    }
    for (int t = 0; t < T; ++t) {
      for (int b = 0; b < B; ++b) {
        mbar_init1(&s_full[t][b], 1);                       // scores computed
        mbar_init1(&p_full[t][b], 4);                       // one arrival per softmax warp
        mbar_init1(&o_done[t][b], 1);                       // values added: O readable, the weights read
      }
      mbar_init1(&q_full[t], 4);
      mbar_init1(&turn[t][0], 1);                           // scores issued
      mbar_init1(&turn[t][1], 1);
    }
    mbar_init1(&drain, T);
    mbar_init_fence();
    timeout_flag = 0;
    found[0] = -1;
  }

  // this CTA's request and row tile, the last rows first: they see the most
  auto tiles_of = [&](const Request& r, int row0, int n_rows) {     // of the tokens that the last of the rows sees
    const int rows = r.q_len * a.group;
    if (row0 >= rows) return 0;
    const int last = min(row0 + n_rows, rows) - 1;
    const int seen = min(r.len, r.shown + last / a.group + 1);
    return seen > 0 ? (seen + BN - 1) / BN : 0;
  };
  {
    const int per = (a.batch + C::kThreads - 1) / C::kThreads;
    const int i0 = min(a.batch, (int)threadIdx.x * per), i1 = min(a.batch, i0 + per);
    auto items_of = [&](const Request& r) { return (r.q_len * a.group + C::kRows - 1) / C::kRows; };
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
      if (blockIdx.x == 0 && (int64_t)a.kv_lens[i] > ((int64_t)a.width << a.log2_bs))
        raise_flag(a.status, LQ_DEV_RANGE);
      sum += items_of(load_request(a, i));
    }
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) inc += wsum[w];
      total += wsum[w];
    }
    int begin = inc - sum;
    if (ta.items == 0) {
      const int h = blockIdx.x % a.kv_heads, item = blockIdx.x / a.kv_heads;
      if (item >= begin && item < inc) {
        for (int i = i0; i < i1; ++i) {
          const int n = items_of(load_request(a, i));
          if (item < begin + n) {
            found[0] = i;
            found[1] = begin + n - 1 - item;
            found[2] = h;
            found[3] = 0;
            found[4] = 1;
            break;
          }
          begin += n;
        }
      }
    } else {
      // every item's tiles, request and row tile, where the query rows will be
      int* const item_tiles = reinterpret_cast<int*>(sq);
      int* const item_req = item_tiles + ta.items;
      int* const item_at = item_req + ta.items;
      for (int i = i0; i < i1; ++i) {
        const Request r = load_request(a, i);
        const int n = items_of(r);
        for (int k = 0; k < n && begin + k < ta.items; ++k) {
          item_tiles[begin + k] = tiles_of(r, (n - 1 - k) * C::kRows, C::kRows);
          item_req[begin + k] = i;
          item_at[begin + k] = n - 1 - k;
        }
        begin += n;
      }
      __syncthreads();
      total = min(total, ta.items);
      int longest = 0;
      for (int i = lane; i < total; i += 32) longest = max(longest, item_tiles[i]);
      longest = __reduce_max_sync(0xffffffffu, longest);
      // Ranges per tile, 1 / P, such that the longest item makes j ranges, at most one for every
      // four tiles; and an item's ranges, rounded up (five tiles: two and three).  (Every CTA
      // has the same numbers: their last place may be off.  With divisions of whole numbers
      // this took 4200 clocks, so 2900.)
      auto ranges_of = [](int tiles, float density) { return max(1, (int)ceilf(fmaf((float)tiles, density, -1e-3f))); };
      // the end is that of the last wave of CTAs, each as long as its longest, and of the
      // rows' joining
      unsigned long long least = ~0ull;
      const float per_sm = 1.f / (float)ta.sms;
      for (int j = 1 + warp; j <= kMostShares && (j == 1 || j * a.kv_heads <= (int)gridDim.x); j += C::kThreads / 32) {
        const float density = fminf(0.25f, __fdividef((float)j, (float)max(1, longest)));
        int count = 0;
        for (int i = lane; i < total; i += 32) count += ranges_of(item_tiles[i], density);
        count = __reduce_add_sync(0xffffffffu, count) * a.kv_heads;
        if (j > 1 && count > (int)gridDim.x) continue;
        const float waves = ceilf((float)count * per_sm - 1e-3f);
        const float cost = waves * ((float)kFixedTiles + __fdividef(1.f, density)) + 0.125f * (float)j;
        least = min(least, (unsigned long long)__float_as_uint(cost) << 32 | __float_as_uint(density));
      }
      if (lane == 0) best[warp] = least;
      __syncthreads();
      if (warp == 0) {
        least = lane < C::kThreads / 32 ? best[lane] : ~0ull;
        for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        const float density = __uint_as_float((uint32_t)least);
        int before = 0;
        for (int at32 = 0; at32 < total && before <= (int)blockIdx.x; at32 += 32) {
          const int i = at32 + lane, shares = i < total ? ranges_of(item_tiles[i], density) : 0;
          int end = shares * a.kv_heads;
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += x;
          }
          end += before;
          const int at = (int)blockIdx.x - (end - shares * a.kv_heads);
          if (at >= 0 && (int)blockIdx.x < end) {
            found[0] = item_req[i];
            found[1] = item_at[i];
            found[2] = at / shares;
            found[3] = at % shares;
            found[4] = shares;
          }
          before = __shfl_sync(0xffffffffu, end, 31);
        }
      }
    }
    __syncthreads();
  }
  // rows that no request owns
  {
    const int64_t end = max(a.cu_q[a.batch], 0), cols = (int64_t)a.q_heads * D;
    for (int64_t t = end + blockIdx.x; t < a.total_q; t += gridDim.x)
      for (int64_t c = threadIdx.x; c < cols; c += C::kThreads) {
        reinterpret_cast<uint16_t*>(a.out)[t * a.ldo + c] = 0;
      }
  }
  if (found[0] < 0) {                                       // fewer units than CTAs
    return;
  }
  const int req = found[0], row0 = found[1] * C::kRows, h = found[2], share = found[3], shares = found[4];
  const Request r = load_request(a, req);
  const int rows = r.q_len * a.group;
  const int all0 = tiles_of(r, row0, kTileRows), all1 = T > 1 ? tiles_of(r, row0 + kTileRows, kTileRows) : 0;
  const int all = max(all0, all1);
  if (ta.items > 0 && share == 0) {                         // where the rows' pieces are
    for (int i = threadIdx.x; i < C::kRows && row0 + i < rows; i += C::kThreads) {
      const int j = (row0 + i) / a.group;
      ta.places[(int64_t)(r.q0 + j) * a.q_heads + h * a.group + row0 + i - j * a.group] =
          make_int2((int)blockIdx.x * ta.stride + i, shares);
    }
  }
  // this CTA's tiles: `first` and the ones after it
  const int first = (int)((int64_t)all * share / shares), past = (int)((int64_t)all * (share + 1) / shares);
  const int n0 = max(0, min(all0, past) - first), n1 = max(0, min(all1, past) - first), tiles = max(n0, n1);
  const int seen = min(r.len, past * BN);                   // tokens fetched end here
  const int32_t* table = a.table + (int64_t)req * a.ldt;

  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&tmem_base)), "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  // columns: the row tiles' scores, then their outputs, then query rows
  const uint32_t tmem_s = tmem_base, tmem_o = tmem_base + T * B * BN, tmem_q = tmem_o + T * D;
  // Tile j's buffer for scores, and the parity of the buffer's barriers.  A parity tells a
  // phase from the next only, so a wait for a phase comes neither when the phase after it may
  // have completed too nor while the one before it may be missing.  Each buffer has its own
  // o_done for that: after tile j's phase comes that of tile j + B, whose weights are announced
  // only after the last wait for tile j; and tile j - B's had completed when the scores of
  // tile j were issued, which whoever waits for tile j's values has issued or waited for.
  auto buf_of = [](int j) { return B == 2 ? j & 1 : 0; };
  auto parity_of = [](int j) { return (uint32_t)(B == 2 ? j >> 1 : j) & 1; };

  if (warp < 4 || warp >= C::kMoreWarp) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kConvertRegs));
    // ------------------------------------------------------------ codes to fp16
    // 16 codes per thread and pass.  The eight lanes of a shared-memory phase write
    // chunks 2 q (+ 1) of two neighbouring tokens' lines, whose swizzles keep them off
    // each other's banks; what they read is contiguous.
    const Masks masks;
    const int t = threadIdx.x - (warp < 4 ? 0 : 32 * (C::kMoreWarp - 4)), q = t & 3, sub = (t >> 3) & (C::kSub - 1);
    const int r0 = (t >> 2 & 1) + 2 * (t / (8 * C::kSub));
    const int grp = (64 * sub + 16 * q) >> ta.ca.log2_group;
    const uint32_t to0 = sub * BN * 128 + r0 * 128 + (((2 * q) ^ (r0 & 7)) << 4), to1 = to0 ^ 16;
    // lim: the tile's tokens that are there; others are zeros, whatever their slots hold
    int slot = 0;                                           // of the next half tile, and its phase
    uint32_t phase = 0;
    auto convert = [&](uint8_t* dst, int lim, uint64_t* full) {
      const uint8_t* src = raw + slot * C::kRawBytes + r0 * (D / 2) + sub * 32 + q * 8;
      const uint32_t* par = reinterpret_cast<const uint32_t*>(params + slot * C::kParamBytes) + r0 * groups + grp;
#pragma unroll
      for (int p = 0; p < C::kPasses; ++p) {
        const uint2 x = *reinterpret_cast<const uint2*>(src + p * C::kPassRows * (D / 2));
        uint32_t pr = par[p * C::kPassRows * groups];
        if (p * C::kPassRows + r0 >= lim) pr = 0u;
        const uint32_t s = twice_low(pr), b = twice_high(pr);
        uint8_t* line = dst + p * C::kPassRows * 128;
        *reinterpret_cast<uint4*>(line + to0) =
            make_uint4(fma_h2(masks.pair<0>(x.x), s, b), fma_h2(masks.pair<1>(x.x), s, b),
                       fma_h2(masks.pair<2>(x.x), s, b), fma_h2(masks.pair<3>(x.x), s, b));
        *reinterpret_cast<uint4*>(line + to1) =
            make_uint4(fma_h2(masks.pair<0>(x.y), s, b), fma_h2(masks.pair<1>(x.y), s, b),
                       fma_h2(masks.pair<2>(x.y), s, b), fma_h2(masks.pair<3>(x.y), s, b));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        arrive(&raw_free[slot]);
        arrive(full);
      }
      if (++slot == C::kRaw) {
        slot = 0;
        phase ^= 1;
      }
    };
    for (int j = 0; j < tiles; ++j) {
      const int st = j & 1, lim = seen - (first + j) * BN;
      const uint32_t before = (uint32_t)(j / 2 + 1) & 1;    // the stage's previous use
      bool ok = wait_on(&raw_full[slot], phase, timeout);
      if (j >= 2) ok = ok && wait_on(&k_free[st], before, timeout);
      if (!__all_sync(0xffffffffu, ok)) break;
      convert(sk + st * C::kValueBytes, lim, &k_full[st]);
      ok = wait_on(&raw_full[slot], phase, timeout);
      if (j >= 2) ok = ok && wait_on(&v_free[st], before, timeout);
      if (!__all_sync(0xffffffffu, ok)) break;
      convert(sv + st * C::kValueBytes, lim, &v_full[st]);
    }
  } else if (warp >= C::kMmaWarp) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
    if (warp == C::kFetchWarp) {
      // ------------------------------------------------------------ codes from the cache
      // lane g: the g-th part of the tile, a block or BN tokens of one
      const int step = min(1 << a.log2_bs, BN), parts = BN / step;
      auto look_up = [&](int j) {
        const int pos = (first + j) * BN + step * lane;
        return lane < parts && pos < seen ? table[pos >> a.log2_bs] : -1;
      };
      int blk = look_up(0), issued = 0, slot = 0;
      uint32_t phase = 1;                                   // of the slot's last read
      for (int j = 0; j < tiles; ++j) {
        const int pos = (first + j) * BN + step * lane;
        const bool ok = (unsigned)blk < (unsigned long long)a.num_blocks;
        const bool lost = !ok && lane < parts && pos < seen;
        if (lost) raise_flag(a.status, LQ_DEV_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * step * (D / 2 + 4 * groups);
        const int64_t row = (((int64_t)blk * a.kv_heads + h) << a.log2_bs) + (pos & ((1 << a.log2_bs) - 1));
        blk = look_up(j + 1);
        bool go = true;
        for (int v = 0; v < 2 && go; ++v) {
          if (issued >= C::kRaw) go = __all_sync(0xffffffffu, wait_on(&raw_free[slot], phase, timeout));
          if (!go) break;
          uint8_t* codes = raw + slot * C::kRawBytes + lane * step * (D / 2);
          uint32_t* par = reinterpret_cast<uint32_t*>(params + slot * C::kParamBytes) + lane * step * groups;
          if (lost) {                                       // a block that is not there: zeros
            for (int i = 0; i < step * groups; ++i) par[i] = 0u;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&raw_full[slot], bytes);
          __syncwarp();
          if (ok) {
            bulk_load(codes, (v ? ta.ca.vc : ta.ca.kc) + row * (D / 2), step * (D / 2), &raw_full[slot]);
            bulk_load(par, (v ? ta.ca.vs : ta.ca.ks) + row * groups, step * groups * 4, &raw_full[slot]);
          }
          ++issued;
          if (++slot == C::kRaw) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (!go) break;
      }
      // after a timeout: let the copies in flight land before the CTA ends
      if (*timeout)
        for (int q = max(0, issued - C::kRaw); q < issued; ++q)
          mbar_wait_bounded(&raw_full[q % C::kRaw], (uint32_t)(q / C::kRaw) & 1, kWaitCycles / 8);
    } else if (warp < C::kFetchWarp) {
      // ------------------------------------------------------------ products
      // A warp per row tile: the products of one then run while the other's warp
      // waits (one warp for both, in line: 3950 clocks a step, 2050 of them
      // products).  The whole warp runs the loop, so that descriptors are uniform
      // values; one elected lane issues.
      const int t = warp - C::kMmaWarp, n = t == 0 ? n0 : n1;
      const uint64_t dq = desc_k_major(smem_addr(sq + t * C::kQBytes)), dk = desc_k_major(smem_addr(sk));
      const uint64_t dv = desc_mn_major(smem_addr(sv), C::kSub > 1 ? BN * 128 : 1024);
      const uint32_t my_s = tmem_s + t * B * BN, my_o = tmem_o + t * D;
      auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
      // scores of tile j; past this row tile's last, the other's codes are let go
      auto scores = [&](int j) {
        if (j >= tiles) return true;
        const int st = j & 1;
        bool ok = wait_on(&k_full[st], (uint32_t)(j >> 1) & 1, timeout);
        if (j < n) {
          if (j == 0) ok = ok && wait_on(&q_full[t], 0, timeout);
          // they overwrite the weights of the buffer's last tile
          else if (j >= B) ok = ok && wait_on(&o_done[t][buf_of(j - B)], parity_of(j - B), timeout);
        }
        if (!all(ok)) return false;
        tc_after();
        if (elect()) {
          if (j < n) {
            const uint64_t kd = dk + (uint64_t)(st * C::kValueBytes >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t kk = kd + (((k >> 2) * BN * 128 + (k & 3) * 32) >> 4);
              if constexpr (C::kQueriesInTmem)
                mma_ts(my_s + buf_of(j) * BN, tmem_q + k * 8, kk, Idesc<BN, false, false>::v, k > 0);
              else
                mma_ss(my_s + buf_of(j) * BN, dq + (((k >> 2) * kTileRows * 128 + (k & 3) * 32) >> 4), kk,
                       Idesc<BN, false, false>::v, k > 0);
            }
            mma_commit(&s_full[t][buf_of(j)]);
            mma_commit(&k_free[st]);
            arrive(&turn[t][st]);
          } else {
            arrive(&k_free[st]);
          }
        }
        __syncwarp();
        return true;
      };
      auto add_values = [&](int j) {
        const int st = j & 1;
        bool ok = wait_on(&v_full[st], (uint32_t)(j >> 1) & 1, timeout);
        if (j < n) ok = ok && wait_on(&p_full[t][buf_of(j)], parity_of(j), timeout);
        // In turn, values and next scores of one row tile, then of the other: when
        // both had weights ready together, they would stay in step and neither's
        // exponentials run under the other's products.  (Neither can be two tiles
        // ahead here: a parity tells.  The turn passes when the scores have been
        // issued: passed before, the two warps' products interleave and the row
        // tile that is ahead loses its lead, 252 us to 242.)
        if (T > 1 && t == 0 && j < min(n, n1)) ok = ok && wait_on(&turn[T - 1][st], (uint32_t)(j >> 1) & 1, timeout);
        if (T > 1 && t == 1 && j < n && j + 1 < n0) ok = ok && wait_on(&turn[0][st ^ 1], (uint32_t)((j + 1) >> 1) & 1, timeout);
        if (!all(ok)) return false;
        tc_after();
        if (elect()) {
          if (j < n) {
            const uint64_t vd = dv + (uint64_t)(st * C::kValueBytes >> 4);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts(my_o, my_s + buf_of(j) * BN + k * 8, vd + (k * 2048 >> 4), Idesc<D, false, true>::v, j > 0 || k > 0);
            mma_commit(&o_done[t][buf_of(j)]);
            mma_commit(&v_free[st]);
          } else {
            arrive(&v_free[st]);
          }
        }
        __syncwarp();
        return true;
      };
      bool ok = scores(0);
      for (int j = 0; j < tiles && ok; ++j)
        ok = B == 2 ? scores(j + 1) && add_values(j) : add_values(j) && scores(j + 1);
    }
  } else {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;                          // row tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tile_s = tmem_s + lanes + t * B * BN, my_o = tmem_o + lanes + t * D;
    const int R0 = row0 + t * kTileRows, R = R0 + row, j_tok = R / a.group;
    const int n = t == 0 ? n0 : n1;
    const bool mine = R < rows;
    const int head = h * a.group + R - j_tok * a.group;
    const int lim = mine ? min(r.shown + j_tok, r.len - 1) : r.len - 1;     // last position the row sees
    const int lim_min = min(r.shown + R0 / a.group, r.len - 1);           // of the tile's first row

    // The warp's query rows go to shared memory as they are, D / 8 lanes to a
    // row; rows past the request's are zeros.
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    uint8_t* my_line = sq + t * C::kQBytes + row * 128;
    auto chunk_of = [&](int c) {                            // 16-byte part c of this thread's row
      return reinterpret_cast<uint4*>(my_line + (c >> 3) * kTileRows * 128 + (((c & 7) ^ (row & 7)) << 4));
    };
    auto line_of = [&](int r32, int c) {                    // 16-byte part c of the warp's row
      const int rr = (warp & 3) * 32 + r32;
      return sq + t * C::kQBytes + (c >> 3) * kTileRows * 128 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
    };
    {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q);
      if (mine) src += (int64_t)(r.q0 + j_tok) * a.ldq + (int64_t)head * D;
      const uint32_t have = __ballot_sync(0xffffffffu, mine);
      const int c = lane & (kLanes - 1);
#pragma unroll 8
      for (int pass = 0; pass < kLanes; ++pass) {
        const int from = pass * kAtOnce + lane / kLanes;
        const uint16_t* p =
            reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), from));
        copy16(line_of(from, c), p + 8 * c, have >> from & 1 ? 16 : 0);
      }
    }

    // lane g < BN / 16: whether the tile's g-th 16 tokens lie in a block that is not
    // there, a tile ahead
    bool lost = false;
    auto look_up = [&](int j) {
      const int pos = (first + j) * BN + 16 * lane;
      lost = lane < BN / 16 && pos < seen && (unsigned)table[pos >> a.log2_bs] >= (unsigned long long)a.num_blocks;
    };
    if (n > 0) look_up(0);

    // To fp16, in place or in tensor memory, each word of eight dimensions in the values' order, after a
    // power of two that brings the row's largest to [2^13, 2^14).
    float fac;
    {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t top = 0;                                     // of the two halves' magnitudes
#pragma unroll 8
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = *chunk_of(c);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
      }
      top = max(top >> 16, top & 0xFFFFu);
      const int ex = min(126, max(-116, 140 - (int)(top >> 7)));
      const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
      fac = a.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
      const auto halves = [&](const uint4& x) {
        const auto low = [&](uint32_t v) { return __uint_as_float(v << 16) * up; };
        const auto high = [&](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u) * up; };
        return make_uint4(pack_f16(low(x.x), low(x.z)), pack_f16(high(x.x), high(x.z)), pack_f16(low(x.y), low(x.w)),
                          pack_f16(high(x.y), high(x.w)));
      };
      if constexpr (C::kQueriesInTmem) {
#pragma unroll 2
        for (int c = 0; c < D / 8; c += 4) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 x = halves(*chunk_of(c + e));
            w[4 * e] = x.x; w[4 * e + 1] = x.y; w[4 * e + 2] = x.z; w[4 * e + 3] = x.w;
          }
          tmem_st16(tmem_q + lanes + 4 * c, w);
        }
        tmem_wait_st();
        tc_before();
      } else {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) *chunk_of(c) = halves(*chunk_of(c));
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) arrive(&q_full[t]);
    }
    float mx = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t gone = __ballot_sync(0xffffffffu, lost);
      if (j + 1 < n) look_up(j + 1);
      const int vis0 = lim - (first + j) * BN;
      const bool masked = (first + j + 1) * BN - 1 > lim_min || gone != 0;
      const uint32_t my_s = tile_s + buf_of(j) * BN;
      ok = __all_sync(0xffffffffu, wait_on(&s_full[t][buf_of(j)], parity_of(j), timeout));
      if (!ok) break;
      tc_after();
      __syncwarp();
      bool common = !masked && !__any_sync(0xffffffffu, mx == -INFINITY);
      if (common) {
        uint32_t w[BN / 2];
        float sum = l;
        const uint32_t top = row_weights<BN>(my_s, fac, kShift - mx, w, sum);
        common = !__any_sync(0xffffffffu, top > kTopWeight);
        if (common) {
          l = sum;
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) tmem_st16(my_s + 16 * c, w + 16 * c);
        }
      }
      if (!common) {
        // where the maximum moves, what there is so far shrinks
        const float top = row_top<BN>(my_s, fac, gone, vis0);
        const bool moves = mx == -INFINITY ? top != -INFINITY : top > mx + kLead;
        const float to = moves ? ceilf(top) : mx, f = moves ? pow2(mx - to) : 1.f;
        l *= f;
        mx = to;
        if (j > 0 && __any_sync(0xffffffffu, moves)) {
          if (B == 2) {                                     // (one buffer: these scores came after the last values)
            ok = __all_sync(0xffffffffu, wait_on(&o_done[t][buf_of(j - 1)], parity_of(j - 1), timeout));
            if (!ok) break;
            tc_after();
            __syncwarp();
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(my_o + 32 * c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(my_o + 32 * c, o);
            tmem_st16(my_o + 32 * c + 16, o + 16);
          }
        }
        store_weights<BN>(my_s, fac, kShift - (mx == -INFINITY ? 0.f : mx), gone, vis0, l);
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) arrive(&p_full[t][buf_of(j)]);
    }

    // Outputs, by way of the rows of shared memory where the queries were (the
    // products with them are done): a warp's stores then cover whole lines.
    // (Products complete in their order: the last tile's values are there, so all are.)
    if (ok && n > 0) ok = __all_sync(0xffffffffu, wait_on(&o_done[t][buf_of(n - 1)], parity_of(n - 1), timeout));
    tc_after();
    __syncwarp();
    const uint32_t rows_out = __ballot_sync(0xffffffffu, mine);
    if (ok && rows_out) {
      const bool whole = shares == 1;
      // with the positions split: the row's sums as they are
      float* piece = a.part + ((int64_t)blockIdx.x * ta.stride + R - row0) * (D + 4);
      uint8_t* dst = reinterpret_cast<uint8_t*>(
          whole ? reinterpret_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + j_tok) * a.ldo + (int64_t)head * D
                : reinterpret_cast<uint16_t*>(piece));
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // 2 D bytes of each row: all of it as bf16, or half of it
#pragma unroll 1
      for (int part = 0; part < (whole ? 1 : 2); ++part) {
#pragma unroll 1
        for (int c = 0; c < (whole ? D / 32 : D / 64); ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(my_o + part * (D / 2) + 32 * c, o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          // columns 0, 2, 4, 6 of eight are dimensions 0 .. 3, columns 1, 3, 5, 7 the others
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t u[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int at = 8 * e + 4 * (q & 1) + (q >> 1);
                const __nv_bfloat162 b =
                    __floats2bfloat162_rn(__uint_as_float(o[at]) * inv, __uint_as_float(o[at + 2]) * inv);
                u[q] = *reinterpret_cast<const uint32_t*>(&b);
              }
              *chunk_of(4 * c + e) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = 8 * (e >> 1) + (e & 1);
              *chunk_of(8 * c + e) = make_uint4(o[at], o[at + 2], o[at + 4], o[at + 6]);
            }
          }
        }
        __syncwarp();
        // (reads of eight passes first: the compiler keeps them behind the stores before)
#pragma unroll 1
        for (int pass = 0; pass < kLanes; pass += 8) {
          const int c = lane & (kLanes - 1);
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = *reinterpret_cast<const uint4*>(line_of((pass + i) * kAtOnce + lane / kLanes, c));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int from = (pass + i) * kAtOnce + lane / kLanes;
            uint8_t* p = reinterpret_cast<uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), from));
            if (rows_out >> from & 1) *reinterpret_cast<uint4*>(p + part * 2 * D + 16 * c) = x[i];
          }
        }
        __syncwarp();
      }
      if (!whole && mine) {
        piece[D] = mx;
        piece[D + 1] = l;
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_before();
  __syncthreads();
  if (timeout_flag && warp >= C::kMmaWarp && warp < C::kFetchWarp) {
    // products may still be in flight: all have completed once this arrives
    if (elect()) mma_commit(&drain);
    __syncwarp();
  }
  if (warp == C::kMmaWarp) {
    if (timeout_flag) mbar_wait_bounded(&drain, 0, kWaitCycles);
    __syncwarp();
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::kCols));
  }
  if (threadIdx.x == 0 && timeout_flag) raise_flag(a.status, LQ_DEV_TIMEOUT);
}

// Joins what the CTAs that share a row's positions left of it: a warp per row, D / 32
// neighbouring dimensions per lane.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ TileArgs ta) {
  constexpr int E = D / 32;
  const Args& a = ta.ca.a;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), tokens = min((int64_t)a.cu_q[a.batch], a.total_q);
  const int64_t token = row / a.q_heads;
  if (token >= tokens) return;                              // no request's: zeros already
  const int2 place = ta.places[row];
  // one CTA's already (or of no request, in offsets that are not in order)
  if (place.y <= 1 || place.y > ta.ctas || place.x < 0 || place.x >= (ta.ctas - place.y + 1) * ta.stride) return;
  const float* piece = a.part + (int64_t)place.x * (D + 4);
  const int64_t next = (int64_t)ta.stride * (D + 4);
  float M = -INFINITY;
#pragma unroll 4
  for (int p = 0; p < place.y; ++p) M = fmaxf(M, piece[p * next + D]);
  float o[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < place.y; ++p) {
    const float m = piece[p * next + D], f = m == M ? 1.f : pow2(m - M);
    l = fmaf(piece[p * next + D + 1], f, l);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = *reinterpret_cast<const float2*>(piece + p * next + E * lane + e);
      o[e] = fmaf(v.x, f, o[e]);
      o[e + 1] = fmaf(v.y, f, o[e + 1]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t dst = token * a.ldo + (row - token * a.q_heads) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + dst + e) =
        __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
}

template <int D>
lq_status launch(const TileArgs& ta, void* stream) {
  using C = TileCfg<D>;
  static_assert(C::kSmem + 1536 <= 227 * 1024, "shared memory");
  auto kern = tiles_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  const lq_status st = serve::launch(kern, (unsigned)ta.ctas, C::kThreads, C::kSmem, stream, ta);
  if (st != LQ_OK || ta.items == 0) return st;
  const int64_t rows = ta.ca.a.total_q * ta.ca.a.q_heads;
  return serve::launch(merge_kernel<D>, (unsigned)((rows + 7) / 8), 256, 0, stream, ta);
}

// Row tiles, or pairs of them, of a request's rows, at least `group` of them, rounded up.
static int64_t items_of(int batch, int64_t total_q, int group, int head_dim) {
  const int rows = head_dim == 256 ? TileCfg<256>::kRows : TileCfg<128>::kRows;
  const int64_t requests = batch < total_q ? batch : total_q;
  return (total_q * group - requests) / rows + requests;
}
// CTAs per SM where they may share units: two for each unit, so that a wave is at least
// two thirds full whatever their number is, and four at most; 0: a unit is one CTA's, and
// as long as its request is.  (37 requests of 500 tokens and one of 60000, five query tokens
// each of 8 heads for 8 kv heads of 128: 750 us, all of them the long one's.)
static int waves_of(int64_t units, int sms) {
  const int64_t n = (2 * units + sms - 1) / sms;
  return n <= 4 ? (int)n : 0;
}
// A CTA's piece has as many rows as a request can have.
static int stride_of(int64_t total_q, int group, int head_dim) {
  const int rows = head_dim == 256 ? TileCfg<256>::kRows : TileCfg<128>::kRows;
  return total_q * group < rows ? (int)(total_q * group) : rows;
}

size_t tiles_workspace(int batch, int64_t total_q, int q_heads, int kv_heads, int head_dim, int sms) {
  const int group = q_heads / kv_heads, waves = waves_of(items_of(batch, total_q, group, head_dim) * kv_heads, sms);
  if (waves == 0) return 0;
  const size_t places = ((size_t)total_q * q_heads * sizeof(int2) + 15) & ~(size_t)15;
  return places + (size_t)waves * sms * stride_of(total_q, group, head_dim) * (head_dim + 4) * sizeof(float);
}

lq_status launch_tiles(const CacheArgs& ca, int head_dim, int64_t most_tokens, int sms, void* workspace, void* stream) {
  const Args& a = ca.a;
  const int64_t items = items_of(a.batch, a.total_q, a.group, head_dim);
  const int bn = head_dim == 256 ? TileCfg<256>::BN : TileCfg<128>::BN;
  // (no unit is shared that has fewer than eight tiles)
  const int waves = most_tokens >= 8 * bn ? waves_of(items * a.kv_heads, sms) : 0;
  const int64_t ctas = waves > 0 ? (int64_t)waves * sms : items * a.kv_heads;
  if (ctas > INT32_MAX) return LQ_ERR_SHAPE;
  TileArgs ta;
  ta.ca = ca;
  ta.items = waves > 0 ? (int)items : 0;
  ta.ctas = (int)ctas;
  ta.sms = sms;
  ta.stride = stride_of(a.total_q, a.group, head_dim);
  ta.places = reinterpret_cast<int2*>(workspace);
  ta.ca.a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) +
                                          (((size_t)a.total_q * a.q_heads * sizeof(int2) + 15) & ~(size_t)15));
  switch (head_dim) {
    case 64: return launch<64>(ta, stream);
    case 128: return launch<128>(ta, stream);
    default: return launch<256>(ta, stream);
  }
}

}  // namespace q4
}  // namespace lq
