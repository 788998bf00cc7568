// Paged attention for many query rows per kv head (prompts and chunks of
// them), on the 5th-generation tensor cores.
//
// The formulas are those of lq_attn_paged.cu.  With hundreds of rows per code
// the matrix products bound the work (4 head_dim flops per row and position),
// so here a CTA takes 256 query rows of one kv head as two row tiles (one for
// head_dim 256) and walks the positions they see in tiles of 128 (64):
//     S = Q C_k^T     tcgen05.mma in bf16, both operands in shared memory, S in
//                     TMEM (queries as they are; codes are whole numbers)
//     W = 2^(x - max) by one thread per row, from TMEM and back: the fp16
//                     weights take the columns of the scores
//     O += W C_v      tcgen05.mma in fp16 with W from TMEM, O in TMEM
// One warp fetches the codes of a tile by TMA, up to two half tiles (K, V)
// ahead; warps 0..3 turn them into bf16 and fp16, exactly, in two stages of
// shared memory; four warps per row tile hold its rows' maxima and sums, and one
// issues its products.  (Codes fetched through registers instead made the
// converting warps the slowest part: the L1 that this much shared
// memory leaves holds too few loads in flight.)
// K and V tiles have the same layout, rows of 64 dimensions in the 128-byte
// swizzle, which the products read along either axis (K-major for the scores,
// MN-major for the values).  The two row tiles run half a period apart, so that
// one's products run under the other's exponentials, and share every tile of
// codes: shared memory (operands read at 128 bytes a clock, tiles written) and
// the conversions would otherwise bound the kernel before the tensor core does.
// Scores are overwritten only after the products that read the weights there
// have completed.  A step of 128 tokens takes 1.99 us for the 256 rows (the
// products alone would 1.07), and a CTA's start, first and last tiles and
// outputs about 9 us: what happens once per CTA is serial, so queries are
// copied without a pass over them in registers, masked tiles go through short
// loops, and outputs leave by whole lines.  (CTAs that go on from one group of
// rows to the next, an equal part of all positions each, took longer: 285 us
// to 257 for chunks of 1900 tokens over 2300 to 5400, now 245.)
//
// As in the split kernel the running maximum may lag by 2^7, so that a row's
// weights are made in one pass and O is rescaled (TMEM to registers and back)
// only when the maximum really moves.  bf16 only: the tensor core's accumulator
// truncates, 6e-5 of the output after 30000 positions (measured), which fp32
// outputs would show; they stay with the split kernel at any number of rows.
// Few row tiles (a short chunk over a long cache) would leave SMs idle: then
// several CTAs share one, a range of the positions each, and a second kernel
// joins their outputs, in the order of the positions.
//
// Every wait is bounded (about a second of clock cycles); on expiry
// LQ_DEV_TIMEOUT is recorded and the CTA winds down.
#include "lq_attn_paged.cuh"
#include "lq_attn_tiles.cuh"

namespace lq {
namespace attn {

// Which weights may go into a row's sum as weight / value scale: those of blocks
// whose value scale is at least a floor.  With lv its log2 and lv >= mx - un - 60,
// the score of a weight that is flushed (x < mx - 134) is below un - 74, and no
// score is above un + 67.  Blocks below the floor (zeros above all) go into the sum
// by their scores, 2^(score - un), at the cost of an exponential of their own; so
// does everything where mx - un is so low that a row's factor would leave fp32's
// range.
constexpr float kFloorGap = 60.f, kFloorLeast = -100.f, kUnitLeast = -100.f;

// The warp's floor under value scales for the rows of its lanes (mx of -inf: a row
// without a weight yet); infinite where a row's factor is out of range: no block is above it.
struct Floor {
  int most = -300, least = 300;
  __device__ __forceinline__ void add(float mx, float un) {
    if (mx == -INFINITY) return;
    const int d = (int)fminf(fmaxf(mx - un, -300.f), 300.f);
    most = max(most, d);
    least = min(least, d);
  }
  __device__ __forceinline__ float over_warp() const {
    const int hi = __reduce_max_sync(0xffffffffu, most), lo = __reduce_min_sync(0xffffffffu, least);
    return lo < (int)kUnitLeast ? INFINITY : pow2(fmaxf((float)hi - kFloorGap, kFloorLeast));
  }
};

template <int D>
struct TileCfg : TileShape<D> {
  using TileShape<D>::T;
  using TileShape<D>::BN;
  using TileShape<D>::kSub;
  static constexpr int kQBytes = kTileRows * D * 2;         // of a row tile
  static constexpr int kCodeBytes = BN * D * 2;             // a K or V tile as fp16
  static constexpr int kRawBytes = BN * D;                  // a K or V tile's codes
  static constexpr int kSmem = T * kQBytes + 4 * kCodeBytes + 2 * kRawBytes + 1024;
  static constexpr uint32_t kCols = 512;
  static_assert(T * (BN + D) <= (int)kCols, "S and O fit TMEM");
  static constexpr int kMmaWarp = 4 + 4 * T;                // and the next, one per row tile
  static constexpr int kFetchWarp = kMmaWarp + T;
  static constexpr int kThreads = 32 * (8 + 4 * T);         // whole groups of four warps
  // Registers per thread: the launch gives every warp 65536 / 512 = 128 (T = 2)
  // and the groups then divide those up, 80 + 2 x 184 + 64 = 4 x 128.
  static constexpr bool kSplitRegs = T == 2;
  static constexpr int kConvertRegs = 80, kSoftmaxRegs = 184, kIssueRegs = 64;
  static_assert(!kSplitRegs || kConvertRegs + 2 * kSoftmaxRegs + kIssueRegs <= 4 * 128, "the launch's registers");
  // rows of codes that the 128 converting threads take in one pass (4 lanes
  // of 16 codes for each 64 dimensions), and passes per tile
  static constexpr int kPassRows = 32 / kSub;
  static constexpr int kPasses = BN / kPassRows;
};

struct TileArgs {
  CUtensorMap map_k, map_v;      // boxes of a block's codes, or of BN tokens of it
  Args a;
  int splits;                    // CTAs per pair of row tiles and kv head
};

// Two codes, placed by `sel`, as bf16 numbers.  0x4300 + (the low seven bits) is
// 128 + those, and 0x4300 or 0x4380 is 128 or 256, as the sign bit is clear or
// set: their difference is the code, exactly.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t codes, uint32_t sel) {
  const uint32_t p = __byte_perm(codes, 0x43434343u, sel), x = p & 0xFF7FFF7Fu, y = p & 0xFF80FF80u;
  const __nv_bfloat162 v =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A row's weights of one tile from its scores: packed fp16 weights, the sum of
// weight / value scale in the row's unit; returns the largest weight's bits, or more (positive
// fp16 numbers are in the order of their bits, with infinity and NaN above, and
// take three-way integer maxima two at a time).  scales[g], of the g-th 16
// tokens: key scale, log2 and reciprocal of the value scale; the exponent of a
// token is score * fac * .x + .y + base.
template <int BN>
__device__ __forceinline__ uint32_t row_weights(uint32_t tmem, float fac, float base, float unit, const float4* scales,
                                             uint32_t (&w)[BN / 2], float& l) {
  uint32_t top = 0;
  uint32_t s[2][32];
  float4 sc[2] = {scales[0], scales[1]};
  tmem_ld32_async(tmem, s[0]);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t (&x32)[32] = s[c & 1];
    tmem_wait_ld(x32);
    if (c + 1 < BN / 32) tmem_ld32_async(tmem + 32 * (c + 1), s[(c + 1) & 1]);
    const float4 now[2] = {sc[0], sc[1]};
    if (c + 1 < BN / 32) {
      sc[0] = scales[2 * c + 2];
      sc[1] = scales[2 * c + 3];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float k = fac * now[half].x, d = now[half].y + base;
      const float2 k2 = make_float2(k, k), d2 = make_float2(d, d);
      float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t* y = x32 + 16 * half + 2 * e;
        float2 x = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), k2, d2);
        x = make_float2(ex2(x.x), ex2(x.y));
        if (e & 1) sum1 = add2(sum1, x);
        else sum0 = add2(sum0, x);
        w[16 * c + 8 * half + e] = pack_f16(x.x, x.y);
        if (e & 1) top = __vimax3_u16x2(top, w[16 * c + 8 * half + e - 1], w[16 * c + 8 * half + e]);
      }
      sum0 = add2(sum0, sum1);
      l = fmaf(sum0.x + sum0.y, now[half].z * unit, l);
    }
  }
  return max(top >> 16, top & 0xFFFFu);
}

// The tiles that the above does not serve, few of a unit: tokens that a row does
// not see (beyond vis0, or in a block that is gone), blocks below the floor of
// value scales, rows whose maximum moves.  Two short loops, the largest exponent
// (.x) and score (.y) and then the weights: code that runs so seldom comes from
// far away, and unrolled twice over it took three times as long as the common
// tiles' (3.5 us a tile to 1.1).
template <int BN>
__device__ __forceinline__ float2 row_top(uint32_t tmem, float fac, const float4* scales, uint32_t gone, int vis0) {
  float2 top = make_float2(-INFINITY, -INFINITY);
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t x32[32];
    tmem_ld32(tmem + 32 * c, x32);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int g = 2 * c + half, vis = (gone >> g & 1) ? -1 : vis0 - 16 * g;      // tokens 0 .. vis are seen
      const float4 sc = scales[g];
      const float k = fac * sc.x;
      float most = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, e > vis ? -INFINITY : __uint_as_float(x32[16 * half + e]) * k);
      // (fmaxf passes over the NaN of a block of infinite scale that the row does not see)
      top = make_float2(fmaxf(top.x, most + sc.y), fmaxf(top.y, most));
    }
  }
  return top;
}
template <int BN>
__device__ __forceinline__ void store_weights(uint32_t tmem, float fac, float base, float unit, float un,
                                              const float4* scales, uint32_t low, uint32_t gone, int vis0, float& l) {
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t x32[32], w[16];
    tmem_ld32(tmem + 32 * c, x32);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int g = 2 * c + half, vis = (gone >> g & 1) ? -1 : vis0 - 16 * g;
      const float4 sc = scales[g];
      const float k = fac * sc.x, d = sc.y + base;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = ex2(2 * e > vis ? -INFINITY : fmaf(__uint_as_float(x32[16 * half + 2 * e]), k, d));
        const float x1 = ex2(2 * e + 1 > vis ? -INFINITY : fmaf(__uint_as_float(x32[16 * half + 2 * e + 1]), k, d));
        sum0 += x0;
        sum1 += x1;
        w[8 * half + e] = pack_f16(x0, x1);
      }
      if (low >> g & 1) {                                   // below the floor: by the scores
        sum0 = sum1 = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          sum0 += e > vis ? 0.f : ex2(fmaf(__uint_as_float(x32[16 * half + e]), k, -un));
        l += sum0;
      } else {
        const float total = sum0 + sum1;
        // a block the row does not see may have any scale: its sum is 0, not 0 * NaN
        l = fmaf(total, total > 0.f ? sc.z * unit : 0.f, l);
      }
    }
    tmem_st16(tmem + 16 * c, w);                            // over scores read before
  }
}

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1) attn_tiles_kernel(const __grid_constant__ TileArgs ta) {
  using C = TileCfg<D>;
  constexpr int BN = C::BN, T = C::T;
  const Args& a = ta.a;
  extern __shared__ uint8_t tiles_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tiles_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;                                       // the query rows
  uint8_t* sk = sq + T * C::kQBytes;                        // two stages each
  uint8_t* sv = sk + 2 * C::kCodeBytes;
  uint8_t* raw = sv + 2 * C::kCodeBytes;                    // codes as fetched, K and V
  __shared__ uint64_t k_full[2], k_free[2], v_full[2], v_free[2];   // per stage
  __shared__ uint64_t raw_full[2], raw_free[2];             // K, V
  __shared__ uint64_t s_full[T], p_full[T], o_done[T], q_full[T], turn[T][2], drain;
  __shared__ uint32_t tmem_base;
  __shared__ int timeout_flag, found[2];
  __shared__ int wsum[C::kThreads / 32];
  __shared__ float4 scales[4 * T][BN / 16];                 // per softmax warp
  volatile int* timeout = &timeout_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init1(&raw_full[i], 1);
      mbar_init1(&raw_free[i], 4);                          // one arrival per converting warp
      mbar_init1(&k_full[i], 4);
      mbar_init1(&v_full[i], 4);
      mbar_init1(&k_free[i], T);                            // the row tiles' products that read the stage are done
      mbar_init1(&v_free[i], T);
    }
    for (int t = 0; t < T; ++t) {
      mbar_init1(&s_full[t], 1);                            // scores computed
      mbar_init1(&p_full[t], 4);                            // one arrival per softmax warp
      mbar_init1(&o_done[t], 1);                            // values added: O readable, the weights read
      mbar_init1(&q_full[t], 4);
      mbar_init1(&turn[t][0], 1);                           // scores issued
      mbar_init1(&turn[t][1], 1);
    }
    mbar_init1(&drain, T);
    mbar_init_fence();
    timeout_flag = 0;
    found[0] = -1;
  }

  // rows that no request owns
  {
    const int64_t end = max(a.cu_q[a.batch], 0), cols = (int64_t)a.q_heads * D;
    for (int64_t t = end + blockIdx.x; t < a.total_q; t += gridDim.x)
      for (int64_t c = threadIdx.x; c < cols; c += C::kThreads) {
        reinterpret_cast<uint16_t*>(a.out)[t * a.ldo + c] = 0;
      }
  }

  // this CTA's request and row tile, the last rows first: they see the most
  const int split = blockIdx.x % ta.splits, unit = blockIdx.x / ta.splits;
  const int h = unit % a.kv_heads, item = unit / a.kv_heads;
  {
    const int per = (a.batch + C::kThreads - 1) / C::kThreads;
    const int i0 = min(a.batch, (int)threadIdx.x * per), i1 = min(a.batch, i0 + per);
    auto tiles_of = [&](int i) {
      const Request r = load_request(a, i);
      return (r.q_len * a.group + C::kRows - 1) / C::kRows;
    };
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
      if (blockIdx.x == 0 && (int64_t)a.kv_lens[i] > ((int64_t)a.width << a.log2_bs))
        raise_flag(a.status, LQ_DEV_RANGE);
      sum += tiles_of(i);
    }
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += wsum[w];
    int begin = inc - sum;
    if (item >= begin && item < inc) {
      for (int i = i0; i < i1; ++i) {
        const int n = tiles_of(i);
        if (item < begin + n) {
          found[0] = i;
          found[1] = begin + n - 1 - item;
          break;
        }
        begin += n;
      }
    }
    __syncthreads();
  }
  if (found[0] < 0) {                                       // fewer row tiles than CTAs
    if (ta.splits > 1 && split == 0 && threadIdx.x == 0) a.meta[unit].valid = 0;
    return;
  }
  const int req = found[0], row0 = found[1] * C::kRows;
  const Request r = load_request(a, req);
  const int rows = r.q_len * a.group;
  // tiles of the tokens that a row tile's last row sees; none if it has no rows
  auto tiles_seen = [&](int t) {
    if (row0 + t * kTileRows >= rows) return 0;
    const int last = min(row0 + (t + 1) * kTileRows, rows) - 1;
    const int seen = min(r.len, r.shown + last / a.group + 1);
    return seen > 0 ? (seen + BN - 1) / BN : 0;
  };
  const int all0 = tiles_seen(0), all1 = T > 1 ? tiles_seen(1) : 0, all = max(all0, all1);
  // this CTA's tiles: `first` and the ones after it
  const int first = (int)((int64_t)all * split / ta.splits), past = (int)((int64_t)all * (split + 1) / ta.splits);
  const int n0 = max(0, min(all0, past) - first), n1 = max(0, min(all1, past) - first), tiles = max(n0, n1);
  const int seen = min(r.len, past * BN);                   // tokens fetched end here
  if (ta.splits > 1 && split == 0 && threadIdx.x == 0) {
    Tag tag = {};
    tag.i = req; tag.h = h; tag.rt = found[1]; tag.q0 = r.q0; tag.q_len = r.q_len; tag.valid = 1;
    a.meta[unit] = tag;
  }
  const int32_t* table = a.table + (int64_t)req * a.ldt;

  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&tmem_base)), "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  // columns: the row tiles' scores, then their outputs
  const uint32_t tmem_s = tmem_base, tmem_o = tmem_base + T * BN;

  if (warp < 4) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kConvertRegs));
    // ------------------------------------------------------------ codes to fp16
    // 16 codes per thread and pass.  The eight lanes of a shared-memory phase
    // take four neighbouring chunks of two rows that differ in bits 0 and 2,
    // which keeps them off each other's banks when they read codes and when
    // they write fp16, both in the 128-byte swizzle.
    const int t = threadIdx.x, c4 = t & 3, sub = t / (4 * C::kPassRows), q8 = (t >> 2) & 7;
    const int r0 = ((q8 >> 1) ^ (q8 & 1 ? 5 : 0)) + ((t >> 2) % C::kPassRows & ~7);
    auto convert = [&](auto one, const uint8_t* src, uint8_t* dst, uint64_t* src_free, uint64_t* full) {
      uint4 x[C::kPasses];
#pragma unroll
      for (int p = 0; p < C::kPasses; ++p) {
        const uint32_t off = (uint32_t)((p * C::kPassRows + r0) * D + 64 * sub + 16 * c4);
        x[p] = *reinterpret_cast<const uint4*>(src + (off ^ ((off >> 7 & 7u) << 4)));
      }
#pragma unroll
      for (int p = 0; p < C::kPasses; ++p) {
        const int row = p * C::kPassRows + r0;
        uint8_t* line = dst + sub * BN * 128 + row * 128;
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          o[2 * q] = one(w[q], 0);
          o[2 * q + 1] = one(w[q], 1);
        }
        *reinterpret_cast<uint4*>(line + (((2 * c4) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(line + (((2 * c4 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        arrive(src_free);
        arrive(full);
      }
    };
    const auto as_bf16 = [](uint32_t bytes, int half) { return codes_bf16(bytes, half ? 0x4342 : 0x4140); };
    const auto as_f16 = [](uint32_t bytes, int half) { return codes_f16(bytes ^ 0x80808080u, half ? 0x4342 : 0x4140); };
    for (int j = 0; j < tiles; ++j) {
      const int st = j & 1;
      const uint32_t before = (uint32_t)(j / 2 + 1) & 1;    // the stage's previous use
      bool ok = wait_on(&raw_full[0], (uint32_t)j & 1, timeout);
      if (j >= 2) ok = ok && wait_on(&k_free[st], before, timeout);
      if (!__all_sync(0xffffffffu, ok)) break;
      convert(as_bf16, raw, sk + st * C::kCodeBytes, &raw_free[0], &k_full[st]);
      ok = wait_on(&raw_full[1], (uint32_t)j & 1, timeout);
      if (j >= 2) ok = ok && wait_on(&v_free[st], before, timeout);
      if (!__all_sync(0xffffffffu, ok)) break;
      convert(as_f16, raw + C::kRawBytes, sv + st * C::kCodeBytes, &raw_free[1], &v_full[st]);
    }
  } else if (warp >= C::kMmaWarp) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
    if (warp == C::kFetchWarp) {
      // ------------------------------------------------------------ codes from the cache
      // lane g: the g-th part of the tile, a block or BN tokens of one
      const int step = min(1 << a.log2_bs, BN), parts = BN / step;
      const int block_lines = (D << a.log2_bs) >> 7;
      auto look_up = [&](int j) {
        const int pos = (first + j) * BN + step * lane;
        return lane < parts && pos < seen ? table[pos >> a.log2_bs] : -1;
      };
      int blk = look_up(0), issued = 0;
      for (int j = 0; j < tiles; ++j) {
        const int pos = (first + j) * BN + step * lane;
        const bool ok = (unsigned)blk < (unsigned long long)a.num_blocks;
        if (!ok && lane < parts && pos < seen) raise_flag(a.status, LQ_DEV_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * step * D;
        const int line = (blk * a.kv_heads + h) * block_lines + (((pos & ((1 << a.log2_bs) - 1)) * D) >> 7);
        blk = look_up(j + 1);
        bool go = true;
        for (int v = 0; v < 2 && go; ++v) {
          if (j > 0) go = __all_sync(0xffffffffu, wait_on(&raw_free[v], (uint32_t)(j - 1) & 1, timeout));
          if (!go) break;
          if (lane == 0) mbar_expect_tx(&raw_full[v], bytes);
          __syncwarp();
          if (ok)
            tma_load_2d(raw + v * C::kRawBytes + lane * step * D, v ? &ta.map_v : &ta.map_k, &raw_full[v], 0, line);
          ++issued;
        }
        if (!go) break;
      }
      // after a timeout: let the copies in flight land before the CTA ends
      if (*timeout)
        for (int q = max(0, issued - 2); q < issued; ++q)
          mbar_wait_bounded(&raw_full[q & 1], (uint32_t)(q >> 1) & 1, kWaitCycles / 8);
    } else if (warp < C::kFetchWarp) {
      // ------------------------------------------------------------ products
      // A warp per row tile: the products of one then run while the other's warp
      // waits (one warp for both, in line: 3950 clocks a step, 2050 of them
      // products).  The whole warp runs the loop, so that descriptors are uniform
      // values; one elected lane issues.
      const int t = warp - C::kMmaWarp, n = t == 0 ? n0 : n1;
      const uint64_t dq = desc_k_major(smem_addr(sq + t * C::kQBytes)), dk = desc_k_major(smem_addr(sk));
      const uint64_t dv = desc_mn_major(smem_addr(sv), C::kSub > 1 ? BN * 128 : 1024);
      const uint32_t my_s = tmem_s + t * BN, my_o = tmem_o + t * D;
      auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
      // scores of tile j; past this row tile's last, the other's codes are let go
      auto scores = [&](int j) {
        if (j >= tiles) return true;
        const int st = j & 1;
        bool ok = wait_on(&k_full[st], (uint32_t)(j >> 1) & 1, timeout);
        if (j < n) {
          if (j == 0) ok = ok && wait_on(&q_full[t], 0, timeout);
          // they overwrite the weights of the tile before
          else ok = ok && wait_on(&o_done[t], (uint32_t)(j - 1) & 1, timeout);
        }
        if (!all(ok)) return false;
        tc_after();
        if (elect()) {
          if (j < n) {
            const uint64_t kd = dk + (uint64_t)(st * C::kCodeBytes >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(my_s, dq + (((k >> 2) * kTileRows * 128 + (k & 3) * 32) >> 4),
                     kd + (((k >> 2) * BN * 128 + (k & 3) * 32) >> 4), Idesc<BN, true, false>::v, k > 0);
            mma_commit(&s_full[t]);
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
        if (j < n) ok = ok && wait_on(&p_full[t], (uint32_t)j & 1, timeout);
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
            const uint64_t vd = dv + (uint64_t)(st * C::kCodeBytes >> 4);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts(my_o, my_s + k * 8, vd + (k * 2048 >> 4), Idesc<D, false, true>::v, j > 0 || k > 0);
            mma_commit(&o_done[t]);
            mma_commit(&v_free[st]);
          } else {
            arrive(&v_free[st]);
          }
        }
        __syncwarp();
        return true;
      };
      bool ok = scores(0);
      for (int j = 0; j < tiles && ok; ++j) ok = add_values(j) && scores(j + 1);
    }
  } else {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;                          // row tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t my_s = tmem_s + lanes + t * BN, my_o = tmem_o + lanes + t * D;
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
    auto line_of = [&](int r32, int c) {                    // 16-byte part c of the warp's row
      const int rr = (warp & 3) * 32 + r32;
      return sq + t * C::kQBytes + (c >> 3) * kTileRows * 128 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
    };
    {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q);
      if (mine) src += (int64_t)(r.q0 + j_tok) * a.ldq + (int64_t)head * D;
      const uint32_t have = __ballot_sync(0xffffffffu, mine);
      const int c = lane & (kLanes - 1);
#pragma unroll 4
      for (int pass = 0; pass < kLanes; ++pass) {
        const int from = pass * kAtOnce + lane / kLanes;
        const uint16_t* p =
            reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), from));
        copy16(line_of(from, c), p + 8 * c, have >> from & 1 ? 16 : 0);
      }
    }

    // lane g < BN / 16: the scales of the tile's g-th 16 tokens, a tile ahead;
    // value scale -1: a block that is not there
    float nk = 0.f, nv = -1.f;
    auto fetch_scales = [&](int j) {
      const int pos = (first + j) * BN + 16 * lane;
      nk = 0.f;
      nv = -1.f;
      if (lane < BN / 16 && pos < seen) {
        const int blk = table[pos >> a.log2_bs];
        if ((unsigned)blk < (unsigned long long)a.num_blocks) {
          nk = a.ks[(int64_t)blk * a.kv_heads + h];
          nv = a.vs[(int64_t)blk * a.kv_heads + h];
        }
      }
    };
    if (n > 0) fetch_scales(0);

    // The factor of the row's scores.  Rows so large (or small) that the sums of
    // products could leave fp32's range are brought nearer to 1 by a power of two.
    float fac = a.scale_log2;
    {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t top = 0;                                     // of the two halves' magnitudes
#pragma unroll 8
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x =
            *reinterpret_cast<const uint4*>(my_line + (c >> 3) * kTileRows * 128 + (((c & 7) ^ (row & 7)) << 4));
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
      }
      top = max(top >> 16, top & 0xFFFFu);
      const int up = top >= 0x7080u ? -64 : top < 0x2000u && top != 0 ? 64 : 0;      // 2^98, 2^-63
      if (__any_sync(0xffffffffu, up != 0)) {
        const float f = __uint_as_float((uint32_t)(up + 127) << 23);
        fac *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          uint4* x = reinterpret_cast<uint4*>(my_line + (c >> 3) * kTileRows * 128 + (((c & 7) ^ (row & 7)) << 4));
          uint32_t v[4] = {x->x, x->y, x->z, x->w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[e] << 16) * f,
                                                           __uint_as_float(v[e] & 0xFFFF0000u) * f);
            v[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *x = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(&q_full[t]);
    }
    float mx = -INFINITY, un = -INFINITY, l = 0.f, unit = 0.f, floor = pow2(kFloorLeast);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const float cv = nv;
      const uint32_t parts = (1u << (BN / 16)) - 1;
      const uint32_t gone = __ballot_sync(0xffffffffu, cv < 0.f) & parts;
      uint32_t low = __ballot_sync(0xffffffffu, cv < floor) & parts;          // a missing block too; NaN is not
      float4* sc = scales[warp - 4];
      __syncwarp();
      if (lane < BN / 16) sc[lane] = make_float4(nk, log2_scale(cv), rcp(cv), 0.f);
      __syncwarp();
      if (j + 1 < n) fetch_scales(j + 1);
      const int vis0 = lim - (first + j) * BN;
      const bool masked = (first + j + 1) * BN - 1 > lim_min || low != 0;
      ok = __all_sync(0xffffffffu, wait_on(&s_full[t], (uint32_t)j & 1, timeout));
      if (!ok) break;
      tc_after();
      __syncwarp();
      bool common = !masked && !__any_sync(0xffffffffu, mx == -INFINITY);
      if (common) {
        uint32_t w[BN / 2];
        float sum = l;
        const uint32_t top = row_weights<BN>(my_s, fac, kShift - mx, unit, sc, w, sum);
        common = !__any_sync(0xffffffffu, top > kTopWeight);
        if (common) {
          l = sum;
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) tmem_st16(my_s + 16 * c, w + 16 * c);
        }
      }
      if (!common) {
        // where the maximum moves, the output so far shrinks; where the unit does, the sum
        const float2 top = row_top<BN>(my_s, fac, sc, gone, vis0);
        const bool moves = mx == -INFINITY ? top.x != -INFINITY : top.x > mx + kLead;
        const float to = moves ? ceilf(top.x) : mx, f = moves ? pow2(mx - to) : 1.f;
        const float un_to = fmaxf(un, ceilf(top.y));
        l *= pow2(un - un_to);                              // (NaN before any score: 0 of 0)
        mx = to;
        un = un_to;
        unit = unit_of(mx, un);
        Floor fl;
        fl.add(mx, un);
        floor = fl.over_warp();
        low = __ballot_sync(0xffffffffu, cv < floor || floor == INFINITY) & parts;
        if (j > 0 && __any_sync(0xffffffffu, moves)) {
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
        store_weights<BN>(my_s, fac, kShift - (mx == -INFINITY ? 0.f : mx), unit, un, sc, low, gone, vis0, l);
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) arrive(&p_full[t]);
    }

    // Outputs, by way of the rows of shared memory where the queries were (the
    // products with them are done): a warp's stores then cover whole lines.
    if (ok && n > 0) ok = __all_sync(0xffffffffu, wait_on(&o_done[t], (uint32_t)(n - 1) & 1, timeout));
    tc_after();
    __syncwarp();
    if (ok) {
      const bool whole = ta.splits == 1;
      const uint32_t rows_out = whole ? __ballot_sync(0xffffffffu, mine) : 0xffffffffu;
      // with the positions split: the row's sums as they are
      float* piece = a.part + ((int64_t)blockIdx.x * C::kRows + t * kTileRows + row) * (D + 4);
      uint8_t* dst = reinterpret_cast<uint8_t*>(
          whole ? reinterpret_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + j_tok) * a.ldo + (int64_t)head * D
                : reinterpret_cast<uint16_t*>(piece));
      const float inv = l == 0.f ? 0.f : 1.f / l;
      auto put = [&](int c, uint4 v) {
        *reinterpret_cast<uint4*>(my_line + (c >> 3) * kTileRows * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
      };
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
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t u[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * q]) * inv * unit,
                                                               __uint_as_float(o[8 * e + 2 * q + 1]) * inv * unit);
                u[q] = *reinterpret_cast<const uint32_t*>(&b);
              }
              put(4 * c + e, make_uint4(u[0], u[1], u[2], u[3]));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) put(8 * c + e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int pass = 0; pass < kLanes; ++pass) {
          const int from = pass * kAtOnce + lane / kLanes, c = lane & (kLanes - 1);
          uint8_t* p = reinterpret_cast<uint8_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), from));
          if (rows_out >> from & 1)
            *reinterpret_cast<uint4*>(p + part * 2 * D + 16 * c) = *reinterpret_cast<const uint4*>(line_of(from, c));
        }
        __syncwarp();
      }
      if (!whole) {
        piece[D] = mx;
        piece[D + 1] = l;
        piece[D + 2] = un;
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

// Joins the pieces of rows whose positions were split: a warp per row, D / 32
// neighbouring dimensions per lane.
template <int D>
__global__ void __launch_bounds__(256) attn_tiles_merge_kernel(const __grid_constant__ TileArgs ta) {
  using C = TileCfg<D>;
  constexpr int E = D / 32;
  const Args& a = ta.a;
  pdl_wait();
  pdl_launch();
  const int unit = blockIdx.x / (C::kRows / 8), row = (blockIdx.x % (C::kRows / 8)) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const Tag tag = a.meta[unit];
  const int R = tag.rt * C::kRows + row, j = R / a.group;
  if (!tag.valid || j >= tag.q_len) return;
  const float* piece = a.part + ((int64_t)unit * ta.splits * C::kRows + row) * (D + 4);
  constexpr int64_t next = (int64_t)C::kRows * (D + 4);
  float M = -INFINITY, U = -INFINITY;
  for (int p = 0; p < ta.splits; ++p) {
    M = fmaxf(M, piece[p * next + D]);
    U = fmaxf(U, piece[p * next + D + 2]);
  }
  float o[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < ta.splits; ++p) {
    const float f = pow2(piece[p * next + D] - M);
    l = fmaf(piece[p * next + D + 1], pow2(piece[p * next + D + 2] - U), l);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = *reinterpret_cast<const float2*>(piece + p * next + E * lane + e);
      o[e] = fmaf(v.x, f, o[e]);
      o[e + 1] = fmaf(v.y, f, o[e + 1]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l, back = unit_of(M, U);
  const int64_t dst = (int64_t)(tag.q0 + j) * a.ldo + (int64_t)(tag.h * a.group + R - j * a.group) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + dst + e) =
        __floats2bfloat162_rn(o[e] * inv * back, o[e + 1] * inv * back);
}

template <int D>
lq_status launch_tiles(const TileArgs& ta, const TilePlan& plan, void* stream) {
  using C = TileCfg<D>;
  static_assert(C::kSmem + 1536 <= 227 * 1024, "shared memory");
  static_assert(C::kRows * (D + 4) <= work_floats(D), "a CTA's piece fits its SM's share of the workspace");
  auto kern = attn_tiles_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  const lq_status st =
      serve::launch(kern, (unsigned)(plan.units * plan.splits), C::kThreads, C::kSmem, stream, ta);
  if (st != LQ_OK || plan.splits == 1) return st;
  return serve::launch(attn_tiles_merge_kernel<D>, (unsigned)(plan.units * (C::kRows / 8)), 256, 0, stream, ta);
}

TilePlan plan_tiles(int batch, int64_t total_q, int group, int kv_heads, int head_dim, int64_t most_tokens, int sms) {
  TilePlan p;
  const int rows = head_dim == 256 ? TileCfg<256>::kRows : TileCfg<128>::kRows;
  const int bn = head_dim == 256 ? TileCfg<256>::BN : TileCfg<128>::BN;
  // as many row tiles as there can be: every request's last one may be partial
  p.units = (total_q * group / rows + (batch < total_q ? batch : total_q)) * kv_heads;
  // split the positions where half the SMs or more would have no CTA, into parts
  // of at least four tiles
  int64_t splits = p.units > 0 ? sms / p.units : 1;
  const int64_t most = most_tokens / (4 * bn);
  if (splits > most) splits = most;
  p.splits = splits > 1 ? (int)splits : 1;
  return p;
}

lq_status launch_attn_tiles(const Args& a, const int8_t* kc, const int8_t* vc, int64_t cache_bytes, int head_dim,
                            const TilePlan& plan, void* stream) {
  if (plan.units * plan.splits > INT32_MAX) return LQ_ERR_SHAPE;
  TileArgs ta;
  ta.a = a;
  ta.splits = plan.splits;
  const int most = head_dim == 256 ? TileCfg<256>::BN : TileCfg<128>::BN, bs = 1 << a.log2_bs;
  const int box = (bs < most ? bs : most) * head_dim / 128;
  if (!encode_cache(&ta.map_k, kc, cache_bytes, box) || !encode_cache(&ta.map_v, vc, cache_bytes, box))
    return LQ_ERR_CUDA;
  switch (head_dim) {
    case 64: return launch_tiles<64>(ta, plan, stream);
    case 128: return launch_tiles<128>(ta, plan, stream);
    default: return launch_tiles<256>(ta, plan, stream);
  }
}

}  // namespace attn
}  // namespace lq
