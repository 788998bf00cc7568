// Attention of a ragged batch of query tokens over the paged 4-bit KV cache
// (the format: lq_q4.cuh).
//
// Request i has q_len_i = cu_q[i+1] - cu_q[i] query tokens, the last of its
// kv_len_i tokens, so query token j sees positions <= kv_len_i - q_len_i + j:
//     out[t, h] = sum_p w_p v_p,  w = softmax over visible p of sm_scale * q[t, h] . k_p,
// k_p and v_p of kv head h / (q_heads / kv_heads).  A query token that sees
// nothing gets zeros.
//
// The split kernel: every warp of one CTA per SM takes an equal, contiguous part
// of the batch's list of 64-token tiles (lq_attn_split.cuh) and streams it through
// its own ring of half tiles (K, V, K, V, ...): codes by TMA in rows of 128 bytes
// with the 128-byte swizzle, scales and bases by untiled bulk copies, one barrier
// per half.  Codes become fp16 values in registers (one shift, one logic and one
// fma instruction for two) and are the 16-row operand of mma.sync m16n8k16, eight
// query rows the other: scores S^T = K q^T, then O^T += V^T w^T with the weights
// transposed in registers.  Values being exact operands, the softmax knows nothing
// of scales.  bf16 queries are exact in fp16 after a power-of-two factor per row;
// fp32 queries and weights are split into two fp16 terms (22 bits).  The running
// maximum, a whole number, may fall behind by up to 2^7: most tiles only compare
// with it.
//
// Token order inside a half tile: row i of a 16-token product is token
// 4 (i / 2) + i % 2 for i < 8, two further for i + 8, so that the pairs of tokens
// a lane holds for the second product are neighbours (2 tid, 2 tid + 1, ... in the
// operand's order, 4 tid .. 4 tid + 3 in the tile's) and the lanes' reads of V
// spread over the banks.
#include "lq_attn_paged.cuh"
#include "lq_attn_q4.cuh"
#include "lq_attn_split.cuh"

namespace lq {
namespace q4 {

using namespace attn;

constexpr int kTokens = 64;                    // tokens per tile
constexpr int kMTiles = kTokens / 16;

struct SplitArgs {
  CacheArgs ca;
  int halves;                // of a warp's ring
};

template <int D, int NT, bool F32>
struct Cfg {
  // 12 warps of at most 168 registers where the output tile and the queries
  // leave room, else 8 of at most 255
  static constexpr int kWarps = D * NT * (F32 ? 2 : 1) <= 128 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalfBytes = kTokens * D / 2;         // the K or the V codes of a tile
  static constexpr int kPiece = piece_floats(kRows, D);
  static constexpr int kEnds = 2 * kWarps;                 // pieces that the warps may leave
  static constexpr int kRowBytes = 5 * kEnds * kRows * 4;                // the pieces' rows
  static constexpr int kMostHalves = 8;
  // a half: codes, scales, what tile it is, its barrier
  static constexpr int per_half(int groups) { return kHalfBytes + 4 * kTokens * groups + 24; }
  static constexpr int halves(int groups) {
    const int fit = (227 * 1024 - 1024 - 2048 - kRowBytes) / (kWarps * per_half(groups));
    return fit < kMostHalves ? fit : kMostHalves;
  }
  static constexpr int smem(int groups) { return kWarps * halves(groups) * per_half(groups) + kRowBytes + 1024; }
};

// Codes of a half lie in lines of 128 bytes whose 16-byte chunks are swizzled by the
// line's number.  A lane reads at one offset (k_at, v_at) and others that differ from
// it by constants alone: some bits flipped, then a distance.
template <int D>
struct At {
  static constexpr int row = D / 2;            // bytes of a token
  static __device__ __forceinline__ uint32_t swizzled(uint32_t off) { return off ^ ((off >> 7 & 7u) << 4); }
  // scores: token tg of the first product, bytes tid * D / 8 ...; of product m, `two`
  // tokens further, chunk j
  static __device__ __forceinline__ uint32_t k_at(int tg, int tid) { return swizzled(tg * row + tid * (D / 8)); }
  static __device__ __forceinline__ uint32_t k_at(uint32_t at, int m, int two, int j) {
    const uint32_t flip = (D == 64 ? (m & 1) * 64u ^ two * 64u : D == 128 ? two * 16u : two * 32u) ^ j * 16u;
    return (at ^ flip) + m * 16 * row + (D == 64 ? 0 : two * 2 * row);
  }
  // values: token 4 tid of the first product, bytes g * D / 16 ...; of product m, r
  // tokens further
  static __device__ __forceinline__ uint32_t v_at(int g, int tid) { return swizzled(4 * tid * row + g * (D / 16)); }
  static __device__ __forceinline__ uint32_t v_at(uint32_t at, int m, int r) {
    const uint32_t flip =
        D == 64 ? (m & 1) * 64u ^ r * 32u : D == 128 ? (r & 1) * 64u ^ (r >> 1) * 16u : (uint32_t)r * 16u;
    return (at ^ flip) + m * 16 * row + (D == 64 ? 0 : D == 128 ? (r >> 1) * 128 : r * 128);
  }
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  }
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(Cfg<D, NT, F32>::kThreads, 1)
split_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
             const __grid_constant__ SplitArgs sa) {
  using C = Cfg<D, NT, F32>;
  const Args& a = sa.ca.a;
  constexpr int kWarps = C::kWarps, kRows = C::kRows;
  constexpr int KS = D / 16;                   // k steps of the scores, m tiles of the output
  constexpr int Q2 = F32 ? 2 : 1;              // fp16 terms of a query or weight
  extern __shared__ uint8_t q4_smem_raw[];
  // (an offset, not a cast to and from a number, lets the compiler see shared memory)
  uint8_t* smem = q4_smem_raw + ((0u - smem_addr(q4_smem_raw)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tid = lane & 3;
  const int S = sa.halves, groups = D >> sa.ca.log2_group;
  const Masks masks;
  uint8_t* ring = smem + warp * S * C::kHalfBytes;
  uint8_t* after = smem + kWarps * S * C::kHalfBytes;
  uint32_t* scales = reinterpret_cast<uint32_t*>(after) + warp * S * kTokens * groups;
  after += kWarps * S * kTokens * groups * 4;
  int4* infos = reinterpret_cast<int4*>(after) + warp * S;                         // which tile a K half is of
  after += kWarps * S * 16;
  uint64_t* bars = reinterpret_cast<uint64_t*>(after) + warp * S;
  after += kWarps * S * 8;
  // maxima, sums and units of the warps' pieces, and their weights when they are joined
  float* piece_m = reinterpret_cast<float*>(after);
  float* piece_l = piece_m + C::kEnds * kRows;
  float* piece_u = piece_l + C::kEnds * kRows;
  float* piece_f = piece_u + C::kEnds * kRows;
  float* piece_w = piece_f + C::kEnds * kRows;
  __shared__ Tag tags[2 * kWarps];
  __shared__ int order[2 * kWarps];            // the pieces that are there, in order
  __shared__ long long wsum[kWarps];
  __shared__ int2 asked[kWarps];               // the warp's current request: first query token, how many
  __shared__ int timeout, q_end;
  // a tile is one block, or part of one, or up to four
  const int log2_step = min(a.log2_bs, 6), step = 1 << log2_step, parts = kTokens >> log2_step;
  // where the warps' first pieces go when more follow; a last one takes the
  // warp's ring, which is not filled again
  float* firsts = a.part + ((int64_t)gridDim.x * 2 + (int64_t)blockIdx.x * kWarps) * C::kPiece;

  if (lane == 0) {
#pragma unroll 1
    for (int s = 0; s < S; ++s) mbar_init1(bars + s, 1);
    mbar_init_fence();
    tags[2 * warp].valid = tags[2 * warp + 1].valid = 0;
  }
  pdl_wait();
  pdl_launch();
  if (threadIdx.x == 0) {
    timeout = 0;
    q_end = a.cu_q[a.batch];
  }
  Cursor ci;                                   // the tile whose halves are fetched next
  const int n = part_of_warp<kRows, kWarps, kTokens>(a, reinterpret_cast<long long*>(smem), wsum, ci);

  if (n > 0) {
    // lane i < parts: the block of the tile's i-th part, and its head's place in the pool
    int blk = -1, at_head = 0;
    bool blk_ok = false;
    uint32_t there = 0;                        // the parts whose block is in the pool
    auto load_block = [&]() {
      const int p = ci.t * kTokens + step * lane;
      blk = -1;
      if (lane < parts && p < ci.len) blk = a.table[ci.i * a.ldt + (p >> a.log2_bs)];
    };
    const int rows_per_block = (D / 2 << a.log2_bs) >> 7;
    int qi = 0;                                // halves issued
    auto issue = [&](int s) {
      const bool is_v = qi & 1;
      if (!is_v) {
        blk_ok = (unsigned)blk < (unsigned long long)a.num_blocks;
        at_head = blk * a.kv_heads + ci.h;
        if (lane < parts && !blk_ok && ci.t * kTokens + step * lane < ci.len)
          raise_flag(a.status, LQ_DEV_RANGE);  // a block id outside the pool
        there = __ballot_sync(0xffffffffu, blk_ok);
        // bit 16: the rows' last tile; from 17 on, the parts that are not there
        if (lane == 0)
          infos[s] = make_int4(ci.i, ci.rt, ci.h | (ci.t + 1 == ci.nt ? 1 << 16 : 0) |
                                                (int)(~there & ((1u << parts) - 1)) << 17, ci.t);
      }
      if (lane == 0) mbar_expect_tx(bars + s, __popc(there) * step * (D / 2 + 4 * groups));
      __syncwarp();
      if (blk_ok) {
        const int off = (ci.t * kTokens) & ((1 << a.log2_bs) - 1);
        tma_load_2d(ring + s * C::kHalfBytes + lane * step * (D / 2), is_v ? &map_v : &map_k, bars + s, 0,
                    at_head * rows_per_block + ((off * (D / 2)) >> 7));
        bulk_load(scales + (s * kTokens + lane * step) * groups,
                  (is_v ? sa.ca.vs : sa.ca.ks) + (((int64_t)at_head << a.log2_bs) + off) * groups, step * groups * 4, bars + s);
      }
      if (++qi < 2 * n && is_v) {
        advance<kRows, kTokens>(a, ci);
        load_block();
      }
    };

    load_block();
    int4 info = make_int4(ci.i, ci.rt, ci.h, ci.t);
    uint32_t qf[NT][KS][2][Q2];
    float acc[KS][NT][4];
    float mx[NT][2], sum_l[NT][2], fac[NT][2];
    int lim[NT][2];                            // last position each of this thread's rows sees
    int lim_min = 0, len = 0;
    bool fresh = true, seg_starts = false, more_before = false, dead = false;
    float sc[kMTiles][NT][4];                  // the tile's scores, then exponents
    const int tg = (g >> 1) * 4 + (g & 1);     // the token of row g of a product
    const uint32_t k_at = At<D>::k_at(tg, tid), v_at = At<D>::v_at(g, tid);
    const int v_grp = (g * (D / 8)) >> sa.ca.log2_group;
    int s = 0;
    uint32_t ph = 1;

    // half tiles one after the other, K and V in turn; the first S steps only
    // fill the ring, so that fetching stands in the code once
#pragma unroll 1
    for (int st = -S; st < 2 * n; ++st) {
      const bool skip = st < 0;
      if (st == -S || (!skip && !(st & 1))) {
        // (the first segment's rows are fetched beside its first block id)
        if (!skip) info = infos[s];            // written when the half was issued
        if (fresh) {
          fresh = false;
          const int h = info.z & 0xFFFF;
          seg_starts = info.w == 0;
          // this segment's query rows: lane (g, tid) holds row g's dimensions
          // tid * D/4 ...; a power of two per row brings them into fp16's range
          const Request r = load_request(a, info.x);
          len = r.len;
          __syncwarp();                        // every lane has read the segment before's
          if (lane == 0) asked[warp] = make_int2(r.q0, r.q_len);
          lim_min = INT_MAX;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float v[D / 4];
            int64_t at;
            if (row_at(a, r.q0, r.q_len, info.y * kRows + nt * 8 + g, h, a.ldq, D, &at)) {
              at += tid * (D / 4);
              if constexpr (F32) {
                const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  const float4 x = p[c];
                  v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
                }
              } else {
                const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) + at);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                  const uint4 x = p[c];
                  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    v[8 * c + 2 * e] = __uint_as_float(u[e] << 16);
                    v[8 * c + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                  }
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 4; ++c) v[c] = 0.f;
            }
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < D / 4; ++c) top = fmaxf(top, fabsf(v[c]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^e with the row's largest value in [2^13, 2^14)
            const int eb = (int)(__float_as_uint(top) >> 23);
            const int ex = min(126, max(-116, 140 - eb));
            const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
            const float down = a.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
            // step (word w of codes, half e): codes 2 e and 2 e + 4, then 2 e + 1 and 2 e + 5
#pragma unroll
            for (int c = 0; c < KS; ++c) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at8 = 8 * (c >> 1) + 2 * (c & 1) + e;
                const float x = v[at8] * up, y = v[at8 + 4] * up;
                qf[nt][c][e][0] = pack_f16(x, y);
                if constexpr (F32) qf[nt][c][e][1] = rest_f16(qf[nt][c][e][0], x, y);
              }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              fac[nt][c] = __shfl_sync(0xffffffffu, down, 4 * (2 * tid + c));
              const int j = (info.y * kRows + nt * 8 + 2 * tid + c) / a.group;
              lim[nt][c] = j < r.q_len ? min(r.shown + j, r.len - 1) : r.len - 1;
              lim_min = min(lim_min, lim[nt][c]);
              mx[nt][c] = -INFINITY;
              sum_l[nt][c] = 0.f;
            }
          }
          lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
          lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));
#pragma unroll
          for (int c = 0; c < KS; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[c][nt][e] = 0.f;
        }
      }
      if (!skip) {
        if (!mbar_wait_bounded(bars + s, ph, kWaitCycles)) {
          timeout = 1;
          dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
      }
      const bool ends = info.z >> 16 & 1;
      const uint8_t* codes = ring + s * C::kHalfBytes;
      uint32_t* params = scales + s * kTokens * groups;
      if (!skip && !(st & 1)) {
        // scores S^T [64 tokens x 8 NT rows]
#pragma unroll
        for (int mt = 0; mt < kMTiles; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
          constexpr int NW = D == 64 ? 2 : 4;          // words of codes per load, of one group
#pragma unroll
          for (int j = 0; j < D / 32 / NW; ++j) {
            const int grp = (tid * (D / 4) + 32 * j) >> sa.ca.log2_group;
            uint32_t x[NW], y[NW];
            load_words(codes + At<D>::k_at(k_at, mt, 0, j), x);
            load_words(codes + At<D>::k_at(k_at, mt, 1, j), y);
            const uint32_t px = params[(16 * mt + tg) * groups + grp], py = params[(16 * mt + tg + 2) * groups + grp];
            const uint32_t sx = twice_low(px), bx = twice_high(px), sy = twice_low(py), by = twice_high(py);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
              const uint32_t vx[4] = {fma_h2(masks.pair<0>(x[w]), sx, bx), fma_h2(masks.pair<1>(x[w]), sx, bx),
                                      fma_h2(masks.pair<2>(x[w]), sx, bx), fma_h2(masks.pair<3>(x[w]), sx, bx)};
              const uint32_t vy[4] = {fma_h2(masks.pair<0>(y[w]), sy, by), fma_h2(masks.pair<1>(y[w]), sy, by),
                                      fma_h2(masks.pair<2>(y[w]), sy, by), fma_h2(masks.pair<3>(y[w]), sy, by)};
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int f = 0; f < Q2; ++f) {
                    const int c = 2 * (NW * j + w) + e;
                    mma16816(sc[mt][nt], vx[2 * e], vy[2 * e], vx[2 * e + 1], vy[2 * e + 1], qf[nt][c][0][f],
                             qf[nt][c][1][f]);
                  }
            }
          }
        }
      } else if (!skip) {
        const int p0 = info.w * kTokens;
        // exponents less the running maximum, plus the shift
        float lead = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float b0 = kShift - (mx[nt][0] == -INFINITY ? 0.f : mx[nt][0]);
          const float b1 = kShift - (mx[nt][1] == -INFINITY ? 0.f : mx[nt][1]);
#pragma unroll
          for (int mt = 0; mt < kMTiles; ++mt) {
            sc[mt][nt][0] = fmaf(sc[mt][nt][0], fac[nt][0], b0);
            sc[mt][nt][1] = fmaf(sc[mt][nt][1], fac[nt][1], b1);
            sc[mt][nt][2] = fmaf(sc[mt][nt][2], fac[nt][0], b0);
            sc[mt][nt][3] = fmaf(sc[mt][nt][3], fac[nt][1], b1);
          }
        }
        const int gone = info.z >> 17;
        if (p0 + kTokens - 1 > lim_min || gone) {
          // tokens that some row does not see, or of a block that is not there
#pragma unroll
          for (int mt = 0; mt < kMTiles; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (p0 + 16 * mt + tg + (e & 2) > lim[nt][e & 1] || (gone >> (16 * mt >> log2_step) & 1))
                  sc[mt][nt][e] = -INFINITY;
          // what the slots without a token hold must not meet the weights, 0 though they are
          for (int t = lane; t < kTokens; t += 32)
            if (p0 + t >= len || (gone >> (t >> log2_step) & 1))
              for (int k = 0; k < groups; ++k) params[t * groups + k] = 0u;
          fence_proxy_async_smem();
          __syncwarp();
        }
        bool empty = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          empty |= mx[nt][0] == -INFINITY || mx[nt][1] == -INFINITY;
#pragma unroll
          for (int mt = 0; mt < kMTiles; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) lead = fmaxf(lead, sc[mt][nt][e]);
        }
        // a weight too large for the shift, or a row without a maximum: take the
        // tile's maxima in
        if (__any_sync(0xffffffffu, lead > kShift + kLead || empty)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < kMTiles; ++mt) {
              m0 = fmaxf(m0, fmaxf(sc[mt][nt][0], sc[mt][nt][2]));
              m1 = fmaxf(m1, fmaxf(sc[mt][nt][1], sc[mt][nt][3]));
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
              m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // how far the maximum moves; everything so far shrinks by as much
              float d = ceilf((c ? m1 : m0) - kShift);   // by whole powers of two
              const bool none = mx[nt][c] == -INFINITY;
              if (!none) d = fmaxf(d, 0.f);
              if (d == -INFINITY) d = 0.f;               // still nothing
              else mx[nt][c] = none ? d : mx[nt][c] + d;
              const float f = none ? 0.f : ex2(-d);
              sum_l[nt][c] *= f;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                acc[j][nt][c] *= f;
                acc[j][nt][c + 2] *= f;
              }
#pragma unroll
              for (int mt = 0; mt < kMTiles; ++mt) {
                sc[mt][nt][c] -= d;
                sc[mt][nt][c + 2] -= d;
              }
            }
          }
        }
        // O^T [D x 8 NT rows] += V^T w^T; lane g holds dimensions g * D/8 ...
#pragma unroll
        for (int mt = 0; mt < kMTiles; ++mt) {
          // weights and their sums; the weights transposed, as fp16
          uint32_t pb[NT][2][Q2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(sc[mt][nt][e]);
            sum_l[nt][0] += w[0] + w[2];
            sum_l[nt][1] += w[1] + w[3];
            const uint32_t x0 = pack_f16(w[0], w[1]), x1 = pack_f16(w[2], w[3]);
            pb[nt][0][0] = transpose8(x0);
            pb[nt][1][0] = transpose8(x1);
            if constexpr (F32) {
              pb[nt][0][1] = transpose8(rest_f16(x0, w[0], w[1]));
              pb[nt][1][1] = transpose8(rest_f16(x1, w[2], w[3]));
            }
          }
          constexpr int NW = D / 64;             // words of codes per token and lane
          uint32_t v[4][NW], pr[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            load_words(codes + At<D>::v_at(v_at, mt, r), v[r]);
            pr[r] = params[(16 * mt + 4 * tid + r) * groups + v_grp];
          }
          const uint32_t s01 = __byte_perm(pr[0], pr[1], 0x5410), b01 = __byte_perm(pr[0], pr[1], 0x7632);
          const uint32_t s23 = __byte_perm(pr[2], pr[3], 0x5410), b23 = __byte_perm(pr[2], pr[3], 0x7632);
#pragma unroll
          for (int c = 0; c < 2 * NW; ++c) {
            // four dimensions of two tokens side by side
            const uint32_t sel = c & 1 ? 0x7632 : 0x5410;
            const uint32_t x = __byte_perm(v[0][c >> 1], v[1][c >> 1], sel), y = __byte_perm(v[2][c >> 1], v[3][c >> 1], sel);
            const uint32_t vx[4] = {fma_h2(masks.pair<0>(x), s01, b01), fma_h2(masks.pair<1>(x), s01, b01),
                                    fma_h2(masks.pair<2>(x), s01, b01), fma_h2(masks.pair<3>(x), s01, b01)};
            const uint32_t vy[4] = {fma_h2(masks.pair<0>(y), s23, b23), fma_h2(masks.pair<1>(y), s23, b23),
                                    fma_h2(masks.pair<2>(y), s23, b23), fma_h2(masks.pair<3>(y), s23, b23)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float (&o)[4] = acc[2 * c + half][nt];
                const uint32_t a0 = vx[2 * half], a1 = vx[2 * half + 1], a2 = vy[2 * half], a3 = vy[2 * half + 1];
                if constexpr (F32) {
                  // the matrix unit truncates its sums: over thousands of
                  // positions that would be a bias, so they are added here
                  float d[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(d, a0, a1, a2, a3, pb[nt][0][1], pb[nt][1][1]);
                  mma16816(d, a0, a1, a2, a3, pb[nt][0][0], pb[nt][1][0]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] += d[e];
                } else {
                  mma16816(o, a0, a1, a2, a3, pb[nt][0][0], pb[nt][1][0]);
                }
              }
            }
          }
        }
      }
      __syncwarp();                            // every lane has read the half: refill it
      if (qi < 2 * n) issue(s);
      if (++s == S) { s = 0; ph ^= 1; }

      if ((ends || st + 1 == 2 * n) && !skip && (st & 1)) {
        float l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = sum_l[nt][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            l[nt][c] = x;
          }
        const int h = info.z & 0xFFFF;
        if (ends && seg_starts) {
          // all of the rows' tokens: the outputs, D/8 dimensions per lane and row
          const int2 q = asked[warp];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              int64_t at;
              if (row_at(a, q.x, q.y, info.y * kRows + nt * 8 + 2 * tid + c, h, a.ldo, D, &at)) {
                at += g * (D / 8);
                const float inv = inverse(l[nt][c]);
                if constexpr (F32) {
                  float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at);
#pragma unroll
                  for (int j = 0; j < KS / 2; ++j)
                    p[j] = make_float4(acc[2 * j][nt][c] * inv, acc[2 * j][nt][c + 2] * inv,
                                       acc[2 * j + 1][nt][c] * inv, acc[2 * j + 1][nt][c + 2] * inv);
                } else {
                  uint32_t w[KS];
#pragma unroll
                  for (int j = 0; j < KS; ++j) {
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(acc[j][nt][c] * inv, acc[j][nt][c + 2] * inv);
                    w[j] = *reinterpret_cast<const uint32_t*>(&h2);
                  }
                  uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at);
#pragma unroll
                  for (int j = 0; j < KS / 4; ++j)
                    p[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                }
              }
            }
        } else {
          const int slot = more_before ? 1 : 0;
          float* dst = st + 1 == 2 * n ? reinterpret_cast<float*>(ring) : firsts + warp * C::kPiece;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int row = nt * 8 + 2 * tid + c;
#pragma unroll
              for (int j = 0; j < KS; ++j)
                *reinterpret_cast<float2*>(dst + row * D + g * (D / 8) + 2 * j) =
                    make_float2(acc[j][nt][c], acc[j][nt][c + 2]);
              if (g == 0) {
                const int at = (2 * warp + slot) * kRows + row;
                piece_m[at] = mx[nt][c];
                piece_l[at] = l[nt][c];
                piece_u[at] = mx[nt][c] - kShift;      // the unit of the sum: 2^that
              }
            }
          if (lane == 0) {
            Tag& t = tags[2 * warp + slot];
            t.i = info.x; t.rt = info.y; t.h = h; t.q0 = asked[warp].x; t.q_len = asked[warp].y;
            t.starts = seg_starts; t.ends = ends; t.valid = st + 1 == 2 * n ? 1 : 2;
          }
        }
        fresh = true;
        more_before = true;
      }
    }
    if (dead) {
      // let the copies in flight land before the CTA ends
#pragma unroll 1
      for (int i = 0; i < S; ++i) mbar_wait_bounded(bars + i, ph ^ (i < s ? 1u : 0u), kWaitCycles / 8);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && timeout) raise_flag(a.status, LQ_DEV_TIMEOUT);
  zero_unowned<D, C::kThreads, F32>(a, q_end);
  join_pieces<D, kRows, kWarps, F32>(a, tags, order, piece_m, piece_l, piece_u, piece_f, piece_w, [&](int w, int valid) {
    return valid == 2 ? firsts + w * C::kPiece : reinterpret_cast<const float*>(smem + w * S * C::kHalfBytes);
  });
}

template <int D, int NT, bool F32>
lq_status launch_split(const CacheArgs& ca, const CUtensorMap& mk, const CUtensorMap& mv, int ctas, void* stream) {
  using C = Cfg<D, NT, F32>;
  static_assert(C::halves(D / 32) >= 2 && C::smem(1) + 2048 <= 227 * 1024 && C::smem(D / 32) + 2048 <= 227 * 1024,
                "shared memory");
  static_assert(C::halves(D / 32) * C::kHalfBytes >= C::kRows * D * 4, "a warp's last piece fits its ring");
  static_assert(C::kWarps * C::halves(D / 32) * C::kHalfBytes >= LQ_MAX_REQUESTS * 8, "the prefix sums fit the rings");
  static_assert((2 + C::kWarps) * C::kPiece <= work_floats(D), "the pieces fit the workspace");
  auto kern = split_kernel<D, NT, F32>;
  const int groups = D >> ca.log2_group, smem = C::smem(groups);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  const SplitArgs args{ca, C::halves(groups)};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mk, mv, args);
  if (e == cudaSuccess) {
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, attn_merge_kernel<D, NT, F32>, ca.a, ctas);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  return check_launch();
}

// Whether the tensor-core kernel takes a bf16 call: by the query rows that an
// average request has for each kv head.  Its time hardly depends on them up to 128,
// the split kernel's grows with every 16 (every 8 for head_dim 256).  Measured at 8 kv
// heads of one to four query heads, this kernel's time against the split kernel's at
// 16 / 24 / 32 / 48 / 64 rows, in us:
//   head_dim                      64                   128                        256
//   16 requests of 4000  55: 27/41/41/56/70    65: 37/62/62/84/109      83: 83/116/155/215/293
//   one of 32000 tokens  41: 21/27/27/34/41    44: 29/38/38/48/59       59: 50/63/80/108/139
//   one of 4000 tokens   21: 13/13/13/14/17    23: 16/17/17/21/21       31: 19/26/26/30/35
//   24 of 500 to 12000   96: 36/59/60/81/101  114: 58/92/95/130/159    144: 123/167/211/305/397
// With more units than CTAs can share, its 9 us beside a unit's tiles show where contexts
// are short, of which the host knows a bound:
//   256 requests of 300  149: 39/60/61/81/103 180: 66/97/97/139/171    190: 140/188/240/337/422
//   256 of 1000          248: 82/144/148/204/272  291: 128/223/224/318/422  360: 326/470/617/861/1157
// (Passes of 32 rows, queries in shared memory, were no better than two of 16: 69 us to
// 62 for 32 rows of 16 requests of 4000, head_dim 128.)
// All of these are requests with equal rows.  The average decides for a mixed batch as a
// whole: a chunk of 512 tokens among 63 decode requests of 100 to 16000 (32 query heads for
// 8 kv heads of 128) takes this kernel and 305 us, the two apart 41 and 83; one of 2000
// among 127 472, apart 129 and 110.
bool many_rows(int batch, int64_t total_q, int group, int kv_heads, int head_dim, int64_t most_tokens, int sms) {
  if (batch <= 0) return false;
  const int64_t rows = (total_q + batch - 1) / batch * group;
  if (rows <= (head_dim == 64 ? 48 : head_dim == 128 ? 32 : 16)) return false;
  if (rows > (head_dim == 64 ? 64 : head_dim == 128 ? 48 : 24)) return true;
  return (int64_t)batch * kv_heads <= 4 * sms || most_tokens >= (head_dim == 256 ? 320 : 704);
}

}  // namespace q4
}  // namespace lq

using namespace lq;

extern "C" size_t lq_attention_paged_q4_workspace_size(int batch, int64_t total_q, int q_heads, int kv_heads,
                                                       int head_dim) {
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || total_q > INT32_MAX || kv_heads <= 0 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || q_heads > 1024 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const int ctas = attn::cta_count();
  const size_t split = attn::meta_bytes(ctas) + (size_t)ctas * attn::work_floats(head_dim) * sizeof(float);
  if (!q4::many_rows(batch, total_q, q_heads / kv_heads, kv_heads, head_dim, INT64_MAX, ctas)) return split;
  const size_t tiles = q4::tiles_workspace(batch, total_q, q_heads, kv_heads, head_dim, ctas);
  return split > tiles ? split : tiles;
}

extern "C" lq_status lq_attention_paged_q4(const void* q_dev, int64_t ldq, int dtype, int64_t total_q,
                                           const int32_t* cu_q_dev, const int32_t* kv_lens_dev, int batch,
                                           const int32_t* block_table_dev, int64_t table_stride, int table_width,
                                           const uint8_t* k_cache_dev, const uint16_t* k_scales_dev,
                                           const uint8_t* v_cache_dev, const uint16_t* v_scales_dev,
                                           int64_t num_blocks, int block_size, int q_heads, int kv_heads,
                                           int head_dim, int group_size, float sm_scale, void* out_dev, int64_t ldo,
                                           void* workspace_dev, size_t workspace_bytes, int32_t* dev_status_dev,
                                           void* stream) {
  LQ_NVTX_RANGE("lq_attention_paged_q4");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  if (!serve::valid_block_size(block_size) || !q4::valid_dims(head_dim, group_size)) return LQ_ERR_UNSUPPORTED;
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || q_heads > 1024) return LQ_ERR_SHAPE;
  const int64_t esize = dtype == LQ_BF16 ? 2 : 4, cols = (int64_t)q_heads * head_dim;
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || total_q > INT32_MAX || num_blocks < 0 ||
      num_blocks > INT32_MAX || table_width < 0 || table_stride < table_width || ldq < cols || ldo < cols ||
      (ldq * esize) % 16 != 0 || (ldo * esize) % 16 != 0)
    return LQ_ERR_SHAPE;
  // rows of 128 bytes of codes are counted in 32 bits (a pool of 256 GB for K alone)
  const int64_t block_rows = (int64_t)kv_heads * block_size * head_dim / 256;
  if (num_blocks > INT32_MAX / block_rows) return LQ_ERR_SHAPE;
  if (total_q > INT32_MAX / q_heads) return LQ_ERR_SHAPE;       // query rows are counted in 32 bits
  if (!(fabsf(sm_scale) <= 3.402823466e38f)) return LQ_ERR_ARG;
  if (total_q == 0) return LQ_OK;
  if (batch == 0) return LQ_ERR_SHAPE;
  if (q_dev == nullptr || out_dev == nullptr || cu_q_dev == nullptr || kv_lens_dev == nullptr ||
      workspace_dev == nullptr || !aligned16(q_dev) || !aligned16(out_dev) || !aligned4(cu_q_dev) ||
      !aligned4(kv_lens_dev) || !aligned16(workspace_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  if (table_width > 0 && (block_table_dev == nullptr || !aligned4(block_table_dev))) return LQ_ERR_ARG;
  if (num_blocks > 0 && (k_cache_dev == nullptr || v_cache_dev == nullptr || k_scales_dev == nullptr ||
                         v_scales_dev == nullptr || !aligned16(k_cache_dev) || !aligned16(v_cache_dev) ||
                         !aligned16(k_scales_dev) || !aligned16(v_scales_dev)))
    return LQ_ERR_ARG;
  if (workspace_bytes < lq_attention_paged_q4_workspace_size(batch, total_q, q_heads, kv_heads, head_dim))
    return LQ_ERR_SHAPE;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  q4::CacheArgs ca;
  attn::Args& a = ca.a;
  a = attn::Args{};
  a.q = q_dev; a.ldq = ldq; a.total_q = total_q; a.cu_q = cu_q_dev; a.kv_lens = kv_lens_dev; a.batch = batch;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width; a.num_blocks = num_blocks;
  a.log2_bs = serve::log2_of(block_size); a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads;
  a.scale_log2 = sm_scale * 1.4426950408889634f; a.out = out_dev; a.ldo = ldo; a.status = dev_status_dev;
  a.meta = reinterpret_cast<attn::Tag*>(workspace_dev);
  const int ctas = attn::cta_count();
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace_dev) + attn::meta_bytes(ctas));
  ca.ks = reinterpret_cast<const uint32_t*>(k_scales_dev); ca.vs = reinterpret_cast<const uint32_t*>(v_scales_dev);
  ca.log2_group = serve::log2_of(group_size);
  ca.kc = k_cache_dev; ca.vc = v_cache_dev;
  const int64_t most_tokens = (int64_t)table_width * block_size;
  if (dtype == LQ_BF16 && q4::many_rows(batch, total_q, a.group, kv_heads, head_dim, most_tokens, ctas))
    return q4::launch_tiles(ca, head_dim, most_tokens, ctas, workspace_dev, stream);
  // a pool without blocks: no copy is issued, any valid map will do
  const void* kc = num_blocks > 0 ? (const void*)k_cache_dev : workspace_dev;
  const void* vc = num_blocks > 0 ? (const void*)v_cache_dev : workspace_dev;
  const int64_t bytes = num_blocks > 0 ? num_blocks * block_rows * 128 : 32768;
  CUtensorMap mk, mv;
  const int box = (block_size < q4::kTokens ? block_size : q4::kTokens) * head_dim / 256;
  if (!attn::encode_cache(&mk, kc, bytes, box) || !attn::encode_cache(&mv, vc, bytes, box)) return LQ_ERR_CUDA;
  // eight query rows per pass over the codes, sixteen where the average request has more
  const bool few = ((total_q + batch - 1) / batch) * a.group <= 8;
  if (dtype == LQ_F32) {
    if (head_dim == 64) return q4::launch_split<64, 1, true>(ca, mk, mv, ctas, stream);
    if (head_dim == 128) return q4::launch_split<128, 1, true>(ca, mk, mv, ctas, stream);
    return q4::launch_split<256, 1, true>(ca, mk, mv, ctas, stream);
  }
  if (head_dim == 256) return q4::launch_split<256, 1, false>(ca, mk, mv, ctas, stream);
  if (head_dim == 64) return few ? q4::launch_split<64, 1, false>(ca, mk, mv, ctas, stream)
                                 : q4::launch_split<64, 2, false>(ca, mk, mv, ctas, stream);
  return few ? q4::launch_split<128, 1, false>(ca, mk, mv, ctas, stream)
             : q4::launch_split<128, 2, false>(ca, mk, mv, ctas, stream);
}
