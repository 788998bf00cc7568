// Attention of a ragged batch of query tokens over the paged 8-bit KV cache.
//
// Request i has q_len_i = cu_q[i+1] - cu_q[i] query tokens, the last of its
// kv_len_i tokens, so query token j sees positions <= kv_len_i - q_len_i + j:
//     out[t, h] = sum_p w_p v_p,  w = softmax over visible p of
//                 sm_scale * q[t, h] . k_p,   k_p = s_k[block, g] c_k, v_p = s_v[block, g] c_v,
// g = h / (q_heads / kv_heads).  A query token that sees nothing gets zeros.
//
// With x_p = sm_scale log2(e) s_k (q . c_k) + log2(s_v) the output is
//     (sum_p 2^x_p c_v) / (sum_p 2^x_p / s_v):
// the value scale rides in the exponent, so one weight per position serves
// both sums, codes enter the matrix products as they are, and value scales of
// any size cannot push a weight out of fp16's range (the running maximum is
// that of x, not of the score).
//
// The split kernel, for few query rows per kv head (decode steps, drafted
// tokens), is bound by reading the codes from HBM: every code is used for at
// most 16 rows.  The batch's work is a list of 32-token tiles (request, tile of
// rows, kv head, tokens), and every warp of one CTA per SM takes an equal,
// contiguous part of it, whatever the lengths are: no request waits for
// another's long tail.  A warp streams its tiles through its own ring of
// stages by TMA (the codes' rows of 128 bytes in the 128-byte swizzle, so that
// the fragment loads below meet no bank twice) with no barrier shared between
// warps, keeps running maxima, sums and the output tile in registers, and
// writes an output when it has seen all of a row's tiles.  Pieces of rows are
// joined through shared memory within a CTA and by the merge kernel between
// CTAs, in the order of the tiles, so that equal calls give equal bits.
//
// Products on mma.sync m16n8k16 with the codes as the 16-row operand (fp16,
// exact) and eight query rows as the other: scores S^T = C_k q^T, then
// O^T += C_v^T w^T with the weights transposed in registers.  tcgen05 needs 64
// or 128 rows to earn its operand traffic through shared memory; at 8 or 16
// rows it would still be the codes' bytes that bound the kernel.  bf16 queries
// are exact in fp16 after a power-of-two factor per row; fp32 queries and
// weights are split into two fp16 terms (22 bits).
#include "lq_attn_paged.cuh"

namespace lq {
namespace attn {

constexpr int kTile = 32;                      // tokens per tile

template <int D, int NT>
struct Cfg {
  static constexpr int kWarps = D == 256 ? 4 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * kTile * D;        // K codes, then V codes
  // in shared memory: the rings, the warps' first pieces, scales and barriers
  static constexpr int kPiece = kRows * (D + 2);           // floats: output rows, maxima, sums
  static constexpr int kFixed = kWarps * kPiece * 4 + 1024 + 640;   // with the alignment and the static part
  static constexpr int kFit = (227 * 1024 - kFixed) / (kWarps * (kStageBytes + 24));
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRing + kWarps * kPiece * 4 + kWarps * kStages * 24 + 1024;
};

// A place in the list of tiles.
struct Cursor {
  int i;             // request
  int64_t rt;        // tile of rows
  int h;             // kv head
  int t, nt;         // tile of tokens, and how many the request has
  int64_t nrt;
  Request r;
};

template <int ROWS>
__device__ __forceinline__ void enter(const Args& a, Cursor& c) {
  c.r = load_request(a, c.i);
  c.nrt = ((int64_t)c.r.q_len * a.group + ROWS - 1) / ROWS;
  c.nt = c.r.len > 0 ? (c.r.len + kTile - 1) / kTile : 1;
}

template <int ROWS>
__device__ __forceinline__ void advance(const Args& a, Cursor& c) {
  if (++c.t < c.nt) return;
  c.t = 0;
  if (++c.h < a.kv_heads) return;
  c.h = 0;
  if (++c.rt < c.nrt) return;
  c.rt = 0;
  c.nrt = 0;
  while (++c.i < a.batch) {
    enter<ROWS>(a, c);
    if (c.nrt > 0) break;
  }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Byte of a stage's codes that holds code `b` of token `t`, after the swizzle.
template <int D>
__device__ __forceinline__ uint32_t code_at(int t, int b) {
  const uint32_t off = (uint32_t)(t * D + b);
  return off ^ (((off >> 7) & 7u) << 4);
}

// What a piece of a row tile belongs to, in shared memory: request, row tile,
// kv head, and whether it begins or ends the tile's tokens.
struct Tag {
  int64_t rt;
  int i, h;
  int valid, starts, ends;
};
__device__ __forceinline__ bool same(const Tag& x, const Tag& y) { return x.i == y.i && x.rt == y.rt && x.h == y.h; }

// ints of a CTA's meta record: two tags of {valid, starts, ends, i, h, rt lo, rt hi}
constexpr int kTagInts = 8;
constexpr int kMetaInts = 2 * kTagInts;

template <bool F32>
__device__ __forceinline__ void store_out(const Args& a, int64_t at, float v) {
  if constexpr (F32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

// What turns a row's accumulated values into its output: 1 / l without the
// weights' shift, 0 for a row that sees nothing; NaN stays NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : kUnshift / l; }

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
attn_split_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ Args a) {
  using C = Cfg<D, NT>;
  constexpr int kWarps = C::kWarps, kRows = C::kRows, S = C::kStages;
  constexpr int KS = D / 16;                   // k steps of the scores, m tiles of the output
  constexpr int Q2 = F32 ? 2 : 1;              // fp16 terms of a query or weight
  extern __shared__ uint8_t attn_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tid = lane & 3;
  uint8_t* ring = smem + warp * S * C::kStageBytes;
  float* pieces = reinterpret_cast<float*>(smem + C::kRing);          // the warps' first pieces
  uint64_t* bars = reinterpret_cast<uint64_t*>(pieces + kWarps * C::kPiece) + warp * S;
  float* scales = reinterpret_cast<float*>(reinterpret_cast<uint64_t*>(pieces + kWarps * C::kPiece) + kWarps * S) +
                  warp * S * 4;
  __shared__ Tag tags[2 * kWarps];
  __shared__ long long wsum[kWarps];
  __shared__ int timeout;
  const int bs = 1 << a.log2_bs;

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init1(bars + s, 5);
    mbar_init_fence();
    tags[2 * warp].valid = tags[2 * warp + 1].valid = 0;
  }
  if (threadIdx.x == 0) timeout = 0;
  pdl_wait();
  pdl_launch();

  // rows that no request owns
  {
    const int64_t end = __ldg(a.cu_q + a.batch), cols = (int64_t)a.q_heads * D;
    for (int64_t t = (end < 0 ? 0 : end) + blockIdx.x; t < a.total_q; t += gridDim.x)
      for (int64_t c = threadIdx.x; c < cols; c += C::kThreads) store_out<F32>(a, t * a.ldo + c, 0.f);
  }

  // prefix sums of the requests' tiles (in the rings, which are still empty);
  // the list's length, and this warp's part of it
  long long* pre = reinterpret_cast<long long*>(smem);
  const int per = (a.batch + C::kThreads - 1) / C::kThreads;
  const int i0 = min(a.batch, (int)threadIdx.x * per), i1 = min(a.batch, i0 + per);
  auto tiles_of = [&](int i) {
    if (blockIdx.x == 0 && (int64_t)__ldg(a.kv_lens + i) > ((int64_t)a.width << a.log2_bs))
      raise_flag(a.status, LQ_DEV_RANGE);
    Cursor c;
    c.i = i;
    enter<kRows>(a, c);
    return (long long)c.nrt * a.kv_heads * c.nt;
  };
  long long sum = 0;
  for (int i = i0; i < i1; ++i) {
    const long long n = tiles_of(i);
    pre[i] = n;
    sum += n;
  }
  long long inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) inc += total;
    total += wsum[w];
  }
  long long run = inc - sum;
  for (int i = i0; i < i1; ++i) {
    const long long n = pre[i];
    pre[i] = run;
    run += n;
  }
  __syncthreads();
  // equal parts for the CTAs, then for their warps, the first ones a tile longer
  long long u0 = 0;
  int64_t n = total;
  auto part_of = [&](int parts, int i) {
    const long long base = n / parts, more = n % parts;
    u0 += base * i + (i < more ? i : more);
    n = base + (i < more ? 1 : 0);
  };
  part_of(gridDim.x, blockIdx.x);
  part_of(kWarps, warp);
  Cursor cc, ci;
  if (n > 0) {
    int lo = 0, hi = a.batch;                  // last request with pre[i] <= u0 (it has tiles: the next one starts later)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u0) lo = mid; else hi = mid;
    }
    cc.i = lo;
    enter<kRows>(a, cc);
    long long rem = u0 - pre[lo];
    cc.t = (int)(rem % cc.nt);
    rem /= cc.nt;
    cc.h = (int)(rem % a.kv_heads);
    cc.rt = rem / a.kv_heads;
  }
  // the prefix sums have been read: the rings may fill
  fence_proxy_async_smem();
  __syncthreads();

  if (n > 0) {
    ci = cc;
    // block of part e (lanes 0 and 1) of the tile at the issue cursor
    auto load_block = [&]() {
      int blk = -1;
      const int p = ci.t * kTile + (bs < kTile ? 16 * lane : 0);
      if (lane < 2 && p < ci.r.len) blk = __ldg(a.table + ci.i * a.ldt + (p >> a.log2_bs));
      return blk;
    };
    auto issue = [&](int s, int blk) {
      const int e = bs < kTile ? (lane >> 1) & 1 : 0;
      const int b = __shfl_sync(0xffffffffu, blk, e);
      const bool ok = b >= 0 && b < a.num_blocks;
      const uint32_t oks = __ballot_sync(0xffffffffu, ok);
      if (lane < 4) {
        const int64_t sc = (int64_t)b * a.kv_heads + ci.h;
        float* dst = scales + 4 * s + lane;    // k and v of part 0, of part 1
        if (ok) {
          cp_async4(smem_addr(dst), ((lane & 1) ? a.vs : a.ks) + sc);
          cp_async_arrive(bars + s);
        } else {
          *dst = -1.f;                         // its tokens are left out
          mbar_arrive(bars + s);
        }
      }
      if (lane == 0) {
        uint8_t* dst = ring + s * C::kStageBytes;
        if (bs < kTile) {
          const uint32_t part = 16 * D;
          const bool ok1 = (oks >> 2) & 1;
          mbar_expect_tx(bars + s, 2 * part * ((ok ? 1 : 0) + (ok1 ? 1 : 0)));
          if (ok) {
            const int row = (int)((((int64_t)b * a.kv_heads + ci.h) << a.log2_bs) * D >> 7);
            tma_load_2d(dst, &map_k, bars + s, 0, row);
            tma_load_2d(dst + kTile * D, &map_v, bars + s, 0, row);
          }
        } else {
          mbar_expect_tx(bars + s, ok ? C::kStageBytes : 0);
          if (ok) {
            const int off = (ci.t * kTile) & (bs - 1);
            const int row = (int)(((((int64_t)b * a.kv_heads + ci.h) << a.log2_bs) + off) * D >> 7);
            tma_load_2d(dst, &map_k, bars + s, 0, row);
            tma_load_2d(dst + kTile * D, &map_v, bars + s, 0, row);
          }
        }
      } else if (lane == 2 && bs < kTile && ok) {
        // the second half of a tile of two blocks; its bytes are in lane 0's count
        uint8_t* dst = ring + s * C::kStageBytes + 16 * D;
        const int row = (int)((((int64_t)b * a.kv_heads + ci.h) << a.log2_bs) * D >> 7);
        tma_load_2d(dst, &map_k, bars + s, 0, row);
        tma_load_2d(dst + kTile * D, &map_v, bars + s, 0, row);
      }
      // a block id outside the pool, or a length past the table
      const int p = ci.t * kTile + (bs < kTile ? 16 * e : 0);
      if (lane < 4 && !ok && p < ci.r.len) raise_flag(a.status, LQ_DEV_RANGE);
    };

    int blk = load_block();
    int64_t issued = 0;
    for (int s = 0; s < S && issued < n; ++s) {
      issue(s, blk);
      if (++issued < n) {
        advance<kRows>(a, ci);
        blk = load_block();
      }
    }

    uint32_t qf[NT][KS][2][Q2];
    float acc[KS][NT][4];
    float mx[NT][2], sum_l[NT][2], fac[NT][2];
    int lim[NT][2];                            // last position each of this thread's rows sees
    int lim_min = 0;
    bool fresh = true, first_seg = true;
    const bool begins = cc.t == 0;             // whether the first segment starts here
    bool seg_starts = begins;
    int s = 0;
    uint32_t ph = 0;
    bool dead = false;

    for (int64_t k = 0; k < n; ++k) {
      if (fresh) {
        fresh = false;
        // this segment's query rows: lane (g, tid) holds row g's dimensions
        // tid * D/4 ...; a power of two per row brings them into fp16's range
        const int64_t rows = (int64_t)cc.r.q_len * a.group;
        lim_min = INT_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int64_t R = cc.rt * kRows + nt * 8 + g;
          float v[D / 4];
          if (R < rows) {
            const int64_t at = (cc.r.q0 + R / a.group) * a.ldq + ((int64_t)cc.h * a.group + R % a.group) * D +
                               tid * (D / 4);
            if constexpr (F32) {
              const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at);
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                const float4 x = __ldg(p + c);
                v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
              }
            } else {
              const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) + at);
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                const uint4 x = __ldg(p + c);
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
#pragma unroll
          for (int c = 0; c < KS; ++c) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = v[4 * c + 2 * e] * up, y = v[4 * c + 2 * e + 1] * up;
              qf[nt][c][e][0] = pack_f16(x, y);
              if constexpr (F32) qf[nt][c][e][1] = rest_f16(qf[nt][c][e][0], x, y);
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            fac[nt][c] = __shfl_sync(0xffffffffu, down, 4 * (2 * tid + c));
            const int64_t Rc = cc.rt * kRows + nt * 8 + 2 * tid + c;
            lim[nt][c] = Rc < rows ? cc.r.shown + (int)(Rc / a.group) : INT_MAX;
            lim_min = min(lim_min, lim[nt][c]);
            mx[nt][c] = -INFINITY;
            sum_l[nt][c] = 0.f;
          }
        }
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));
        lim_min = min(lim_min, cc.r.len - 1);
#pragma unroll
        for (int c = 0; c < KS; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][nt][e] = 0.f;
      }

      if (!dead && !mbar_wait_bounded(bars + s, ph, kWaitCycles)) {
        dead = true;
        timeout = 1;
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const uint8_t* kst = ring + s * C::kStageBytes;
      const uint8_t* vst = kst + kTile * D;
      const float4 sc4 = *reinterpret_cast<const float4*>(scales + 4 * s);
      const float sk[2] = {sc4.x, sc4.z}, sv[2] = {sc4.y, sc4.w};

      // scores S^T [32 tokens x 8 NT rows]
      float sc[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const int b = tid * (D / 4) + 16 * j;
          const uint4 x = *reinterpret_cast<const uint4*>(kst + code_at<D>(16 * mt + g, b));
          const uint4 y = *reinterpret_cast<const uint4*>(kst + code_at<D>(16 * mt + g + 8, b));
          const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = xa[e] ^ 0x80808080u, v = ya[e] ^ 0x80808080u;
            const uint32_t a0 = codes_f16(u, 0x4140), a2 = codes_f16(u, 0x4342);
            const uint32_t a1 = codes_f16(v, 0x4140), a3 = codes_f16(v, 0x4342);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int f = 0; f < Q2; ++f)
                mma16816(sc[mt][nt], a0, a1, a2, a3, qf[nt][4 * j + e][0][f], qf[nt][4 * j + e][1][f]);
          }
        }
      }

      // exponents x, their running maximum, weights 2^(x - max + 14)
      const int p0 = cc.t * kTile;
      const bool masked = p0 + kTile - 1 > lim_min || sv[0] < 0.f || sv[1] < 0.f;
      float lv[2], iv[2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float v = fmaxf(sv[mt], kMinScale);
        const float vn = sv[mt] == sv[mt] ? v : sv[mt];          // NaN stays NaN
        lv[mt] = log2f(vn);
        iv[mt] = kUnshift / vn;
      }
      uint32_t pb[2][NT][2][Q2];
      float mnew[NT][2];
      bool grows = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float c0 = fac[nt][0] * sk[mt], c1 = fac[nt][1] * sk[mt];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = fmaf(sc[mt][nt][e], (e & 1) ? c1 : c0, lv[mt]);
            if (masked) {
              const int p = p0 + 16 * mt + g + (e & 2 ? 8 : 0);
              if (p > lim[nt][e & 1] || p >= cc.r.len || sv[mt] < 0.f) x = -INFINITY;
            }
            sc[mt][nt][e] = x;
            if (e & 1) m1 = fmaxf(m1, x);
            else m0 = fmaxf(m0, x);
          }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        mnew[nt][0] = fmaxf(mx[nt][0], m0);
        mnew[nt][1] = fmaxf(mx[nt][1], m1);
        grows |= mnew[nt][0] > mx[nt][0] || mnew[nt][1] > mx[nt][1];
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = mx[nt][c] == mnew[nt][c] ? 1.f : ex2(mx[nt][c] - mnew[nt][c]);
            mx[nt][c] = mnew[nt][c];
            sum_l[nt][c] *= f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              acc[j][nt][c] *= f;
              acc[j][nt][c + 2] *= f;
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float b0 = (mx[nt][0] == -INFINITY ? 0.f : mx[nt][0]) - kShift;
        const float b1 = (mx[nt][1] == -INFINITY ? 0.f : mx[nt][1]) - kShift;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(sc[mt][nt][e] - ((e & 1) ? b1 : b0));
          const float s0 = w[0] + w[2], s1 = w[1] + w[3];
          // a block the row does not see may have any scale: its sum is 0, not 0 * NaN
          sum_l[nt][0] = fmaf(s0, s0 > 0.f ? iv[mt] : 0.f, sum_l[nt][0]);
          sum_l[nt][1] = fmaf(s1, s1 > 0.f ? iv[mt] : 0.f, sum_l[nt][1]);
          const uint32_t x0 = pack_f16(w[0], w[1]), x1 = pack_f16(w[2], w[3]);
          pb[mt][nt][0][0] = transpose8(x0);
          pb[mt][nt][1][0] = transpose8(x1);
          if constexpr (F32) {
            pb[mt][nt][0][1] = transpose8(rest_f16(x0, w[0], w[1]));
            pb[mt][nt][1][1] = transpose8(rest_f16(x1, w[2], w[3]));
          }
        }
      }

      // O^T [D x 8 NT rows] += C_v^T w^T; lane g holds dimensions g * D/8 ...
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        constexpr int NW = D / 32;             // words of codes per token and lane
        uint32_t v[4][NW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * mt + 2 * tid + (r & 1) + (r & 2 ? 8 : 0);
          if constexpr (NW == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(vst + code_at<D>(t, g * (D / 8)));
            v[r][0] = x.x; v[r][1] = x.y;
          } else {
#pragma unroll
            for (int c = 0; c < NW / 4; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(vst + code_at<D>(t, g * (D / 8) + 16 * c));
              v[r][4 * c] = x.x; v[r][4 * c + 1] = x.y; v[r][4 * c + 2] = x.z; v[r][4 * c + 3] = x.w;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < NW; ++c) {
          const uint32_t p = v[0][c] ^ 0x80808080u, q = v[1][c] ^ 0x80808080u;
          const uint32_t r = v[2][c] ^ 0x80808080u, t = v[3][c] ^ 0x80808080u;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = __byte_perm(p, q, half ? 0x7362 : 0x5140);    // token pairs side by side
            const uint32_t y = __byte_perm(r, t, half ? 0x7362 : 0x5140);
            const uint32_t a0 = codes_f16(x, 0x4140), a1 = codes_f16(x, 0x4342);
            const uint32_t a2 = codes_f16(y, 0x4140), a3 = codes_f16(y, 0x4342);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int f = 0; f < Q2; ++f)
                mma16816(acc[2 * c + half][nt], a0, a1, a2, a3, pb[mt][nt][0][f], pb[mt][nt][1][f]);
          }
        }
      }
      __syncwarp();                            // every lane has read the stage
      if (issued < n) {
        issue(s, blk);
        if (++issued < n) {
          advance<kRows>(a, ci);
          blk = load_block();
        }
      }
      if (++s == S) { s = 0; ph ^= 1; }

      const bool ends = cc.t + 1 == cc.nt;
      if (ends || k + 1 == n) {
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
        if (ends && seg_starts) {
          // all of the rows' tokens: the outputs, D/8 dimensions per lane and row
          const int64_t rows = (int64_t)cc.r.q_len * a.group;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int64_t R = cc.rt * kRows + nt * 8 + 2 * tid + c;
              if (R < rows) {
                const int64_t at = (cc.r.q0 + R / a.group) * a.ldo + ((int64_t)cc.h * a.group + R % a.group) * D +
                                   g * (D / 8);
                const float inv = inverse(l[nt][c]);
                if constexpr (F32) {
                  float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at);
#pragma unroll
                  for (int j = 0; j < KS / 2; ++j)
                    p[j] = make_float4(acc[2 * j][nt][c] * inv, acc[2 * j][nt][c + 2] * inv,
                                       acc[2 * j + 1][nt][c] * inv, acc[2 * j + 1][nt][c + 2] * inv);
                } else {
                  uint32_t u[KS];
#pragma unroll
                  for (int j = 0; j < KS; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[j][nt][c] * inv, acc[j][nt][c + 2] * inv);
                    u[j] = *reinterpret_cast<const uint32_t*>(&h);
                  }
                  uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at);
#pragma unroll
                  for (int j = 0; j < KS / 4; ++j)
                    p[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                }
              }
            }
        } else {
          // a piece: the first one of the warp has a place of its own, the last
          // one takes the warp's ring, which is not filled again
          const int slot = first_seg ? 0 : 1;
          float* dst = slot == 0 ? pieces + warp * C::kPiece : reinterpret_cast<float*>(ring);
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
                dst[kRows * D + row] = mx[nt][c];
                dst[kRows * D + kRows + row] = l[nt][c];
              }
            }
          if (lane == 0) {
            Tag& t = tags[2 * warp + slot];
            t.rt = cc.rt; t.i = cc.i; t.h = cc.h;
            t.starts = seg_starts; t.ends = ends; t.valid = 1;
          }
        }
        fresh = true;
        first_seg = false;
        seg_starts = true;
      }
      if (k + 1 < n) advance<kRows>(a, cc);
    }
    if (dead) {
      // let the copies in flight land before the CTA ends
      for (int i = 0; i < S; ++i) mbar_wait_bounded(bars + i, ph ^ (i < s ? 1u : 0u), kWaitCycles / 8);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && timeout) raise_flag(a.status, LQ_DEV_TIMEOUT);

  // join the warps' pieces: runs of consecutive pieces of the same row tile
  int* meta = a.meta + (int64_t)blockIdx.x * kMetaInts;
  if (threadIdx.x < 2) meta[threadIdx.x * kTagInts] = 0;
  __syncthreads();
  int e = 0;
  while (e < 2 * kWarps) {
    if (!tags[e].valid) { ++e; continue; }
    const Tag head = tags[e];
    int f = e + 1, last = e;
    for (; f < 2 * kWarps; ++f) {
      if (!tags[f].valid) continue;
      if (!same(head, tags[f]) || tags[f].starts) break;
      last = f;
    }
    const bool ends = tags[last].ends;
    // a piece with its beginning and its end here is an output; one that lacks
    // its beginning is the CTA's first (slot 0), one that lacks its end its last
    const bool whole = head.starts && ends;
    const int slot = head.starts ? 1 : 0;
    const Request r = load_request(a, head.i);
    const int64_t rows = (int64_t)r.q_len * a.group;
    float* gp = a.part + ((int64_t)blockIdx.x * 2 + slot) * C::kPiece;
    for (int x = threadIdx.x; x < kRows * D / 4; x += C::kThreads) {
      const int row = x / (D / 4), c = x % (D / 4);
      float M = -INFINITY;
      for (int p = e; p <= last; ++p)
        if (tags[p].valid) {
          const float* src = (p & 1) ? reinterpret_cast<const float*>(smem + (p >> 1) * S * C::kStageBytes)
                                     : pieces + (p >> 1) * C::kPiece;
          M = fmaxf(M, src[kRows * D + row]);
        }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
      for (int p = e; p <= last; ++p)
        if (tags[p].valid) {
          const float* src = (p & 1) ? reinterpret_cast<const float*>(smem + (p >> 1) * S * C::kStageBytes)
                                     : pieces + (p >> 1) * C::kPiece;
          const float m = src[kRows * D + row];
          const float f1 = m == M ? 1.f : ex2(m - M);
          const float4 v = *reinterpret_cast<const float4*>(src + row * D + 4 * c);
          l = fmaf(src[kRows * D + kRows + row], f1, l);
          o.x = fmaf(v.x, f1, o.x); o.y = fmaf(v.y, f1, o.y);
          o.z = fmaf(v.z, f1, o.z); o.w = fmaf(v.w, f1, o.w);
        }
      if (whole) {
        const int64_t R = head.rt * kRows + row;
        if (R < rows) {
          const int64_t at = (r.q0 + R / a.group) * a.ldo + ((int64_t)head.h * a.group + R % a.group) * D + 4 * c;
          const float inv = inverse(l);
          store_out<F32>(a, at, o.x * inv);
          store_out<F32>(a, at + 1, o.y * inv);
          store_out<F32>(a, at + 2, o.z * inv);
          store_out<F32>(a, at + 3, o.w * inv);
        }
      } else {
        *reinterpret_cast<float4*>(gp + row * D + 4 * c) = o;
        if (c == 0) {
          gp[kRows * D + row] = M;
          gp[kRows * D + kRows + row] = l;
        }
      }
    }
    if (!whole && threadIdx.x == 0) {
      int* t = meta + slot * kTagInts;
      t[0] = 1; t[1] = head.starts; t[2] = ends; t[3] = head.i; t[4] = head.h;
      t[5] = (int)(head.rt & 0xffffffff); t[6] = (int)(head.rt >> 32);
    }
    e = f;
  }
}

// Row tiles whose tokens fall to several CTAs: block c merges the pieces that
// CTAs c, c + 1, ... hold of the row tile that begins in CTA c.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(256) attn_merge_kernel(const __grid_constant__ Args a, int ctas) {
  using C = Cfg<D, NT>;
  constexpr int kRows = C::kRows;
  pdl_wait();
  pdl_launch();
  const int* head = a.meta + (int64_t)blockIdx.x * kMetaInts + kTagInts;
  if (!head[0]) return;
  // the CTAs after this one that hold more of the same row tile
  int n = 1;
  while (blockIdx.x + n < ctas) {
    const int* t = a.meta + (int64_t)(blockIdx.x + n) * kMetaInts;
    if (!t[0]) break;
    ++n;
    if (t[2]) break;
  }
  const Request r = load_request(a, head[3]);
  const int h = head[4];
  const int64_t rt = (int64_t)(uint32_t)head[5] | (int64_t)head[6] << 32;
  const int64_t rows = (int64_t)r.q_len * a.group;
  const float* first = a.part + ((int64_t)blockIdx.x * 2 + 1) * C::kPiece;
  const float* next = first + C::kPiece;                 // slot 0 of the CTA after, then every second piece
  for (int x = threadIdx.x; x < kRows * D / 4; x += 256) {
    const int row = x / (D / 4), c = x % (D / 4);
    const int64_t R = rt * kRows + row;
    if (R >= rows) continue;
    float M = first[kRows * D + row];
    for (int p = 1; p < n; ++p) M = fmaxf(M, next[(int64_t)(p - 1) * 2 * C::kPiece + kRows * D + row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float* src = p == 0 ? first : next + (int64_t)(p - 1) * 2 * C::kPiece;
      const float m = src[kRows * D + row];
      const float f = m == M ? 1.f : ex2(m - M);
      const float4 v = *reinterpret_cast<const float4*>(src + row * D + 4 * c);
      l = fmaf(src[kRows * D + kRows + row], f, l);
      o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
    }
    const int64_t at = (r.q0 + R / a.group) * a.ldo + ((int64_t)h * a.group + R % a.group) * D + 4 * c;
    const float inv = inverse(l);
    store_out<F32>(a, at, o.x * inv);
    store_out<F32>(a, at + 1, o.y * inv);
    store_out<F32>(a, at + 2, o.z * inv);
    store_out<F32>(a, at + 3, o.w * inv);
  }
}

template <int D, int NT, bool F32>
lq_status launch_split(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, int sms, void* stream) {
  using C = Cfg<D, NT>;
  static_assert(C::kStages >= 2 && C::kSmem + 640 <= 227 * 1024, "shared memory");
  static_assert(C::kStages * C::kStageBytes >= C::kPiece * 4, "a warp's last piece fits its ring");
  static_assert(C::kRing >= LQ_MAX_REQUESTS * 8, "the prefix sums fit the rings");
  auto kern = attn_split_kernel<D, NT, F32>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
  if (e == cudaSuccess) {
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, attn_merge_kernel<D, NT, F32>, a, sms);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  return check_launch();
}

// Codes of a cache as rows of 128 bytes, copied in boxes of `rows` of them.
bool encode_cache(CUtensorMap* map, const void* codes, int64_t bytes, int rows) {
  TensorMapEncodeTiledFn fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count_or_default() {
  const int sms = device_sm_count();
  return sms > 0 ? sms : 152;
}

}  // namespace attn
}  // namespace lq

using namespace lq;

extern "C" size_t lq_attention_paged_workspace_size(int batch, int64_t total_q, int q_heads, int kv_heads,
                                                    int head_dim) {
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || kv_heads <= 0 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  // two pieces of up to 16 rows per CTA, and what they belong to
  const size_t ctas = (size_t)attn::sm_count_or_default();
  const size_t meta = (ctas * attn::kMetaInts * sizeof(int) + 255) & ~(size_t)255;
  return meta + ctas * 2 * 16 * (size_t)(head_dim + 2) * sizeof(float);
}

extern "C" lq_status lq_attention_paged(const void* q_dev, int64_t ldq, int dtype, int64_t total_q,
                                        const int32_t* cu_q_dev, const int32_t* kv_lens_dev, int batch,
                                        const int32_t* block_table_dev, int64_t table_stride, int table_width,
                                        const int8_t* k_cache_dev, const float* k_scales_dev,
                                        const int8_t* v_cache_dev, const float* v_scales_dev, int64_t num_blocks,
                                        int block_size, int q_heads, int kv_heads, int head_dim, float sm_scale,
                                        void* out_dev, int64_t ldo, void* workspace_dev, size_t workspace_bytes,
                                        int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_attention_paged");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  if (!serve::valid_block_size(block_size)) return LQ_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return LQ_ERR_UNSUPPORTED;
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || q_heads > 1024) return LQ_ERR_SHAPE;
  const int64_t esize = dtype == LQ_BF16 ? 2 : 4, cols = (int64_t)q_heads * head_dim;
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || total_q > INT32_MAX || num_blocks < 0 ||
      num_blocks > INT32_MAX || table_width < 0 || table_stride < table_width || ldq < cols || ldo < cols ||
      (ldq * esize) % 16 != 0 || (ldo * esize) % 16 != 0)
    return LQ_ERR_SHAPE;
  // rows of 128 bytes of codes are counted in 32 bits (a pool of 256 GB for K alone)
  const int64_t block_rows = (int64_t)kv_heads * block_size * head_dim / 128;
  if (num_blocks > INT32_MAX / block_rows) return LQ_ERR_SHAPE;
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
                         !aligned4(k_scales_dev) || !aligned4(v_scales_dev)))
    return LQ_ERR_ARG;
  if (workspace_bytes < lq_attention_paged_workspace_size(batch, total_q, q_heads, kv_heads, head_dim))
    return LQ_ERR_SHAPE;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  attn::Args a;
  a.q = q_dev; a.ldq = ldq; a.total_q = total_q; a.cu_q = cu_q_dev; a.kv_lens = kv_lens_dev; a.batch = batch;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width;
  a.ks = k_scales_dev; a.vs = v_scales_dev; a.num_blocks = num_blocks;
  a.log2_bs = serve::log2_of(block_size); a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads;
  a.scale_log2 = sm_scale * 1.4426950408889634f; a.out = out_dev; a.ldo = ldo; a.status = dev_status_dev;
  a.meta = reinterpret_cast<int*>(workspace_dev);
  const size_t meta = ((size_t)sms * attn::kMetaInts * sizeof(int) + 255) & ~(size_t)255;
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace_dev) + meta);
  CUtensorMap mk, mv;
  // a pool without blocks: no copy is issued, any valid map will do
  const void* kc = num_blocks > 0 ? (const void*)k_cache_dev : workspace_dev;
  const void* vc = num_blocks > 0 ? (const void*)v_cache_dev : workspace_dev;
  const int64_t bytes = num_blocks > 0 ? num_blocks * block_rows * 128 : 4096;
  const int box = (block_size < attn::kTile ? block_size : attn::kTile) * head_dim / 128;
  if (!attn::encode_cache(&mk, kc, bytes, box) || !attn::encode_cache(&mv, vc, bytes, box)) return LQ_ERR_CUDA;
  // eight query rows per pass over the codes, sixteen where the average request has more
  const bool few = ((total_q + batch - 1) / batch) * a.group <= 8;
  if (dtype == LQ_F32) {
    if (head_dim == 64) return attn::launch_split<64, 1, true>(a, mk, mv, sms, stream);
    if (head_dim == 128) return attn::launch_split<128, 1, true>(a, mk, mv, sms, stream);
    return attn::launch_split<256, 1, true>(a, mk, mv, sms, stream);
  }
  if (head_dim == 256) return attn::launch_split<256, 1, false>(a, mk, mv, sms, stream);
  if (head_dim == 64) return few ? attn::launch_split<64, 1, false>(a, mk, mv, sms, stream)
                                 : attn::launch_split<64, 2, false>(a, mk, mv, sms, stream);
  return few ? attn::launch_split<128, 1, false>(a, mk, mv, sms, stream)
             : attn::launch_split<128, 2, false>(a, mk, mv, sms, stream);
}
