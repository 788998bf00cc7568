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
// both sums, codes enter the matrix products as they are, and a large value
// scale cannot push a weight out of fp16's range (the running maximum is that
// of x, not of the score).  Scales too far apart for one exponent to serve both
// sums are looked after separately (the tcgen05 kernel in place, this one by
// rows_apart).  Running maxima are whole numbers: moving one shifts exponents and
// rounds nothing, so how the positions were split shows in fp32 roundings, and
// in an fp16 weight only where it lies that near to the middle of two.
//
// The split kernel, for few query rows per kv head (decode steps, drafted
// tokens), is bound by reading the codes from HBM: every code is used for at
// most 16 rows.  The batch's work is a list of 32-token tiles (request, tile of
// rows, kv head, tokens), and every warp of one CTA per SM takes an equal,
// contiguous part of it, whatever the lengths are: no request waits for
// another's long tail.  A warp streams its tiles through its own ring of half
// tiles (K, V, K, V, ...) by TMA (the codes' rows of 128 bytes in the 128-byte
// swizzle, so that the fragment loads below meet no bank twice) with no
// barrier shared between warps, keeps running maxima, sums and the output tile
// in registers, and writes an output when it has seen all of a row's tiles.
// Pieces of rows are joined by the CTA and by the merge kernel between CTAs, in
// the order of the tiles, so that equal calls give equal bits.  Sixteen warps
// per SM, with half a tile's compute between refills, keep about 128 KB of
// loads in flight and enough warps to issue from while others wait.
//
// Products on mma.sync m16n8k16 with the codes as the 16-row operand (fp16,
// exact) and eight query rows as the other: scores S^T = C_k q^T, then
// O^T += C_v^T w^T with the weights transposed in registers.  tcgen05 needs 64
// or 128 rows to earn its operand traffic through shared memory; at 8 or 16
// rows it would still be the codes' bytes that bound the kernel.  bf16 queries
// are exact in fp16 after a power-of-two factor per row; fp32 queries and
// weights are split into two fp16 terms (22 bits).  The running maximum is let
// fall behind by up to 2^7 (weights are held times 2^8, so 2^15 is in range
// and 2^-22 of the largest still a normal number): most tiles then only compare
// with it and need no exchange between lanes.
#include "lq_attn_paged.cuh"

namespace lq {
namespace attn {

constexpr int kTile = 32;                      // tokens per tile

template <int D, int NT, bool F32>
struct Cfg {
  // 16 warps of at most 128 registers where the output tile and the queries
  // leave room, else 8 of at most 255
  static constexpr int kWarps = D * NT * (F32 ? 2 : 1) <= 128 ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalfBytes = kTile * D;             // the K or the V codes of a tile
  static constexpr int kPiece = kRows * (D + 3);           // floats: output rows, maxima, sums, their units
  static constexpr int kPerHalf = kHalfBytes + 32;         // codes, barrier, scales, what tile it is
  static constexpr int kEnds = 2 * kWarps;                 // pieces that the warps may leave
  static constexpr int kRowBytes = 5 * kEnds * kRows * 4;                // the pieces' rows
  static constexpr int kFit = (227 * 1024 - 1024 - 2048 - kRowBytes) / (kWarps * kPerHalf);
  static constexpr int kHalves = kFit < 8 ? kFit : 8;      // of a warp's ring
  static constexpr int kRing = kWarps * kHalves * kHalfBytes;
  static constexpr int kSmem = kWarps * kHalves * kPerHalf + kRowBytes + 1024;
};

// A place in the list of tiles.
struct Cursor {
  int i;             // request
  int rt, nrt;       // tile of rows, and how many the request has
  int h;             // kv head
  int t, nt;         // tile of tokens, and how many the request has
  int len;
};

template <int ROWS>
__device__ __forceinline__ void enter(const Args& a, Cursor& c) {
  const Request r = load_request(a, c.i);
  c.len = r.len;
  c.nrt = (r.q_len * a.group + ROWS - 1) / ROWS;
  c.nt = r.len > 0 ? (r.len + kTile - 1) / kTile : 1;
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
#pragma unroll 1
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

__device__ __forceinline__ bool same(const Tag& x, const Tag& y) { return x.i == y.i && x.rt == y.rt && x.h == y.h; }

// Where a row of a row tile lies in q or out, in elements; false past the last row.
__device__ __forceinline__ bool row_at(const Args& a, int q0, int q_len, int R, int h, int64_t ld, int dim,
                                       int64_t* at) {
  const int j = R / a.group;
  *at = (int64_t)(q0 + j) * ld + (h * a.group + R - j * a.group) * dim;
  return j < q_len;
}

template <bool F32>
__device__ __forceinline__ void store_out(const Args& a, int64_t at, float v) {
  if constexpr (F32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

template <bool F32>
__device__ __forceinline__ void store_out4(const Args& a, int64_t at, const float4& o, float inv, float unit) {
  if constexpr (F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) =
        make_float4(o.x * inv * unit, o.y * inv * unit, o.z * inv * unit, o.w * inv * unit);
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv * unit, o.y * inv * unit);
    const __nv_bfloat162 y = __floats2bfloat162_rn(o.z * inv * unit, o.w * inv * unit);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}

// What turns a row's accumulated values into its output, with its unit_of: 1 / l,
// or 0 for a row that sees nothing; NaN stays NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// The loop below puts the value scale into the weights.  With scales that differ
// by up to 2^60 (zeros count as 2^-60) every weight that matters in the sum of
// weights is a normal number: x more than 134 below the maximum is a score more
// than 43 below the largest.  What meets any other scale, or zeros that were a
// row's maximum, is done again by rows_apart where there are such scales beside
// others.
constexpr float kScaleBits = 30.f;
constexpr float kLeastScale = 9.31322575e-10f, kMostScale = 1073741824.f;       // 2^-30, 2^30
constexpr float kZeroScale = 8.67361738e-19f;                                   // 2^-60
// Sums of weight / value scale are held times 2^-20: at most 2^55 for a weight.
constexpr float kSumUnit = 9.5367431640625e-7f, kSumUnitBits = 20.f;
__device__ __forceinline__ bool far_scale(float v) { return v > kMostScale || (v < kLeastScale && v > 0.f); }

// Whether tokens [p0, p1) of a request and kv head have value scales that the loop
// does not serve: one out of its range, or zeros beside others.
__device__ __noinline__ bool scales_apart(const Args& a, int req, int h, int p0, int p1) {
  bool far = false, zeros = false, values = false;
  for (int p = (p0 >> a.log2_bs) + (threadIdx.x & 31); p << a.log2_bs < p1; p += 32) {
    const int blk = a.table[req * a.ldt + p];
    if ((unsigned)blk < (unsigned long long)a.num_blocks) {
      const float v = a.vs[(int64_t)blk * a.kv_heads + h];
      far |= far_scale(v);
      zeros |= v == 0.f;
      values |= v >= kLeastScale;
    }
  }
  return __any_sync(0xffffffffu, far) ||
         (__any_sync(0xffffffffu, zeros) && __any_sync(0xffffffffu, values));
}

// Query rows row0 .. row0 + rows - 1 of a request and kv head over the tokens
// [p0, p1), for value scales of any size: one row after the other, 32 tokens at a
// time in fp32, with the two exponents of every row apart.  The outputs where dst is
// null, else the values' sums to dst and maxima, sums and units to the rows' lists.
template <int D, bool F32>
__device__ __noinline__ void rows_apart(const Args& a, int req, int row0, int rows, int h, int p0, int p1, float* dst,
                                        float* rows_m, float* rows_l, float* rows_u) {
  constexpr int E = D / 32;                    // dimensions per lane
  const int lane = threadIdx.x & 31, bs1 = (1 << a.log2_bs) - 1;
  const Request r = load_request(a, req);
  const int32_t* table = a.table + req * a.ldt;
#pragma unroll 1
  for (int row = 0; row < rows; ++row) {
    int64_t at_q, at_out;
    const bool here = row_at(a, r.q0, r.q_len, row0 + row, h, a.ldq, D, &at_q);
    row_at(a, r.q0, r.q_len, row0 + row, h, a.ldo, D, &at_out);
    const int past = here ? min(min(r.shown + (row0 + row) / a.group, r.len - 1) + 1, p1) : p0;
    float mx = -INFINITY, un = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
    for (int t0 = p0; t0 < past; t0 += 32) {
      const int p = t0 + lane, blk = p < past ? table[p >> a.log2_bs] : -1;
      const bool ok = (unsigned)blk < (unsigned long long)a.num_blocks;
      const int64_t head = (int64_t)blk * a.kv_heads + h, line = ((head << a.log2_bs) + (p & bs1)) * D;
      float s = -INFINITY, x = -INFINITY;
      if (ok) {
        float sum = 0.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          const uint4 k = *reinterpret_cast<const uint4*>(a.kc + line + c);
          const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float q;
            if constexpr (F32) q = reinterpret_cast<const float*>(a.q)[at_q + c + e];
            else q = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.q)[at_q + c + e] << 16);
            sum = fmaf(q * a.scale_log2, (float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), sum);
          }
        }
        s = sum * a.ks[head];
        x = s + log2_scale(a.vs[head]);
      }
      float most = s, top = x;
#pragma unroll
      for (int i = 16; i; i >>= 1) {
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, i));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      }
      const float un_to = fmaxf(un, ceilf(most)), mx_to = fmaxf(mx, ceilf(top)), f = pow2(mx - mx_to);
      float w = ok ? ex2(s - un_to) : 0.f;
      const float v = ok && x != -INFINITY ? ex2(x - mx_to + kShift) : 0.f;
#pragma unroll
      for (int i = 16; i; i >>= 1) w += __shfl_xor_sync(0xffffffffu, w, i);
      l = fmaf(l, pow2(un - un_to), w);        // (NaN before any score: 0 of 0)
      un = un_to;
      mx = mx_to;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      const uint32_t there = __ballot_sync(0xffffffffu, ok);
#pragma unroll 4
      for (int t = 0; t < 32; ++t) {
        const int64_t from = __shfl_sync(0xffffffffu, line, t);
        const float vt = __shfl_sync(0xffffffffu, v, t);
        if (there >> t & 1)
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(vt, (float)a.vc[from + lane * E + e], o[e]);
      }
    }
    if (dst != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) dst[row * D + lane * E + e] = o[e];
      if (lane == 0) {
        rows_m[row] = mx;
        rows_l[row] = l;
        rows_u[row] = un;
      }
    } else if (here) {
      const float inv = inverse(l), unit = unit_of(mx, un);
#pragma unroll
      for (int e = 0; e < E; ++e) store_out<F32>(a, at_out + lane * E + e, o[e] * inv * unit);
    }
  }
  __syncwarp();
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(Cfg<D, NT, F32>::kThreads, 1)
attn_split_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ Args a) {
  using C = Cfg<D, NT, F32>;
  constexpr int kWarps = C::kWarps, kRows = C::kRows, S = C::kHalves;
  constexpr int KS = D / 16;                   // k steps of the scores, m tiles of the output
  constexpr int Q2 = F32 ? 2 : 1;              // fp16 terms of a query or weight
  extern __shared__ uint8_t attn_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tid = lane & 3;
  uint8_t* ring = smem + warp * S * C::kHalfBytes;
  int4* infos = reinterpret_cast<int4*>(smem + C::kRing) + warp * S;               // which tile a K half is of
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing + kWarps * S * 16) + warp * S;
  float2* scales = reinterpret_cast<float2*>(smem + C::kRing + kWarps * S * 24) + warp * S;
  // maxima, sums and units of the warps' pieces, and their weights when they are joined
  float* piece_m = reinterpret_cast<float*>(smem + kWarps * S * C::kPerHalf);
  float* piece_l = piece_m + C::kEnds * kRows;
  float* piece_u = piece_l + C::kEnds * kRows;
  float* piece_f = piece_u + C::kEnds * kRows;
  float* piece_w = piece_f + C::kEnds * kRows;
  __shared__ Tag tags[2 * kWarps];
  __shared__ int order[2 * kWarps];            // the pieces that are there, in order
  __shared__ long long wsum[kWarps];
  __shared__ int again[kWarps];                // value scales far apart, or zeros that were a maximum
  __shared__ int4 part_at[kWarps];             // the first tile of the warp's part
  __shared__ int2 asked[kWarps];               // the warp's current request: first query token, how many
  __shared__ int timeout, q_end;
  const bool paired = a.log2_bs < 5;           // a tile spans two blocks of 16
  // where the warps' first pieces go when more follow; a last one takes the
  // warp's ring, which is not filled again
  float* firsts = a.part + ((int64_t)gridDim.x * 2 + (int64_t)blockIdx.x * kWarps) * C::kPiece;

  if (lane == 0) {
#pragma unroll 1
    for (int s = 0; s < S; ++s) mbar_init1(bars + s, 3);
    mbar_init_fence();
    tags[2 * warp].valid = tags[2 * warp + 1].valid = 0;
    again[warp] = 0;
  }
  pdl_wait();
  pdl_launch();
  if (threadIdx.x == 0) {
    timeout = 0;
    q_end = a.cu_q[a.batch];
  }

  // prefix sums of the requests' tiles, the list's length, and this warp's part
  // of it: u0 and part_n
  auto tiles_of = [&](int i) {
    if (blockIdx.x == 0 && (int64_t)a.kv_lens[i] > ((int64_t)a.width << a.log2_bs))
      raise_flag(a.status, LQ_DEV_RANGE);
    Cursor c;
    c.i = i;
    enter<kRows>(a, c);
    return (long long)c.nrt * a.kv_heads * c.nt;
  };
  auto scan = [&](long long x) {               // inclusive, over the warp
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  long long u0 = 0, part_n = 0, before = 0;
  auto part_of = [&](unsigned parts, unsigned i) {
    const long long base = part_n < INT_MAX ? (unsigned)part_n / parts : part_n / parts;
    const unsigned more = (unsigned)(part_n - base * parts);
    u0 += base * i + min(i, more);
    part_n = base + (i < more ? 1 : 0);
  };
  // equal parts for the CTAs, then for their warps, the first ones a tile longer
  auto parts = [&](long long total) {
    part_n = total;
    part_of(gridDim.x, blockIdx.x);
    part_of(kWarps, warp);
  };
  Cursor ci;                                   // the tile whose halves are fetched next
  if (a.batch <= 32) {
    // every warp for itself, a request per lane
    const long long mine = lane < a.batch ? tiles_of(lane) : 0, inc = scan(mine);
    parts(__shfl_sync(0xffffffffu, inc, 31));
    const uint32_t here = __ballot_sync(0xffffffffu, lane < a.batch && inc - mine <= u0);
    ci.i = 31 - __clz(here);                   // last request that starts at or before u0: it has tiles
    before = __shfl_sync(0xffffffffu, inc - mine, ci.i);
    __syncwarp();                              // the barriers are there
  } else {
    // a run of requests per thread (in the rings, which are still empty)
    long long* pre = reinterpret_cast<long long*>(smem);
    const int per = (a.batch + C::kThreads - 1) / C::kThreads;
    const int i0 = min(a.batch, (int)threadIdx.x * per), i1 = min(a.batch, i0 + per);
    long long sum = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const long long n = tiles_of(i);
      pre[i] = n;
      sum += n;
    }
    long long inc = scan(sum);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    long long total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) inc += total;
      total += wsum[w];
    }
    long long run = inc - sum;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const long long n = pre[i];
      pre[i] = run;
      run += n;
    }
    __syncthreads();
    parts(total);
    int lo = 0, hi = a.batch;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u0) lo = mid; else hi = mid;
    }
    ci.i = lo;
    before = pre[lo];
    // the prefix sums have been read: the rings may fill
    fence_proxy_async_smem();
    __syncthreads();
  }
  const int n = (int)(part_n < (1 << 29) ? part_n : (1 << 29));
  if (n > 0) {
    enter<kRows>(a, ci);
    const long long rem = u0 - before;
    const long long hr = rem < INT_MAX ? (unsigned)rem / (unsigned)ci.nt : rem / ci.nt;    // row tile and head
    ci.t = (int)(rem - hr * ci.nt);
    ci.rt = (int)(hr < INT_MAX ? (unsigned)hr / (unsigned)a.kv_heads : hr / a.kv_heads);
    ci.h = (int)(hr - (long long)ci.rt * a.kv_heads);
  }

  if (n > 0) {
    // lanes 0 and 1: the block of half a tile each (the same block where it
    // holds the whole tile), and its place in the scales
    int blk = -1, at_scale = 0;
    bool blk_ok = false;
    auto load_block = [&]() {
      const int p = ci.t * kTile + (paired ? 16 * lane : 0);
      blk = -1;
      if (lane < 2 && p < ci.len) blk = a.table[ci.i * a.ldt + (p >> a.log2_bs)];
    };
    auto info_of = [](const Cursor& c) {
      return make_int4(c.i, c.rt, c.h | (c.t + 1 == c.nt ? 1 << 16 : 0), c.t);
    };
    const int rows_per_block = (D << a.log2_bs) >> 7;
    int qi = 0;                                // halves issued
    auto issue = [&](int s) {
      const bool is_v = qi & 1;
      if (!is_v) {
        blk_ok = (unsigned)blk < (unsigned long long)a.num_blocks;
        at_scale = blk * a.kv_heads + ci.h;
        if (lane < 2 && !blk_ok && ci.t * kTile + (paired ? 16 * lane : 0) < ci.len)
          raise_flag(a.status, LQ_DEV_RANGE);  // a block id outside the pool
        if (lane == 0) infos[s] = info_of(ci);
      }
      const bool ok0 = __shfl_sync(0xffffffffu, blk_ok, 0), ok1 = __shfl_sync(0xffffffffu, blk_ok, 1);
      if (lane < 2) {
        float* dst = reinterpret_cast<float*>(scales + s) + lane;
        if (blk_ok) {
          cp_async4(smem_addr(dst), (is_v ? a.vs : a.ks) + at_scale);
          cp_async_arrive(bars + s);
        } else {
          *dst = -1.f;                         // its tokens are left out
          mbar_arrive(bars + s);
        }
        if (lane == 0)
          mbar_expect_tx(bars + s, paired ? 16 * D * ((ok0 ? 1 : 0) + (ok1 ? 1 : 0)) : (ok0 ? C::kHalfBytes : 0));
        if (blk_ok && (paired || lane == 0)) {
          const int off = paired ? 0 : (ci.t * kTile) & ((1 << a.log2_bs) - 1);
          tma_load_2d(ring + s * C::kHalfBytes + (paired ? lane * 16 * D : 0), is_v ? &map_v : &map_k, bars + s, 0,
                      at_scale * rows_per_block + ((off * D) >> 7));
        }
      }
      if (++qi < 2 * n && is_v) {
        advance<kRows>(a, ci);
        load_block();
      }
    };

    load_block();
    if (lane == 0) part_at[warp] = make_int4(ci.i, ci.rt, ci.h, ci.t);

    uint32_t qf[NT][KS][2][Q2];
    float acc[KS][NT][4];
    float mx[NT][2], sum_l[NT][2], fac[NT][2];
    int lim[NT][2];                            // last position each of this thread's rows sees
    int lim_min = 0;
    bool fresh = true, seg_starts = false, more_before = false, dead = false;
    float sc[2][NT][4];                        // the tile's scores, then exponents
    float2 sk2;
    int4 info;
    int s = 0;
    uint32_t ph = 1;

    // half tiles one after the other, K and V in turn; the first S steps only
    // fill the ring, so that fetching stands in the code once
#pragma unroll 1
    for (int step = -S; step < 2 * n; ++step) {
      const bool skip = step < 0;
      if (step == -S || (!skip && !(step & 1))) {
        // (the first segment's rows are fetched beside its first block id)
        info = skip ? info_of(ci) : infos[s];  // written when the half was issued
        if (fresh) {
          fresh = false;
          const int h = info.z & 0xFFFF;
          seg_starts = info.w == 0;
          // this segment's query rows: lane (g, tid) holds row g's dimensions
          // tid * D/4 ...; a power of two per row brings them into fp16's range
          const Request r = load_request(a, info.x);
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
      const bool ends = info.z >> 16;
      if (!skip && !(step & 1)) {
        // scores S^T [32 tokens x 8 NT rows]
        const uint8_t* kst = ring + s * C::kHalfBytes;
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
        sk2 = scales[s];
      } else if (!skip) {
        const float2 sv2 = scales[s];
        const int p0 = info.w * kTile;
        const uint8_t* vst = ring + s * C::kHalfBytes;

        // exponents x less the running maximum, plus the shift
        const float sk[2] = {sk2.x, sk2.y}, sv[2] = {sv2.x, sv2.y};
        float lv[2], iv[2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float v = sv[mt] < kLeastScale ? kZeroScale : sv[mt];   // NaN stays NaN
          lv[mt] = lg2(v);
          iv[mt] = rcp(v) * kSumUnit;
        }
        if (fmaxf(fabsf(lv[0]), fabsf(lv[1])) > kScaleBits)         // seldom
          if (far_scale(sv[0]) || far_scale(sv[1])) again[warp] = 1;
        float lead = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float b0 = kShift - (mx[nt][0] == -INFINITY ? 0.f : mx[nt][0]);
          const float b1 = kShift - (mx[nt][1] == -INFINITY ? 0.f : mx[nt][1]);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float c0 = fac[nt][0] * sk[mt], c1 = fac[nt][1] * sk[mt];
            const float d0 = lv[mt] + b0, d1 = lv[mt] + b1;
            sc[mt][nt][0] = fmaf(sc[mt][nt][0], c0, d0);
            sc[mt][nt][1] = fmaf(sc[mt][nt][1], c1, d1);
            sc[mt][nt][2] = fmaf(sc[mt][nt][2], c0, d0);
            sc[mt][nt][3] = fmaf(sc[mt][nt][3], c1, d1);
          }
        }
        if (p0 + kTile - 1 > lim_min || sv[0] < 0.f || sv[1] < 0.f) {
          // tokens that some row does not see, or of a block that is not there
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (p0 + 16 * mt + g + (e & 2 ? 8 : 0) > lim[nt][e & 1] || sv[mt] < 0.f) sc[mt][nt][e] = -INFINITY;
        }
        bool empty = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          empty |= mx[nt][0] == -INFINITY || mx[nt][1] == -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
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
            for (int mt = 0; mt < 2; ++mt) {
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
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)             // moved by a token of a block of zeros?
                if (sv[mt] == 0.f && (none || d > 0.f) && d > -INFINITY &&
                    fmaxf(sc[mt][nt][c], sc[mt][nt][c + 2]) == (c ? m1 : m0))
                  again[warp] = 1;
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
              for (int mt = 0; mt < 2; ++mt) {
                sc[mt][nt][c] -= d;
                sc[mt][nt][c + 2] -= d;
              }
            }
          }
        }
        // weights and their sums; the weights transposed, as fp16
        uint32_t pb[2][NT][2][Q2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(sc[mt][nt][e]);
            const float s0 = w[0] + w[2], s1 = w[1] + w[3];
            // a block the row does not see may have any scale: its sum is 0, not 0 * NaN
            sum_l[nt][0] = fmaf(s0, s0 > 0.f ? iv[mt] : 0.f, sum_l[nt][0]);
            sum_l[nt][1] = fmaf(s1, s1 > 0.f ? iv[mt] : 0.f, sum_l[nt][1]);
            if (sv[mt] < kLeastScale) w[0] = w[1] = w[2] = w[3] = 0.f;
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
              for (int nt = 0; nt < NT; ++nt) {
                float (&o)[4] = acc[2 * c + half][nt];
                if constexpr (F32) {
                  // the matrix unit truncates its sums: over thousands of
                  // positions that would be a bias, so they are added here
                  float d[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(d, a0, a1, a2, a3, pb[mt][nt][0][1], pb[mt][nt][1][1]);
                  mma16816(d, a0, a1, a2, a3, pb[mt][nt][0][0], pb[mt][nt][1][0]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] += d[e];
                } else {
                  mma16816(o, a0, a1, a2, a3, pb[mt][nt][0][0], pb[mt][nt][1][0]);
                }
              }
            }
          }
        }
      }
      __syncwarp();                            // every lane has read the half: refill it
      if (qi < 2 * n) issue(s);
      if (++s == S) { s = 0; ph ^= 1; }

      if ((ends || step + 1 == 2 * n) && !skip && (step & 1)) {
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
                const float inv = inverse(l[nt][c]) * kSumUnit;
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
          float* dst = step + 1 == 2 * n ? reinterpret_cast<float*>(ring) : firsts + warp * C::kPiece;
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
                // the sum as a number from 1 to 2 and its unit
                const float e = (float)((int)(__float_as_uint(l[nt][c]) >> 23 & 255u) - 127);
                const int at = (2 * warp + slot) * kRows + row;
                piece_m[at] = mx[nt][c];
                piece_l[at] = l[nt][c] * pow2(-e);
                piece_u[at] = l[nt][c] == 0.f ? -INFINITY : mx[nt][c] - kShift + kSumUnitBits + e;
              }
            }
          if (lane == 0) {
            Tag& t = tags[2 * warp + slot];
            t.i = info.x; t.rt = info.y; t.h = h; t.q0 = asked[warp].x; t.q_len = asked[warp].y;
            t.starts = seg_starts; t.ends = ends; t.valid = step + 1 == 2 * n ? 1 : 2;
          }
        }
        fresh = true;
        more_before = true;
      }
    }
    __syncwarp();
    if (again[warp] && !dead) {
      // value scales far apart in the part, perhaps: the pieces of which that is so, again
      const int4 at = part_at[warp];
      Cursor c;
      c.i = at.x;
      enter<kRows>(a, c);
      c.rt = at.y; c.h = at.z; c.t = at.w;
      int slot = 0;
#pragma unroll 1
      for (int left = n; left > 0;) {
        const int tiles = min(left, c.nt - c.t), rows = (2 * warp + slot) * kRows;
        const bool whole = c.t == 0 && tiles == c.nt;
        left -= tiles;
        if (scales_apart(a, c.i, c.h, c.t * kTile, min((c.t + tiles) * kTile, c.len)))
          rows_apart<D, F32>(a, c.i, c.rt * kRows, kRows, c.h, c.t * kTile, (c.t + tiles) * kTile,
                             whole ? nullptr : left == 0 ? reinterpret_cast<float*>(ring) : firsts + warp * C::kPiece,
                             piece_m + rows, piece_l + rows, piece_u + rows);
        c.t += tiles - 1;
        advance<kRows>(a, c);
        slot = 1;
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

  // rows that no request owns
  {
    const int64_t cols = (int64_t)a.q_heads * D;
#pragma unroll 1
    for (int64_t t = (int64_t)max(q_end, 0) + blockIdx.x; t < a.total_q; t += gridDim.x)
#pragma unroll 1
      for (int64_t c = threadIdx.x; c < cols; c += C::kThreads) store_out<F32>(a, t * a.ldo + c, 0.f);
  }

  // join the warps' pieces.  A run is the pieces of one row tile, which follow
  // each other; lane e of every warp looks at piece e
  const Tag mine = tags[lane < C::kEnds ? lane : 0];
  const bool valid = lane < C::kEnds && mine.valid;
  const uint32_t here = __ballot_sync(0xffffffffu, valid);
  const uint32_t below = here & ((1u << lane) - 1);
  const bool leads = valid && (below == 0 || mine.starts || !same(tags[31 - __clz(below)], mine));
  const uint32_t lead_mask = __ballot_sync(0xffffffffu, leads);
  // the same by number among the pieces that are there
  const int rank = __popc(below), pieces = __popc(here), runs = __popc(lead_mask);
  uint32_t leaders = __reduce_or_sync(0xffffffffu, leads ? 1u << rank : 0u);
  if (warp == 0 && valid) order[rank] = lane;
  __syncthreads();
  auto run_begin = [&](int k) { return 31 - __clz(leaders & ((2u << k) - 1)); };      // of piece k's run
  auto run_end = [&](int k) {
    const uint32_t after = leaders & ~((2u << k) - 1);
    return after ? __ffs(after) - 1 : pieces;
  };
  // each piece's weight against the run's maximum, its sum in the run's unit
  for (int x = threadIdx.x; x < pieces * kRows; x += C::kThreads) {
    const int k = x / kRows, row = x % kRows, end = run_end(k);
    float M = -INFINITY, U = -INFINITY;
#pragma unroll 4
    for (int p = run_begin(k); p < end; ++p) {
      M = fmaxf(M, piece_m[order[p] * kRows + row]);
      U = fmaxf(U, piece_u[order[p] * kRows + row]);
    }
    const int own = order[k] * kRows + row;
    piece_f[x] = piece_m[own] == M ? 1.f : ex2(piece_m[own] - M);
    piece_w[x] = piece_l[own] * (piece_u[own] == U ? 1.f : ex2(piece_u[own] - U));
  }
  if (threadIdx.x < 2) {
    // slot 0: a run without its beginning, the CTA's first; slot 1: one without its end, its last
    Tag t = tags[0];
    t.valid = 0;
    if (pieces) {
      const int last = pieces - 1, k = threadIdx.x == 0 ? 0 : run_begin(last);
      t = tags[order[k]];
      t.ends = tags[order[run_end(k) - 1]].ends;
      t.valid = threadIdx.x == 0 ? !t.starts : t.starts && !t.ends;
    }
    a.meta[2 * blockIdx.x + threadIdx.x] = t;
  }
  __syncthreads();
  constexpr int kItems = kRows * D / 4;
  for (int x = threadIdx.x; x < runs * kItems; x += C::kThreads) {
    int k0 = 0;                                // the run's first piece
    {
      uint32_t m = leaders;
      for (int r = x / kItems; r > 0; --r) m &= m - 1;
      k0 = __ffs(m) - 1;
    }
    const int row = x % kItems / (D / 4), c = x % (D / 4), end = run_end(k0);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, M = -INFINITY, U = -INFINITY;
#pragma unroll 4
    for (int k = k0; k < end; ++k) {
      const int p = order[k];
      const float* src = tags[p].valid == 2 ? firsts + (p >> 1) * C::kPiece
                                            : reinterpret_cast<const float*>(smem + (p >> 1) * S * C::kHalfBytes);
      const float f = piece_f[k * kRows + row];
      const float4 v = *reinterpret_cast<const float4*>(src + row * D + 4 * c);
      M = fmaxf(M, piece_m[p * kRows + row]);
      U = fmaxf(U, piece_u[p * kRows + row]);
      l += piece_w[k * kRows + row];
      o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
    }
    const Tag& head = tags[order[k0]];
    if (head.starts && tags[order[end - 1]].ends) {
      int64_t at;
      if (row_at(a, head.q0, head.q_len, head.rt * kRows + row, head.h, a.ldo, D, &at))
        store_out4<F32>(a, at + 4 * c, o, inverse(l), unit_of(M, U));
    } else {
      float* gp = a.part + ((int64_t)blockIdx.x * 2 + (head.starts ? 1 : 0)) * C::kPiece;
      *reinterpret_cast<float4*>(gp + row * D + 4 * c) = o;
      if (c == 0) {
        gp[kRows * D + row] = M;
        gp[kRows * D + kRows + row] = l;
        gp[kRows * D + 2 * kRows + row] = U;
      }
    }
  }
}

// Row tiles whose tokens fall to several CTAs: block c merges the pieces that
// CTAs c, c + 1, ... hold of the row tile that begins in CTA c.  Thread groups
// take every kGroups-th piece, so that a few loads in flight cover them all,
// and are joined through shared memory in their order.
constexpr int kMergeThreads = 1024;

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kMergeThreads) attn_merge_kernel(const __grid_constant__ Args a, int ctas) {
  using C = Cfg<D, NT, F32>;
  constexpr int kRows = C::kRows, kItems = kRows * D / 4, kGroups = kMergeThreads / kItems;
  __shared__ int first_end;
  __shared__ float4 so[kGroups][kItems];
  __shared__ float sm[kGroups][kItems], sl[kGroups][kItems], su[kGroups][kItems];
  if (threadIdx.x == 0) first_end = ctas;
  pdl_wait();
  pdl_launch();
  // this CTA's open run; the CTAs after it that hold more of the same row tile:
  // up to the first that has none or ends it
  const Tag head = a.meta[2 * blockIdx.x + 1];
  const int other = blockIdx.x + 1 + threadIdx.x;
  int valid = 0, ends = 0;
  if (other < ctas) {
    valid = a.meta[2 * other].valid;
    ends = a.meta[2 * other].ends;
  }
  if (!head.valid) return;
  __syncthreads();
  if (!valid) atomicMin(&first_end, (int)threadIdx.x);
  else if (ends) atomicMin(&first_end, (int)threadIdx.x + 1);
  __syncthreads();
  const int n = 1 + first_end;
  const float* first = a.part + ((int64_t)blockIdx.x * 2 + 1) * C::kPiece;
  const float* next = first + C::kPiece;                 // slot 0 of the CTA after, then every second piece
  const int x = threadIdx.x % kItems, grp = threadIdx.x / kItems;
  const int row = x / (D / 4), c = x % (D / 4);
  float M = -INFINITY, U = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m, float u, float lp, const float4& v) {
    const float Mn = fmaxf(M, m), Un = fmaxf(U, u);
    const float f0 = M == Mn ? 1.f : ex2(M - Mn), f1 = m == Mn ? 1.f : ex2(m - Mn);
    l = fmaf(l, U == Un ? 1.f : ex2(U - Un), lp * (u == Un ? 1.f : ex2(u - Un)));
    M = Mn;
    U = Un;
    o.x = fmaf(o.x, f0, v.x * f1); o.y = fmaf(o.y, f0, v.y * f1);
    o.z = fmaf(o.z, f0, v.z * f1); o.w = fmaf(o.w, f0, v.w * f1);
  };
  for (int p0 = grp; p0 < n; p0 += 4 * kGroups) {
    float m[4], lp[4], up[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + k * kGroups;
      if (p < n) {
        const float* src = p == 0 ? first : next + (int64_t)(p - 1) * 2 * C::kPiece;
        m[k] = src[kRows * D + row];
        lp[k] = src[kRows * D + kRows + row];
        up[k] = src[kRows * D + 2 * kRows + row];
        v[k] = *reinterpret_cast<const float4*>(src + row * D + 4 * c);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (p0 + k * kGroups < n) add(m[k], up[k], lp[k], v[k]);
  }
  so[grp][x] = o;
  sm[grp][x] = M;
  sl[grp][x] = l;
  su[grp][x] = U;
  __syncthreads();
  int64_t at;
  if (grp == 0 && row_at(a, head.q0, head.q_len, head.rt * kRows + row, head.h, a.ldo, D, &at)) {
    for (int k = 1; k < kGroups; ++k) add(sm[k][x], su[k][x], sl[k][x], so[k][x]);
    store_out4<F32>(a, at + 4 * c, o, inverse(l), unit_of(M, U));
  }
}

template <int D, int NT, bool F32>
lq_status launch_split(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, int ctas, void* stream) {
  using C = Cfg<D, NT, F32>;
  static_assert(C::kHalves >= 3 && C::kSmem + 2048 <= 227 * 1024, "shared memory");
  static_assert(C::kHalves * C::kHalfBytes >= C::kPiece * 4, "a warp's last piece fits its ring");
  static_assert(C::kRing >= LQ_MAX_REQUESTS * 8, "the prefix sums fit the rings");
  static_assert((2 + C::kWarps) * C::kPiece <= work_floats(D), "the pieces fit the workspace");
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
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
  if (e == cudaSuccess) {
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, attn_merge_kernel<D, NT, F32>, a, ctas);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  return check_launch();
}

bool encode_cache(CUtensorMap* map, const void* codes, int64_t bytes, int lines) {
  TensorMapEncodeTiledFn fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)lines};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One CTA per SM; the merge looks at all of them with one thread each.
int cta_count() {
  const int sms = device_sm_count();
  return sms <= 0 ? 152 : sms < kMergeThreads ? sms : kMergeThreads;
}

// Whether the tensor-core kernel takes a bf16 call: by the query rows that an
// average request has for each kv head.  Its time hardly depends on them up to
// 256, the split kernel's grows with every 16.  Measured at 8 kv heads, this
// kernel's time against the split kernel's at 16 / 24 / 32 / 64 rows, in us:
//   head_dim                      64                     128                       256
//   16 requests of 4000  55: 45/74/74/134    66: 51/85/85/153    106: 103/146/185/351
//   one of 32000 tokens  37: 31/44/44/73  43-49: 34/49/50/82      65: 61/79/100/178
//   one of 4000 tokens   20: 16/18/18/24     24: 18/21/21/25      32: 24/27/30/39
// (All rows alike: a batch that mixes prompts and single tokens gets one kernel by
// its average.)
bool many_rows(int batch, int64_t total_q, int group) {
  return batch > 0 && (total_q + batch - 1) / batch * group > 16;
}

size_t meta_bytes(int ctas) { return (ctas * 2 * sizeof(Tag) + 255) & ~(size_t)255; }

}  // namespace attn
}  // namespace lq

using namespace lq;

extern "C" size_t lq_attention_paged_workspace_size(int batch, int64_t total_q, int q_heads, int kv_heads,
                                                    int head_dim) {
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || kv_heads <= 0 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const int ctas = attn::cta_count();
  return attn::meta_bytes(ctas) + (size_t)ctas * attn::work_floats(head_dim) * sizeof(float);
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
                         !aligned4(k_scales_dev) || !aligned4(v_scales_dev)))
    return LQ_ERR_ARG;
  if (workspace_bytes < lq_attention_paged_workspace_size(batch, total_q, q_heads, kv_heads, head_dim))
    return LQ_ERR_SHAPE;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  attn::Args a;
  a.kc = k_cache_dev; a.vc = v_cache_dev;
  a.q = q_dev; a.ldq = ldq; a.total_q = total_q; a.cu_q = cu_q_dev; a.kv_lens = kv_lens_dev; a.batch = batch;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width;
  a.ks = k_scales_dev; a.vs = v_scales_dev; a.num_blocks = num_blocks;
  a.log2_bs = serve::log2_of(block_size); a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads;
  a.scale_log2 = sm_scale * 1.4426950408889634f; a.out = out_dev; a.ldo = ldo; a.status = dev_status_dev;
  a.meta = reinterpret_cast<attn::Tag*>(workspace_dev);
  const int ctas = attn::cta_count();
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace_dev) + attn::meta_bytes(ctas));
  // a pool without blocks: no copy is issued, any valid map will do
  const int8_t* kc = num_blocks > 0 ? k_cache_dev : reinterpret_cast<const int8_t*>(workspace_dev);
  const int8_t* vc = num_blocks > 0 ? v_cache_dev : reinterpret_cast<const int8_t*>(workspace_dev);
  const int64_t bytes = num_blocks > 0 ? num_blocks * block_rows * 128 : 32768;
  if (dtype == LQ_BF16 && attn::many_rows(batch, total_q, a.group))
    return attn::launch_attn_tiles(a, kc, vc, bytes, head_dim,
                                   attn::plan_tiles(batch, total_q, a.group, kv_heads, head_dim,
                                                    (int64_t)table_width * block_size, ctas),
                                   stream);
  CUtensorMap mk, mv;
  const int box = (block_size < attn::kTile ? block_size : attn::kTile) * head_dim / 128;
  if (!attn::encode_cache(&mk, kc, bytes, box) || !attn::encode_cache(&mv, vc, bytes, box)) return LQ_ERR_CUDA;
  // eight query rows per pass over the codes, sixteen where the average request has more
  const bool few = ((total_q + batch - 1) / batch) * a.group <= 8;
  if (dtype == LQ_F32) {
    if (head_dim == 64) return attn::launch_split<64, 1, true>(a, mk, mv, ctas, stream);
    if (head_dim == 128) return attn::launch_split<128, 1, true>(a, mk, mv, ctas, stream);
    return attn::launch_split<256, 1, true>(a, mk, mv, ctas, stream);
  }
  if (head_dim == 256) return attn::launch_split<256, 1, false>(a, mk, mv, ctas, stream);
  if (head_dim == 64) return few ? attn::launch_split<64, 1, false>(a, mk, mv, ctas, stream)
                                 : attn::launch_split<64, 2, false>(a, mk, mv, ctas, stream);
  return few ? attn::launch_split<128, 1, false>(a, mk, mv, ctas, stream)
             : attn::launch_split<128, 2, false>(a, mk, mv, ctas, stream);
}
