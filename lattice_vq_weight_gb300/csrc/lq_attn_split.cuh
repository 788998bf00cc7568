// Shared by the split kernels of the paged attention, which spread a batch's
// work over all SMs in equal parts whatever its requests' lengths are (lq_attn_paged.cu
// for the 8-bit cache, lq_attn_q4.cu for the 4-bit one): the list of tiles
// (request, tile of rows, kv head, tokens) and its division, a row's place, the joining
// of pieces of rows in a CTA and between CTAs.  Internal to the library.
#pragma once

#include "lq_attn_paged.cuh"

namespace lq {
namespace attn {

constexpr int kTile = 32;                      // tokens per tile, where a kernel does not say otherwise

// Floats of a piece: output rows, maxima, sums, their units.
__host__ __device__ constexpr int piece_floats(int rows, int head_dim) { return rows * (head_dim + 3); }

// A place in the list of tiles.
struct Cursor {
  int i;             // request
  int rt, nrt;       // tile of rows, and how many the request has
  int h;             // kv head
  int t, nt;         // tile of tokens, and how many the request has
  int len;
};

template <int ROWS, int TILE = kTile>
__device__ __forceinline__ void enter(const Args& a, Cursor& c) {
  const Request r = load_request(a, c.i);
  c.len = r.len;
  c.nrt = (r.q_len * a.group + ROWS - 1) / ROWS;
  c.nt = r.len > 0 ? (r.len + TILE - 1) / TILE : 1;
}

template <int ROWS, int TILE = kTile>
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
    enter<ROWS, TILE>(a, c);
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

// This warp's part of the list of tiles: how many, and ci the first.  Prefix sums
// of the requests' tiles give the list's length; the CTAs, and in them the warps,
// take equal parts (u0 and part_n).  pre: shared room for LQ_MAX_REQUESTS numbers,
// wsum: for one per warp.  All threads come here together.
template <int ROWS, int WARPS, int TILE = kTile>
__device__ __forceinline__ int part_of_warp(const Args& a, long long* pre, long long* wsum, Cursor& ci) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto tiles_of = [&](int i) {
    if (blockIdx.x == 0 && (int64_t)a.kv_lens[i] > ((int64_t)a.width << a.log2_bs))
      raise_flag(a.status, LQ_DEV_RANGE);
    Cursor c;
    c.i = i;
    enter<ROWS, TILE>(a, c);
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
    part_of(WARPS, warp);
  };
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
    const int per = (a.batch + 32 * WARPS - 1) / (32 * WARPS);
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
    for (int w = 0; w < WARPS; ++w) {
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
    enter<ROWS, TILE>(a, ci);
    const long long rem = u0 - before;
    const long long hr = rem < INT_MAX ? (unsigned)rem / (unsigned)ci.nt : rem / ci.nt;    // row tile and head
    ci.t = (int)(rem - hr * ci.nt);
    ci.rt = (int)(hr < INT_MAX ? (unsigned)hr / (unsigned)a.kv_heads : hr / a.kv_heads);
    ci.h = (int)(hr - (long long)ci.rt * a.kv_heads);
  }
  return n;
}

// Zeros to the rows that no request owns, from query token q_end on.
template <int D, int THREADS, bool F32>
__device__ __forceinline__ void zero_unowned(const Args& a, int q_end) {
  const int64_t cols = (int64_t)a.q_heads * D;
#pragma unroll 1
  for (int64_t t = (int64_t)max(q_end, 0) + blockIdx.x; t < a.total_q; t += gridDim.x)
#pragma unroll 1
    for (int64_t c = threadIdx.x; c < cols; c += THREADS) store_out<F32>(a, t * a.ldo + c, 0.f);
}

// Joins the warps' pieces of one CTA: rows that are complete go out, the rest to
// the workspace for the merge between CTAs.  piece_at(w, valid): the sums of a piece
// of warp w; order, piece_f and piece_w are room to work in.  All threads come here
// together, after a barrier behind which the pieces are written.
template <int D, int ROWS, int WARPS, bool F32, typename At>
__device__ __forceinline__ void join_pieces(const Args& a, const Tag* tags, int* order, const float* piece_m,
                                            const float* piece_l, const float* piece_u, float* piece_f, float* piece_w,
                                            At piece_at) {
  constexpr int kEnds = 2 * WARPS, kPiece = piece_floats(ROWS, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A run is the pieces of one row tile, which follow
  // each other; lane e of every warp looks at piece e
  const Tag mine = tags[lane < kEnds ? lane : 0];
  const bool valid = lane < kEnds && mine.valid;
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
  for (int x = threadIdx.x; x < pieces * ROWS; x += 32 * WARPS) {
    const int k = x / ROWS, row = x % ROWS, end = run_end(k);
    float M = -INFINITY, U = -INFINITY;
#pragma unroll 4
    for (int p = run_begin(k); p < end; ++p) {
      M = fmaxf(M, piece_m[order[p] * ROWS + row]);
      U = fmaxf(U, piece_u[order[p] * ROWS + row]);
    }
    const int own = order[k] * ROWS + row;
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
  constexpr int kItems = ROWS * D / 4;
  for (int x = threadIdx.x; x < runs * kItems; x += 32 * WARPS) {
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
      const float* src = piece_at(p >> 1, tags[p].valid);
      const float f = piece_f[k * ROWS + row];
      const float4 v = *reinterpret_cast<const float4*>(src + row * D + 4 * c);
      M = fmaxf(M, piece_m[p * ROWS + row]);
      U = fmaxf(U, piece_u[p * ROWS + row]);
      l += piece_w[k * ROWS + row];
      o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
    }
    const Tag& head = tags[order[k0]];
    if (head.starts && tags[order[end - 1]].ends) {
      int64_t at;
      if (row_at(a, head.q0, head.q_len, head.rt * ROWS + row, head.h, a.ldo, D, &at))
        store_out4<F32>(a, at + 4 * c, o, inverse(l), unit_of(M, U));
    } else {
      float* gp = a.part + ((int64_t)blockIdx.x * 2 + (head.starts ? 1 : 0)) * kPiece;
      *reinterpret_cast<float4*>(gp + row * D + 4 * c) = o;
      if (c == 0) {
        gp[ROWS * D + row] = M;
        gp[ROWS * D + ROWS + row] = l;
        gp[ROWS * D + 2 * ROWS + row] = U;
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
  constexpr int kRows = 8 * NT, kPiece = piece_floats(kRows, D), kItems = kRows * D / 4, kGroups = kMergeThreads / kItems;
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
  const float* first = a.part + ((int64_t)blockIdx.x * 2 + 1) * kPiece;
  const float* next = first + kPiece;                 // slot 0 of the CTA after, then every second piece
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
        const float* src = p == 0 ? first : next + (int64_t)(p - 1) * 2 * kPiece;
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

}  // namespace attn
}  // namespace lq
