// Writing keys and values into the paged 8-bit KV cache, and reading them back.
//
// A cache is [blocks x kv_heads x bs x head_dim] int8 codes and one fp32 scale
// per (block, head); it stands for code * scale.  New rows that fall into one
// block (a run of consecutive slots) share the block's scale with the rows
// already there:
//     s_old = 0 when the run starts the block, else the stored scale
//     s     = max(s_old, max |x| / 127 over the run)
//     new rows: rint(x / s);  rows before the run, when s > s_old: rint(c s_old / s)
// with IEEE fp32 quotients, so the codes depend on nothing but the order in
// which tokens arrive.
//
// Append: runs are found from the slots alone (a token whose predecessor is not
// the slot before it in the same block starts one), so no block list has to be
// built first.  A CTA looks through a window of tokens for one head, four warps
// for K and four for V.  Long runs (prompts) are shared by the four, which hold
// the run in registers between the maximum and the codes, so that it is read
// once and in one round of loads; where a window holds many runs (decode steps)
// each warp takes runs of its own.  An IEEE division per value would bound the
// kernel, so codes come from a product with 1/s wherever that is clear of a
// half by more than its error, and from the exact remainder where it is not.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace paged {

constexpr int kWarps = 4;                          // for each of K and V
constexpr int kThreads = 2 * kWarps * 32;

struct AppendArgs {
  const void* x[2];          // k, v
  int64_t ld[2];
  int8_t* cache[2];
  float* scales[2];
  const int64_t* slots;
  int64_t tokens, slots_in_cache;
  int kv_heads, dim, log2_bs, window;
  int32_t* status;
};

// Eight values of a row as loaded: one 16-byte word of bf16, two of fp32.
template <bool BF16>
struct Raw {
  uint4 w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* p, int64_t i) {
  Raw<BF16> r;
  if constexpr (BF16) {
    r.w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
  } else {
    r.w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + i);
    r.w[1] = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + i)[1];
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void values(const Raw<BF16>& r, float (&v)[8]) {
  if constexpr (BF16) {
    const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[4 * h] = __uint_as_float(r.w[h].x); v[4 * h + 1] = __uint_as_float(r.w[h].y);
      v[4 * h + 2] = __uint_as_float(r.w[h].z); v[4 * h + 3] = __uint_as_float(r.w[h].w);
    }
  }
}

// Running maximum of the magnitudes as bit patterns, which are ordered like
// the numbers and put infinities and NaN on top: two bf16 side by side, or one
// fp32.
constexpr uint32_t kInf = 0x7F800000u;
template <bool BF16>
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const Raw<BF16>& r) {
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
    const uint32_t u[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = BF16 ? __vmaxu2(m, u[e] & 0x7FFF7FFFu) : max(m, u[e] & 0x7FFFFFFFu);
  }
  return m;
}

__device__ __forceinline__ uint32_t pack4(const int (&c)[4]) {
  return (uint32_t)(c[0] & 255) | (uint32_t)(c[1] & 255) << 8 | (uint32_t)(c[2] & 255) << 16 | (uint32_t)c[3] << 24;
}

// rint of the IEEE quotient, clipped to the code range; 0 for a non-finite x.
__device__ __forceinline__ int code_of(float x, float s) {
  const float q = rintf(__fdiv_rn(x, s));
  return fabsf(x) <= 3.402823466e38f ? (int)fminf(fmaxf(q, -127.f), 127.f) : 0;
}

// Eight codes by division: for values that are not finite and for 1/s out of
// the normal range.
__noinline__ __device__ uint2 codes8_exact(float4 a, float4 b, float s) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t out[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) code[e] = code_of(v[4 * q + e], s);
    out[q] = pack4(code);
  }
  return make_uint2(out[0], out[1]);
}
// rint of the IEEE quotient x / s by its remainder, given the sign-carrying
// nearest half h = n +- 1/2 of x * inv: the quotient is h itself (and goes to the
// even neighbour) when |x - h s| is at most half a unit in h's last place times
// s, else on the side of h that the exact remainder tells.  (Below 1/2 units are
// half as large.)
__device__ __forceinline__ float by_remainder(float x, float h, float s) {
  const float e = fmaf(-h, s, x);                  // exact where it is small
  float unit = __uint_as_float(__float_as_uint(h) & 0x7F800000u) * 5.9604644775390625e-8f;      // 2^-24
  const bool away = (__float_as_uint(e) ^ __float_as_uint(h)) >> 31 == 0;       // |x / s| > |h|
  if (fabsf(h) == 0.5f && !away) unit *= 0.5f;
  return fabsf(e) <= unit * s ? rintf(h) : h + copysignf(0.5f, e);
}

// Codes of eight values with |x| <= 127 s (up to rounding): rint(x * inv) by
// adding 1.5 * 2^23, whose low byte is then the code.  The quotient x / s is
// within 127 * 2^-23 of x * inv (two roundings), so rounding agrees unless
// x * inv is within 2^-15 of a half; bf16 values are often exactly there (half of
// the block's largest is), so that case is settled by remainders, not divisions.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv, float s, bool careful) {
  constexpr float kMagic = 12582912.f;
  float t[8], f[8], off = 0.f;
  const float2 inv2 = make_float2(inv, inv), magic2 = make_float2(kMagic, kMagic);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 x = make_float2(v[e], v[e + 1]), t2 = fma2(x, inv2, magic2), f2 = fma2(x, inv2, sub2(magic2, t2));
    t[e] = t2.x; t[e + 1] = t2.y;
    f[e] = f2.x; f[e + 1] = f2.y;
    off = fmaxf(off, fmaxf(fabsf(f2.x), fabsf(f2.y)));
  }
  if (careful) return codes8_exact(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]), s);
  if (off > 0.5f - 0.000030517578125f) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      t[e] = kMagic + by_remainder(v[e], (t[e] - kMagic) + copysignf(0.5f, f[e]), s);
  }
  uint32_t out[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t lo = __byte_perm(__float_as_uint(t[4 * q]), __float_as_uint(t[4 * q + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(t[4 * q + 2]), __float_as_uint(t[4 * q + 3]), 0x0040);
    out[q] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(out[0], out[1]);
}

// Eight codes of a block times the scale they were made with.
__device__ __forceinline__ void old_values(const uint2& w, float s_old, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = (float)(int8_t)(w.x >> (8 * e)) * s_old;
    v[4 + e] = (float)(int8_t)(w.y >> (8 * e)) * s_old;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2) append_kernel(AppendArgs a) {
  constexpr int kHold = 8;                         // rows that a lane of a shared run keeps
  __shared__ uint32_t s_max[2][kWarps];
  __shared__ float s_fin[2][kWarps];
  const int lane = threadIdx.x & 31, which = threadIdx.x >> 7, warp = (threadIdx.x >> 5) & (kWarps - 1);
  pdl_wait();
  pdl_launch();
  const unsigned win = blockIdx.x / (unsigned)a.kv_heads;
  const int h = (int)(blockIdx.x - win * (unsigned)a.kv_heads);
  const int bs1 = (1 << a.log2_bs) - 1;

  // the slots of the window, and of the up to 127 tokens after it that a run
  // may carry on to: lane l has slots l, l + 32, ...
  const int64_t t0 = (int64_t)win * a.window;
  int64_t ahead[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    ahead[i] = (i == 0 || 32 * i < a.window + bs1) && t0 + 32 * i + lane < a.tokens
                   ? a.slots[t0 + 32 * i + lane] : -1;
  const int64_t prev = lane < a.window && t0 + lane > 0 && t0 + lane < a.tokens ? a.slots[t0 + lane - 1] : -1;
  const int64_t mine = ahead[0];
  const bool starts = lane < a.window && mine >= 0 && !(prev >= 0 && prev + 1 == mine && (mine & bs1) != 0);
  if (starts && mine >= a.slots_in_cache) raise_flag(a.status, LQ_DEV_RANGE);
  uint32_t todo = __ballot_sync(0xffffffffu, starts && mine < a.slots_in_cache);
  if (todo == 0) return;                           // the same in every warp
  const bool shared = __popc(todo) < kWarps;

  const void* x = which ? a.x[1] : a.x[0];
  const int64_t ld = which ? a.ld[1] : a.ld[0];
  int8_t* cache = which ? a.cache[1] : a.cache[0];
  float* scales = which ? a.scales[1] : a.scales[0];
  // a lane holds 8 dimensions of a row; 32 / (dim / 8) rows side by side
  const int chunks = a.dim >> 3, rows_step = 32 / chunks;
  const int k0 = 8 * (lane % chunks);
  const int r0 = lane < rows_step * chunks ? lane / chunks + (shared ? warp * rows_step : 0) : 1 << 20;
  const int step = shared ? kWarps * rows_step : rows_step;

  for (int n = 0; todo; ++n) {
    const int first = __ffs(todo) - 1;
    todo &= todo - 1;
    if (!shared && n % kWarps != warp) continue;
    const int64_t slot = __shfl_sync(0xffffffffu, mine, first), t = t0 + first;
    const int off = (int)(slot & bs1), most = bs1 + 1 - off;
    const int64_t sc = (slot >> a.log2_bs) * a.kv_heads + h;
    const float s_old = off > 0 ? scales[sc] : 0.f;
    // the run's length: tokens that carry on with consecutive slots of the block
    int len = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int p = 32 * i + lane - first;         // token of the run
      const uint32_t stop = __ballot_sync(0xffffffffu, p >= 0 && !(p < most && ahead[i] == slot + p));
      if (len == 32 * i - (i ? first : 0)) len = stop ? 32 * i + __ffs(stop) - 1 - first : 32 * (i + 1) - first;
    }
    const int64_t src = t * ld + (int64_t)h * a.dim + k0;
    int8_t* rows = cache + (sc << a.log2_bs) * a.dim + k0;

    Raw<BF16> held[kHold];
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * step < len) held[i] = load_raw<BF16>(x, src + (r0 + i * step) * ld);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * step < len) mb = max_bits<BF16>(mb, held[i]);
#pragma unroll 4
    for (int r = r0 + kHold * step; r < len; r += step) mb = max_bits<BF16>(mb, load_raw<BF16>(x, src + r * ld));
    if constexpr (BF16) mb = max(mb << 16, mb & 0xFFFF0000u);
    mb = __reduce_max_sync(0xffffffffu, mb);
    if (shared) {
      __syncthreads();                             // the run before has been read
      if (lane == 0) s_max[which][warp] = mb;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; ++i) mb = max(mb, s_max[which][i]);
    }
    float mx = __uint_as_float(mb);
    // something non-finite, in K or V where the run is shared: the maximum over the rest
    const bool odd = mb >= kInf;
    if (shared ? __syncthreads_or(odd) : odd) {
      mx = 0.f;
#pragma unroll 1
      for (int r = r0; r < len; r += step) {
        float v[8];
        values<BF16>(load_raw<BF16>(x, src + r * ld), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(v[e]) <= 3.402823466e38f) mx = fmaxf(mx, fabsf(v[e]));
      }
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      if (shared) {
        if (lane == 0) s_fin[which][warp] = mx;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, s_fin[which][i]);
      }
      if (odd && lane == 0) raise_flag(a.status, LQ_DEV_NONFINITE);
    }
    const float s = fmaxf(s_old, __fdiv_rn(mx, 127.f));
    const float d = s > 0.f ? s : 1.f, inv = 1.f / d;
    // non-finite values, or 1/s out of the normal range
    const bool slow = odd || !(inv <= 3.402823466e38f) || d < 1e-37f;
    if (s > s_old && off > 0) {
#pragma unroll 1
      for (int r = r0; r < off; r += step) {
        uint2* p = reinterpret_cast<uint2*>(rows + r * a.dim);
        float v[8];
        old_values(*p, s_old, v);
        *p = codes8(v, inv, d, slow);
      }
    }
    int8_t* to = rows + off * a.dim;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int r = r0 + i * step;
      if (r < len) {
        float v[8];
        values<BF16>(held[i], v);
        *reinterpret_cast<uint2*>(to + r * a.dim) = codes8(v, inv, d, slow);
      }
    }
#pragma unroll 2
    for (int r = r0 + kHold * step; r < len; r += step) {
      float v[8];
      values<BF16>(load_raw<BF16>(x, src + r * ld), v);
      *reinterpret_cast<uint2*>(to + r * a.dim) = codes8(v, inv, d, slow);
    }
    if (lane == 0 && (!shared || warp == 0)) scales[sc] = s;
  }
}

struct GatherArgs {
  const int64_t* slots;
  const int8_t* cache[2];
  const float* scales[2];
  void* out[2];
  int64_t n, slots_in_cache;
  int kv_heads, dim, log2_bs;
  int32_t* status;
};

// out = code * scale, fp32 or rounded once to bf16: a warp per slot and cache,
// 16 bytes of output per lane and step, the loads of eight steps and the next
// slot in flight at once.
template <bool BF16>
__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
  constexpr int E = BF16 ? 8 : 4;                  // codes per lane and step
  constexpr int U = 8;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const unsigned chunks = (unsigned)(a.dim / E), per_row = (unsigned)a.kv_heads * chunks;
  // c / chunks for c < 2^16, chunks <= 64: the high word of c * ceil(2^32 / chunks)
  const unsigned magic = 0xffffffffu / chunks + 1u;
  const int64_t warps = (int64_t)gridDim.x * 8;
  int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  int64_t slot = u < 2 * a.n ? a.slots[u >> 1] : -1;
  for (; u < 2 * a.n; u += warps) {
    const int which = (int)(u & 1);
    const int64_t next = u + warps < 2 * a.n ? a.slots[(u + warps) >> 1] : -1;
    const bool ok = slot >= 0 && slot < a.slots_in_cache;
    if (slot >= a.slots_in_cache && lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
    const int64_t sc0 = (slot >> a.log2_bs) * a.kv_heads;
    const int off = (int)(slot & ((1 << a.log2_bs) - 1));
    const float* scales = (which ? a.scales[1] : a.scales[0]) + sc0;
    const int8_t* codes = (which ? a.cache[1] : a.cache[0]) + ((sc0 << a.log2_bs) + off) * a.dim;
    uint4* out = reinterpret_cast<uint4*>(which ? a.out[1] : a.out[0]) + (u >> 1) * per_row;
    for (unsigned c0 = 0; c0 < per_row; c0 += 32 * U) {
      uint2 w[U];
      float s[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const unsigned c = c0 + 32 * i + lane;
        w[i] = make_uint2(0u, 0u);
        s[i] = 0.f;
        if (ok && c < per_row) {
          const unsigned h = __umulhi(c, magic), k = E * (c - h * chunks);
          const int8_t* p = codes + ((int64_t)h << a.log2_bs) * a.dim + k;
          s[i] = scales[h];
          if constexpr (BF16) w[i] = *reinterpret_cast<const uint2*>(p);
          else w[i].x = *reinterpret_cast<const uint32_t*>(p);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const unsigned c = c0 + 32 * i + lane;
        if (c >= per_row) break;
        float v[8];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (float)(int8_t)((e < 4 ? w[i].x : w[i].y) >> (8 * (e & 3))) * s[i];
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            o[e] = *reinterpret_cast<const uint32_t*>(&b);
          } else {
            o[e] = __float_as_uint(v[e]);
          }
        }
        out[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    slot = next;
  }
}

}  // namespace paged
}  // namespace lq

using namespace lq;

namespace {

// Checks of a cache shared by the calls that take one.
lq_status check_cache(const void* k_cache, const void* k_scales, const void* v_cache, const void* v_scales,
                      int64_t num_blocks, int block_size, int kv_heads, int head_dim) {
  if (!serve::valid_block_size(block_size)) return LQ_ERR_UNSUPPORTED;
  if (head_dim <= 0 || head_dim > 256 || head_dim % 16 != 0) return LQ_ERR_UNSUPPORTED;
  if (num_blocks < 0 || num_blocks > INT32_MAX || kv_heads <= 0 || kv_heads > 1024) return LQ_ERR_SHAPE;
  if (num_blocks > 0 && (k_cache == nullptr || v_cache == nullptr || k_scales == nullptr || v_scales == nullptr ||
                         !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(k_scales) || !aligned4(v_scales)))
    return LQ_ERR_ARG;
  return LQ_OK;
}

}  // namespace

extern "C" lq_status lq_kv_append(const void* k_dev, int64_t ldk, const void* v_dev, int64_t ldv, int dtype,
                                  int64_t tokens, const int64_t* slots_dev, int8_t* k_cache_dev, float* k_scales_dev,
                                  int8_t* v_cache_dev, float* v_scales_dev, int64_t num_blocks, int block_size,
                                  int kv_heads, int head_dim, int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_kv_append");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  const lq_status st = check_cache(k_cache_dev, k_scales_dev, v_cache_dev, v_scales_dev, num_blocks, block_size,
                                   kv_heads, head_dim);
  if (st != LQ_OK) return st;
  const int64_t esize = dtype == LQ_BF16 ? 2 : 4, cols = (int64_t)kv_heads * head_dim;
  if (tokens < 0 || tokens > INT32_MAX || ldk < cols || ldv < cols || (ldk * esize) % 16 != 0 ||
      (ldv * esize) % 16 != 0)
    return LQ_ERR_SHAPE;
  if (tokens == 0) return LQ_OK;
  if (k_dev == nullptr || v_dev == nullptr || slots_dev == nullptr || !aligned16(k_dev) || !aligned16(v_dev) ||
      !serve::aligned8(slots_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  paged::AppendArgs a;
  a.x[0] = k_dev; a.x[1] = v_dev; a.ld[0] = ldk; a.ld[1] = ldv;
  a.cache[0] = k_cache_dev; a.cache[1] = v_cache_dev; a.scales[0] = k_scales_dev; a.scales[1] = v_scales_dev;
  a.slots = slots_dev; a.tokens = tokens; a.slots_in_cache = num_blocks * block_size;
  a.kv_heads = kv_heads; a.dim = head_dim; a.log2_bs = serve::log2_of(block_size); a.status = dev_status_dev;
  // tokens that one CTA looks through for runs: one while that fits one wave of
  // resident CTAs (decode steps: every token is a run), up to 32 for long
  // prompts, where most tokens start none
  const int64_t ctas = tokens * kv_heads, wave = (int64_t)sms * 8;
  int64_t window = (ctas + wave - 1) / wave;
  a.window = (int)(window > 32 ? 32 : window);
  const int64_t grid = (tokens + a.window - 1) / a.window * kv_heads;
  if (grid > INT32_MAX) return LQ_ERR_SHAPE;
  return dtype == LQ_BF16 ? serve::launch(paged::append_kernel<true>, (unsigned)grid, paged::kThreads, 0, stream, a)
                          : serve::launch(paged::append_kernel<false>, (unsigned)grid, paged::kThreads, 0, stream, a);
}

extern "C" lq_status lq_kv_gather(const int64_t* slots_dev, int64_t n, const int8_t* k_cache_dev,
                                  const float* k_scales_dev, const int8_t* v_cache_dev, const float* v_scales_dev,
                                  int64_t num_blocks, int block_size, int kv_heads, int head_dim, void* k_out_dev,
                                  void* v_out_dev, int out_dtype, int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_kv_gather");
  if (out_dtype != LQ_BF16 && out_dtype != LQ_F32) return LQ_ERR_DTYPE;
  const lq_status st = check_cache(k_cache_dev, k_scales_dev, v_cache_dev, v_scales_dev, num_blocks, block_size,
                                   kv_heads, head_dim);
  if (st != LQ_OK) return st;
  if (n < 0 || n > (int64_t(1) << 40) / ((int64_t)kv_heads * head_dim)) return LQ_ERR_SHAPE;
  if (n == 0) return LQ_OK;
  if (slots_dev == nullptr || k_out_dev == nullptr || v_out_dev == nullptr || !serve::aligned8(slots_dev) ||
      !aligned16(k_out_dev) || !aligned16(v_out_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  paged::GatherArgs a;
  a.slots = slots_dev; a.cache[0] = k_cache_dev; a.cache[1] = v_cache_dev;
  a.scales[0] = k_scales_dev; a.scales[1] = v_scales_dev; a.out[0] = k_out_dev; a.out[1] = v_out_dev;
  a.n = n; a.slots_in_cache = num_blocks * block_size;
  a.kv_heads = kv_heads; a.dim = head_dim; a.log2_bs = serve::log2_of(block_size); a.status = dev_status_dev;
  int64_t grid = (2 * n + 7) / 8;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  return out_dtype == LQ_BF16 ? serve::launch(paged::gather_kernel<true>, (unsigned)grid, 256, 0, stream, a)
                              : serve::launch(paged::gather_kernel<false>, (unsigned)grid, 256, 0, stream, a);
}
