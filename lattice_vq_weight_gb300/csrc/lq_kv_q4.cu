// Writing keys and values into the paged 4-bit cache and reading them back
// (the format: lq_q4.cuh).
//
// A group of G values x becomes, in IEEE fp32 steps,
//     s = fp16((max x - min x) / 15),  b = fp16(min x - 16 s),  r = 1 / s,
//     c = rint((x - b) r) - 16, cut to 0 .. 15  (0 where s is 0),
// so codes, scales and bases are functions of the inputs alone, bit for bit.
// Every vector has its own scales: rows of one call do not depend on one
// another or on what the cache holds.
//
// Bound by HBM: reading the values (2 or 4 bytes each) against half a byte of
// codes written, and the other way round.
#include "lq_device.cuh"
#include "lq_host.h"
#include "lq_q4.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace q4 {

constexpr int kThreads = 256;

struct AppendArgs {
  const void* x[2];          // k, v
  int64_t ld[2];
  uint32_t* codes[2];
  uint32_t* scales[2];       // (scale, base) pairs
  const int64_t* slots;
  int64_t tokens, slots_in_cache;
  int kv_heads, log2_dim, log2_bs, log2_group;
  int32_t* status;
};

// Eight values as they are in memory: 16 bytes, or 32.
template <bool BF16>
struct Raw {
  uint4 w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void* p, int64_t i) {
  Raw<BF16> r;
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4));
  r.w[0] = q[0];
  if constexpr (!BF16) r.w[1] = q[1];
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw<BF16>& r, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < (BF16 ? 1 : 2); ++k) {
    const uint32_t u[4] = {r.w[k].x, r.w[k].y, r.w[k].z, r.w[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF16) {
        v[2 * e] = __uint_as_float(u[e] << 16);
        v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      } else {
        v[4 * k + e] = __uint_as_float(u[e]);
      }
    }
  }
}
// Whether one of them is beyond kMost or not a number, by the order of the bits.
template <bool BF16>
__device__ __forceinline__ bool beyond(const Raw<BF16>& r) {
  if constexpr (BF16) {
    const uint32_t m = 0x7FFF7FFFu, top = __vmaxu2(__vimax3_u16x2(r.w[0].x & m, r.w[0].y & m, r.w[0].z & m), r.w[0].w & m);
    return max(top >> 16, top & 0xFFFFu) > (__float_as_uint(kMost) >> 16);
  } else {
    const uint32_t m = 0x7FFFFFFFu;
    const uint32_t top = max(__vimax3_u32(__vimax3_u32(r.w[0].x & m, r.w[0].y & m, r.w[0].z & m), r.w[0].w & m, r.w[1].x & m),
                             __vimax3_u32(r.w[1].y & m, r.w[1].z & m, r.w[1].w & m));
    return top > __float_as_uint(kMost);
  }
}

// A warp per token and cache, eight values per lane and step: a lane's codes are one
// word, a group G / 8 neighbouring lanes.  The loads of kUnroll steps are in flight at
// once (one after the other, the write and read-back of 13 944 tokens took 76 us).
template <bool BF16, int GROUP>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  constexpr int kUnroll = BF16 ? 4 : 2, span = GROUP / 8, log2_span = span == 4 ? 2 : span == 8 ? 3 : 4;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int log2_words = a.log2_dim - 3;
  const int per_row = a.kv_heads << log2_words;
  int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  int64_t slot = u < 2 * a.tokens ? a.slots[u >> 1] : -1;
  for (; u < 2 * a.tokens; u += warps) {
    const int64_t t = u >> 1, here = slot;
    const int which = (int)(u & 1);
    slot = u + warps < 2 * a.tokens ? a.slots[(u + warps) >> 1] : -1;
    if (here < 0) continue;
    if (here >= a.slots_in_cache) {
      if (lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
      continue;
    }
    const int64_t first = ((here >> a.log2_bs) * a.kv_heads << a.log2_bs) + (here & ((1 << a.log2_bs) - 1));
    const void* x = which ? a.x[1] : a.x[0];
    const int64_t row = t * (which ? a.ld[1] : a.ld[0]);
    uint32_t* codes = (which ? a.codes[1] : a.codes[0]) + (first << log2_words);
    uint32_t* scales = (which ? a.scales[1] : a.scales[0]) + (first << (log2_words - log2_span));
    for (int c0 = lane; c0 - lane < per_row; c0 += 32 * kUnroll) {
      Raw<BF16> raw[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        raw[i].w[0] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!BF16) raw[i].w[1] = make_uint4(0u, 0u, 0u, 0u);
        if (c0 + 32 * i < per_row) raw[i] = load8<BF16>(x, row + 8 * (c0 + 32 * i));
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + 32 * i;
        if (c - lane >= per_row) break;
        float v[8];
        unpack8<BF16>(raw[i], v);
        if (beyond<BF16>(raw[i])) {            // seldom
          for (int e = 0; e < 8; ++e) {
            if (fabsf(v[e]) < INFINITY) {
              if (fabsf(v[e]) > kMost) raise_flag(a.status, LQ_DEV_RANGE);
              v[e] = fminf(fmaxf(v[e], -kMost), kMost);
            } else {
              raise_flag(a.status, LQ_DEV_NONFINITE);
              v[e] = 0.f;
            }
          }
        }
        float low = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), fminf(fminf(v[4], v[5]), fminf(v[6], v[7])));
        float high = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
        if constexpr (BF16) {
          // (bf16 numbers both: they cross together)
          __nv_bfloat162 both = __floats2bfloat162_rn(low, -high);
#pragma unroll
          for (int o = 1; o < span; o <<= 1) both = __hmin2(both, __shfl_xor_sync(0xffffffffu, both, o));
          low = __low2float(both);
          high = -__high2float(both);
        } else {
#pragma unroll
          for (int o = 1; o < span; o <<= 1) {
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
          }
        }
        const __half s = __float2half_rn(__fdiv_rn(__fsub_rn(high, low), 15.f));
        const float sf = __half2float(s);
        const __half b = __float2half_rn(__fsub_rn(low, 16.f * sf));
        const float bf = __half2float(b), r = sf > 0.f ? __frcp_rn(sf) : 0.f;
        // (x - b) r rounded: the last places of its sum with 1.5 2^23 (it is below 2^17: a
        // group is at least a last place of its values wide, and b off by 2^-12 of itself)
        // (The products one by one: the packed product and sum would become one fma, which
        // does not round the product.)
        const float2 minus = make_float2(-bf, -bf), magic = make_float2(12582912.f, 12582912.f);
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 d = add2(make_float2(v[e], v[e + 1]), minus);
          const float2 q = add2(make_float2(__fmul_rn(d.x, r), __fmul_rn(d.y, r)), magic);
          word += (uint32_t)__vimin_s32_relu(__float_as_int(q.x) - 0x4B400010, 15) << (4 * e);
          word += (uint32_t)__vimin_s32_relu(__float_as_int(q.y) - 0x4B400010, 15) << (4 * e + 4);
        }
        if (c < per_row) {
          const int h = c >> log2_words, w = c & ((1 << log2_words) - 1);
          codes[(h << (a.log2_bs + log2_words)) + w] = word;
          if ((w & (span - 1)) == 0)
            scales[(h << (a.log2_bs + log2_words - log2_span)) + (w >> log2_span)] =
                (uint32_t)__half_as_ushort(s) | (uint32_t)__half_as_ushort(b) << 16;
        }
      }
    }
  }
}

struct GatherArgs {
  const int64_t* slots;
  const uint32_t* codes[2];
  const uint32_t* scales[2];
  void* out[2];
  int64_t n, slots_in_cache;
  int kv_heads, log2_dim, log2_bs, log2_group;
  int32_t* status;
};

// A warp per slot and cache, 16 bytes of output per lane and step: a word of codes for
// bf16, half of one for fp32; the loads of kUnroll steps in flight at once.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) gather_kernel(GatherArgs a) {
  constexpr int kUnroll = 4;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  // steps of a vector: 8 or 4 values each
  const int log2_steps = a.log2_dim - (BF16 ? 3 : 2), log2_words = a.log2_dim - 3;
  const int log2_groups = a.log2_dim - a.log2_group, per_row = a.kv_heads << log2_steps;
  int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  int64_t next = u < 2 * a.n ? a.slots[u >> 1] : -1;
  for (; u < 2 * a.n; u += warps) {
    const int64_t slot = next;
    const int which = (int)(u & 1);
    next = u + warps < 2 * a.n ? a.slots[(u + warps) >> 1] : -1;
    const bool ok = slot >= 0 && slot < a.slots_in_cache;
    if (slot >= a.slots_in_cache && lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
    const int64_t first = ((slot >> a.log2_bs) * a.kv_heads << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1));
    const uint32_t* codes = (which ? a.codes[1] : a.codes[0]) + (first << log2_words);
    const uint32_t* scales = (which ? a.scales[1] : a.scales[0]) + (first << log2_groups);
    uint4* out = reinterpret_cast<uint4*>(which ? a.out[1] : a.out[0]) + (u >> 1) * per_row;
    for (int c0 = lane; c0 < per_row; c0 += 32 * kUnroll) {
      uint32_t word[kUnroll], pr[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + 32 * i, h = c >> log2_steps, k = c & ((1 << log2_steps) - 1);
        word[i] = pr[i] = 0u;                  // scale and base 0: zeros
        if (ok && c < per_row) {
          word[i] = codes[(h << (a.log2_bs + log2_words)) + (BF16 ? k : k >> 1)];
          pr[i] = scales[(h << (a.log2_bs + log2_groups)) + (k >> (log2_steps - log2_groups))];
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + 32 * i;
        if (c >= per_row) break;
        uint32_t o[4];
        if constexpr (BF16) {
          float v[8];
          values8(word[i], pr[i], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            o[e] = *reinterpret_cast<const uint32_t*>(&p);
          }
        } else {
          // four codes of the word's half: 0 and 2 below 1 and 3
          const uint32_t half = __byte_perm(word[i], 0u, c & 1 ? 0x4432 : 0x4410);
          const uint32_t w = half + (half & 0xFFF0u) * 4096u;
          const uint32_t s = twice_low(pr[i]), b = twice_high(pr[i]);
          const uint32_t x = fma_h2(((w << 6) & 0x03C003C0u) | 0x4C004C00u, s, b);
          const uint32_t y = fma_h2(((w >> 2) & 0x03C003C0u) | 0x4C004C00u, s, b);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&y));
          o[0] = __float_as_uint(f.x);
          o[1] = __float_as_uint(f.y);
          o[2] = __float_as_uint(g.x);
          o[3] = __float_as_uint(g.y);
        }
        out[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace q4
}  // namespace lq

using namespace lq;

namespace {

lq_status check_cache(const void* k_cache, const void* k_scales, const void* v_cache, const void* v_scales,
                      int64_t num_blocks, int block_size, int kv_heads, int head_dim, int group_size) {
  if (!serve::valid_block_size(block_size) || !q4::valid_dims(head_dim, group_size)) return LQ_ERR_UNSUPPORTED;
  if (num_blocks < 0 || num_blocks > INT32_MAX || kv_heads <= 0 || kv_heads > 1024) return LQ_ERR_SHAPE;
  if (num_blocks > 0 && (k_cache == nullptr || v_cache == nullptr || k_scales == nullptr || v_scales == nullptr ||
                         !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) || !aligned16(v_scales)))
    return LQ_ERR_ARG;
  return LQ_OK;
}

}  // namespace

extern "C" lq_status lq_kv_append_q4(const void* k_dev, int64_t ldk, const void* v_dev, int64_t ldv, int dtype,
                                     int64_t tokens, const int64_t* slots_dev, uint8_t* k_cache_dev,
                                     uint16_t* k_scales_dev, uint8_t* v_cache_dev, uint16_t* v_scales_dev,
                                     int64_t num_blocks, int block_size, int kv_heads, int head_dim, int group_size,
                                     int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_kv_append_q4");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  const lq_status st = check_cache(k_cache_dev, k_scales_dev, v_cache_dev, v_scales_dev, num_blocks, block_size,
                                   kv_heads, head_dim, group_size);
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
  q4::AppendArgs a;
  a.x[0] = k_dev; a.x[1] = v_dev; a.ld[0] = ldk; a.ld[1] = ldv;
  a.codes[0] = reinterpret_cast<uint32_t*>(k_cache_dev); a.codes[1] = reinterpret_cast<uint32_t*>(v_cache_dev);
  a.scales[0] = reinterpret_cast<uint32_t*>(k_scales_dev); a.scales[1] = reinterpret_cast<uint32_t*>(v_scales_dev);
  a.slots = slots_dev; a.tokens = tokens; a.slots_in_cache = num_blocks * block_size;
  a.kv_heads = kv_heads; a.log2_dim = serve::log2_of(head_dim); a.log2_bs = serve::log2_of(block_size);
  a.log2_group = serve::log2_of(group_size); a.status = dev_status_dev;
  int64_t grid = (2 * tokens + 7) / 8;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  void (*const kernels[2][3])(q4::AppendArgs) = {
      {q4::append_kernel<false, 32>, q4::append_kernel<false, 64>, q4::append_kernel<false, 128>},
      {q4::append_kernel<true, 32>, q4::append_kernel<true, 64>, q4::append_kernel<true, 128>}};
  return serve::launch(kernels[dtype == LQ_BF16][a.log2_group - 5], (unsigned)grid, q4::kThreads, 0, stream, a);
}

extern "C" lq_status lq_kv_gather_q4(const int64_t* slots_dev, int64_t n, const uint8_t* k_cache_dev,
                                     const uint16_t* k_scales_dev, const uint8_t* v_cache_dev,
                                     const uint16_t* v_scales_dev, int64_t num_blocks, int block_size, int kv_heads,
                                     int head_dim, int group_size, void* k_out_dev, void* v_out_dev, int out_dtype,
                                     int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_kv_gather_q4");
  if (out_dtype != LQ_BF16 && out_dtype != LQ_F32) return LQ_ERR_DTYPE;
  const lq_status st = check_cache(k_cache_dev, k_scales_dev, v_cache_dev, v_scales_dev, num_blocks, block_size,
                                   kv_heads, head_dim, group_size);
  if (st != LQ_OK) return st;
  if (n < 0 || n > (int64_t(1) << 40) / ((int64_t)kv_heads * head_dim)) return LQ_ERR_SHAPE;
  if (n == 0) return LQ_OK;
  if (slots_dev == nullptr || k_out_dev == nullptr || v_out_dev == nullptr || !serve::aligned8(slots_dev) ||
      !aligned16(k_out_dev) || !aligned16(v_out_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  q4::GatherArgs a;
  a.slots = slots_dev;
  a.codes[0] = reinterpret_cast<const uint32_t*>(k_cache_dev);
  a.codes[1] = reinterpret_cast<const uint32_t*>(v_cache_dev);
  a.scales[0] = reinterpret_cast<const uint32_t*>(k_scales_dev);
  a.scales[1] = reinterpret_cast<const uint32_t*>(v_scales_dev);
  a.out[0] = k_out_dev; a.out[1] = v_out_dev; a.n = n; a.slots_in_cache = num_blocks * block_size;
  a.kv_heads = kv_heads; a.log2_dim = serve::log2_of(head_dim); a.log2_bs = serve::log2_of(block_size);
  a.log2_group = serve::log2_of(group_size); a.status = dev_status_dev;
  int64_t grid = (2 * n + 7) / 8;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  return out_dtype == LQ_BF16 ? serve::launch(q4::gather_kernel<true>, (unsigned)grid, q4::kThreads, 0, stream, a)
                              : serve::launch(q4::gather_kernel<false>, (unsigned)grid, q4::kThreads, 0, stream, a);
}
