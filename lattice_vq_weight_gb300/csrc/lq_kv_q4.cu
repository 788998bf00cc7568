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
  int kv_heads, dim, log2_bs, log2_group;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// A warp per token and cache, eight values per lane and step: a lane's codes are
// one word, a group G / 8 neighbouring lanes.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int words = a.dim / 8, per_row = a.kv_heads * words, span = 1 << (a.log2_group - 3);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < 2 * a.tokens; u += warps) {
    const int64_t t = u >> 1, slot = a.slots[t];
    const int which = (int)(u & 1);
    if (slot < 0) continue;
    if (slot >= a.slots_in_cache) {
      if (lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
      continue;
    }
    const int64_t first = ((slot >> a.log2_bs) * a.kv_heads << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1));
    for (int c0 = 0; c0 < per_row; c0 += 32) {
      const int c = c0 + lane;
      const bool in = c < per_row;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      if (in) load8<BF16>(a.x[which], t * a.ld[which] + 8 * c, v);
      float low = INFINITY, high = -INFINITY;
      bool odd = false, far = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!(fabsf(v[e]) <= kMost)) {
          if (fabsf(v[e]) < INFINITY) {
            far = true;
            v[e] = copysignf(kMost, v[e]);
          } else {
            odd = true;
            v[e] = 0.f;
          }
        }
        low = fminf(low, v[e]);
        high = fmaxf(high, v[e]);
      }
      if (odd) raise_flag(a.status, LQ_DEV_NONFINITE);
      if (far) raise_flag(a.status, LQ_DEV_RANGE);
      for (int o = 1; o < span; o <<= 1) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
      }
      const __half s = __float2half_rn(__fdiv_rn(__fsub_rn(high, low), 15.f));
      const float sf = __half2float(s);
      const __half b = __float2half_rn(__fsub_rn(low, 16.f * sf));
      const float bf = __half2float(b), r = sf > 0.f ? __frcp_rn(sf) : 0.f;
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = rintf(__fmul_rn(__fsub_rn(v[e], bf), r)) - 16.f;
        word |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * e);
      }
      if (in) {
        const int h = c / words, w = c - h * words;
        const int64_t row = first + ((int64_t)h << a.log2_bs);
        a.codes[which][row * words + w] = word;
        if ((w & (span - 1)) == 0)
          a.scales[which][row * (words / span) + w / span] =
              (uint32_t)__half_as_ushort(s) | (uint32_t)__half_as_ushort(b) << 16;
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
  int kv_heads, dim, log2_bs, log2_group;
  int32_t* status;
};

// A warp per slot and cache, a word of codes per lane and step.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) gather_kernel(GatherArgs a) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int words = a.dim / 8, per_row = a.kv_heads * words, span = 1 << (a.log2_group - 3);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < 2 * a.n; u += warps) {
    const int64_t slot = a.slots[u >> 1];
    const int which = (int)(u & 1);
    const bool ok = slot >= 0 && slot < a.slots_in_cache;
    if (slot >= a.slots_in_cache && lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
    const int64_t first = ((slot >> a.log2_bs) * a.kv_heads << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1));
    for (int c = lane; c < per_row; c += 32) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      if (ok) {
        const int h = c / words, w = c - h * words;
        const int64_t row = first + ((int64_t)h << a.log2_bs);
        values8(a.codes[which][row * words + w], a.scales[which][row * (words / span) + w / span], v);
      }
      const int64_t at = (u >> 1) * per_row + c;
      if constexpr (BF16) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&p);
        }
        reinterpret_cast<uint4*>(a.out[which])[at] = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float4* out = reinterpret_cast<float4*>(a.out[which]) + 2 * at;
        out[0] = make_float4(v[0], v[1], v[2], v[3]);
        out[1] = make_float4(v[4], v[5], v[6], v[7]);
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
  a.kv_heads = kv_heads; a.dim = head_dim; a.log2_bs = serve::log2_of(block_size);
  a.log2_group = serve::log2_of(group_size); a.status = dev_status_dev;
  int64_t grid = (2 * tokens + 7) / 8;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  return dtype == LQ_BF16 ? serve::launch(q4::append_kernel<true>, (unsigned)grid, q4::kThreads, 0, stream, a)
                          : serve::launch(q4::append_kernel<false>, (unsigned)grid, q4::kThreads, 0, stream, a);
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
  a.kv_heads = kv_heads; a.dim = head_dim; a.log2_bs = serve::log2_of(block_size);
  a.log2_group = serve::log2_of(group_size); a.status = dev_status_dev;
  int64_t grid = (2 * n + 7) / 8;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  return out_dtype == LQ_BF16 ? serve::launch(q4::gather_kernel<true>, (unsigned)grid, q4::kThreads, 0, stream, a)
                              : serve::launch(q4::gather_kernel<false>, (unsigned)grid, q4::kThreads, 0, stream, a);
}
