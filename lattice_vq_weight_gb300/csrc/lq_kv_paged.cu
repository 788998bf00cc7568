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
// Append: a warp per (run, head, K or V).  Runs are found from the slots alone
// (a token whose predecessor is not the slot before it in the same block
// starts one), so no block list has to be built first.  The run is read twice,
// for the maximum and for the codes: at most 64 KB that the first pass has
// left in L1 or L2.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace paged {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct AppendArgs {
  const void* x[2];          // k, v
  int64_t ld[2];
  int8_t* cache[2];
  float* scales[2];
  const int64_t* slots;
  int64_t tokens, units, slots_in_cache;
  int kv_heads, dim, log2_bs, window;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 x = __ldg(f), y = __ldg(f + 1);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
}

__device__ __forceinline__ uint32_t pack4(const int (&c)[4]) {
  return (uint32_t)(c[0] & 255) | (uint32_t)(c[1] & 255) << 8 | (uint32_t)(c[2] & 255) << 16 | (uint32_t)c[3] << 24;
}

// rint of the IEEE quotient, clipped to the code range.
__device__ __forceinline__ int code_of(float x, float s) {
  const float q = rintf(__fdiv_rn(x, s));
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= a.units) return;
  const int per = 2 * a.kv_heads;
  const int64_t win = u / per;
  const int which = (int)(u - win * per) & 1, h = (int)(u - win * per) >> 1;
  const void* x = which ? a.x[1] : a.x[0];
  const int64_t ld = which ? a.ld[1] : a.ld[0];
  int8_t* cache = which ? a.cache[1] : a.cache[0];
  float* scales = which ? a.scales[1] : a.scales[0];
  const int bs1 = (1 << a.log2_bs) - 1;
  const int chunks = a.dim >> 3;                   // 8-element chunks per row

  // which tokens of the window start a run
  const int64_t t0 = win * a.window;
  int64_t mine = -1;
  bool starts = false;
  if (lane < a.window && t0 + lane < a.tokens) {
    mine = __ldg(a.slots + t0 + lane);
    const int64_t prev = t0 + lane > 0 ? __ldg(a.slots + t0 + lane - 1) : -1;
    starts = mine >= 0 && !(prev >= 0 && prev + 1 == mine && (mine & bs1) != 0);
    if (mine >= a.slots_in_cache) raise_flag(a.status, LQ_DEV_RANGE);
  }
  uint32_t todo = __ballot_sync(0xffffffffu, starts);
  while (todo) {
    const int first = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t slot = __shfl_sync(0xffffffffu, mine, first), t = t0 + first;
    const int64_t blk = slot >> a.log2_bs;
    const int off = (int)(slot & bs1);
    if (slot >= a.slots_in_cache) continue;
    // the run's length: tokens that carry on with consecutive slots of the block
    int len = 0;
    for (int c = 0; c <= bs1 - off; c += 32) {
      const int64_t i = t + c + lane;
      const bool in = c + lane <= bs1 - off && i < a.tokens && __ldg(a.slots + i) == slot + c + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      len += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      if (m != 0xffffffffu) break;
    }
    const int n = len * chunks;
    const int64_t src = t * ld + (int64_t)h * a.dim;
    const int64_t sc = blk * a.kv_heads + h;
    int8_t* rows = cache + (sc << a.log2_bs) * a.dim;
    const float s_old = off > 0 ? scales[sc] : 0.f;

    float mx = 0.f;
    bool bad = false;
    for (int c = lane; c < n; c += 32) {
      const int r = c / chunks, k = c - r * chunks;
      float v[8];
      load8<BF16>(x, src + r * ld + 8 * k, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float m = fabsf(v[e]);
        if (m <= 3.402823466e38f) mx = fmaxf(mx, m);
        else bad = true;
      }
    }
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (bad) raise_flag(a.status, LQ_DEV_NONFINITE);
    const float s = fmaxf(s_old, __fdiv_rn(mx, 127.f));

    if (s > s_old && off > 0) {
      for (int c = lane; c < off * chunks; c += 32) {
        uint2* p = reinterpret_cast<uint2*>(rows + 8 * c);
        const uint2 w = *p;
        const uint32_t in[2] = {w.x, w.y};
        uint32_t out[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          int code[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) code[e] = code_of((float)(int8_t)(in[q] >> (8 * e)) * s_old, s);
          out[q] = pack4(code);
        }
        *p = make_uint2(out[0], out[1]);
      }
    }
    const float d = s > 0.f ? s : 1.f;
    for (int c = lane; c < n; c += 32) {
      const int r = c / chunks, k = c - r * chunks;
      float v[8];
      load8<BF16>(x, src + r * ld + 8 * k, v);
      uint32_t out[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        int code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = v[4 * q + e];
          code[e] = fabsf(f) <= 3.402823466e38f ? code_of(f, d) : 0;
        }
        out[q] = pack4(code);
      }
      *reinterpret_cast<uint2*>(rows + (int64_t)(off + r) * a.dim + 8 * k) = make_uint2(out[0], out[1]);
    }
    if (lane == 0) scales[sc] = s;
  }
}

struct GatherArgs {
  const int64_t* slots;
  const int8_t* cache[2];
  const float* scales[2];
  void* out[2];
  int64_t n, chunks, slots_in_cache;     // chunks: 8-code chunks per cache
  int kv_heads, dim, log2_bs;
  int32_t* status;
};

// Eight codes per thread: out = code * scale, fp32 or rounded once to bf16.
template <bool BF16>
__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
  pdl_wait();
  pdl_launch();
  const int per_row = a.kv_heads * (a.dim >> 3);
  for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < 2 * a.chunks;
       c += (int64_t)gridDim.x * blockDim.x) {
    const int which = c >= a.chunks;
    const int64_t cc = which ? c - a.chunks : c;
    const int64_t row = cc / per_row;
    const int rest = (int)(cc - row * per_row);
    const int h = rest / (a.dim >> 3), k = rest - h * (a.dim >> 3);
    const int64_t slot = __ldg(a.slots + row);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (slot >= 0 && slot < a.slots_in_cache) {
      const int64_t sc = (slot >> a.log2_bs) * a.kv_heads + h;
      const int64_t at = ((sc << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1))) * a.dim + 8 * k;
      const float s = __ldg((which ? a.scales[1] : a.scales[0]) + sc);
      const uint2 w = __ldg(reinterpret_cast<const uint2*>((which ? a.cache[1] : a.cache[0]) + at));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)(int8_t)(w.x >> (8 * e)) * s;
        v[4 + e] = (float)(int8_t)(w.y >> (8 * e)) * s;
      }
    } else if (slot >= a.slots_in_cache) {
      raise_flag(a.status, LQ_DEV_RANGE);
    }
    void* out = which ? a.out[1] : a.out[0];
    if constexpr (BF16) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      reinterpret_cast<uint4*>(out)[cc] = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float4* f = reinterpret_cast<float4*>(out) + 2 * cc;
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
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
  // tokens that one warp looks through for runs: one while that fits one wave
  // of resident warps (decode steps: every token is a run), up to 32 for long
  // prompts, where most tokens start none
  const int64_t warps = tokens * 2 * kv_heads, wave = (int64_t)sms * 64;
  int64_t window = (warps + wave - 1) / wave;
  a.window = (int)(window > 32 ? 32 : window);
  a.units = (tokens + a.window - 1) / a.window * 2 * kv_heads;
  const int64_t grid = (a.units + paged::kWarps - 1) / paged::kWarps;
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
  a.n = n; a.chunks = n * kv_heads * (head_dim / 8); a.slots_in_cache = num_blocks * block_size;
  a.kv_heads = kv_heads; a.dim = head_dim; a.log2_bs = serve::log2_of(block_size); a.status = dev_status_dev;
  int64_t grid = (2 * a.chunks + 255) / 256;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  return out_dtype == LQ_BF16 ? serve::launch(paged::gather_kernel<true>, (unsigned)grid, 256, 0, stream, a)
                              : serve::launch(paged::gather_kernel<false>, (unsigned)grid, 256, 0, stream, a);
}
