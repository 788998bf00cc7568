// Attention of a ragged batch of query tokens over the paged 8-bit KV cache.
//
// Request i has q_len_i = cu_q[i+1] - cu_q[i] query tokens, the last of its
// kv_len_i tokens, so query token j sees positions <= kv_len_i - q_len_i + j:
//     out[t, h] = sum_p w_p v_p,  w = softmax over visible p of
//                 sm_scale * q[t, h] . k_p,   k_p = s_k[block, g] c_k, v_p = s_v[block, g] c_v,
// g = h / (q_heads / kv_heads).  A query token that sees nothing gets zeros.
//
// This is the plain form on the GPU: a warp per (query token, head), one
// position at a time, running maximum and sum in fp32.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cmath>
#include <cuda_bf16.h>

namespace lq {
namespace attn {

constexpr int kThreads = 128;

struct Args {
  const void* q;
  int64_t ldq;
  int64_t total_q;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int batch;
  const int32_t* table;
  int64_t ldt;
  int width;
  const int8_t* kc;
  const float* ks;
  const int8_t* vc;
  const float* vs;
  int64_t num_blocks;
  int log2_bs, q_heads, kv_heads, group;
  float scale;
  void* out;
  int64_t ldo;
  int32_t* status;
};

// E: dimensions per lane (head_dim / 32).
template <bool BF16, int E>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(Args a) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = u / a.q_heads;
  const int h = (int)(u - t * a.q_heads), g = h / a.group;
  if (t >= a.total_q) return;
  constexpr int D = 32 * E;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_q + mid) <= t) lo = mid; else hi = mid;
  }
  const int q0 = __ldg(a.cu_q + lo), q1 = __ldg(a.cu_q + lo + 1), len = __ldg(a.kv_lens + lo);
  int64_t see = (int64_t)len - q1 + t + 1;            // visible positions
  const int64_t most = (int64_t)a.width << a.log2_bs;
  if (t < q0 || t >= q1) see = 0;
  if (see > most) {
    if (lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
    see = most;
  }
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t i = t * a.ldq + (int64_t)h * D + lane + 32 * e;
    q[e] = a.scale * (BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[i])
                           : reinterpret_cast<const float*>(a.q)[i]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t p = 0; p < see; ++p) {
    const int32_t blk = __ldg(a.table + lo * a.ldt + (p >> a.log2_bs));
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
      continue;
    }
    const int64_t sc = (int64_t)blk * a.kv_heads + g;
    const int64_t at = ((sc << a.log2_bs) + (p & ((1 << a.log2_bs) - 1))) * D + lane;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], (float)__ldg(a.kc + at + 32 * e), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= __ldg(a.ks + sc);
    const float mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * f + w;
    const float wv = w * __ldg(a.vs + sc);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(wv, (float)__ldg(a.vc + at + 32 * e), acc[e] * f);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t i = t * a.ldo + (int64_t)h * D + lane + 32 * e;
    const float y = l == 0.f ? 0.f : acc[e] / l;      // NaN stays NaN
    if (BF16) reinterpret_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(y);
    else reinterpret_cast<float*>(a.out)[i] = y;
  }
}

template <bool BF16>
lq_status launch_rows(const Args& a, int head_dim, void* stream) {
  const int64_t grid = (a.total_q * a.q_heads + 3) / 4;
  if (grid > INT32_MAX) return LQ_ERR_SHAPE;
  switch (head_dim) {
    case 64: return serve::launch(attn_rows_kernel<BF16, 2>, (unsigned)grid, kThreads, 0, stream, a);
    case 128: return serve::launch(attn_rows_kernel<BF16, 4>, (unsigned)grid, kThreads, 0, stream, a);
    default: return serve::launch(attn_rows_kernel<BF16, 8>, (unsigned)grid, kThreads, 0, stream, a);
  }
}

}  // namespace attn
}  // namespace lq

using namespace lq;

extern "C" size_t lq_attention_paged_workspace_size(int batch, int64_t total_q, int q_heads, int kv_heads,
                                                    int head_dim) {
  if (batch < 0 || batch > LQ_MAX_REQUESTS || total_q < 0 || kv_heads <= 0 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return 256;
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
  attn::Args a;
  a.q = q_dev; a.ldq = ldq; a.total_q = total_q; a.cu_q = cu_q_dev; a.kv_lens = kv_lens_dev; a.batch = batch;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width;
  a.kc = k_cache_dev; a.ks = k_scales_dev; a.vc = v_cache_dev; a.vs = v_scales_dev; a.num_blocks = num_blocks;
  a.log2_bs = serve::log2_of(block_size); a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads;
  a.scale = sm_scale; a.out = out_dev; a.ldo = ldo; a.status = dev_status_dev;
  return dtype == LQ_BF16 ? attn::launch_rows<true>(a, head_dim, stream)
                          : attn::launch_rows<false>(a, head_dim, stream);
}
