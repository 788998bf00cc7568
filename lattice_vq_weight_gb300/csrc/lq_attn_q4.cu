// Attention of a ragged batch of query tokens over the paged 4-bit KV cache
// (the format: lq_q4.cuh).
//
// Request i has q_len_i = cu_q[i+1] - cu_q[i] query tokens, the last of its
// kv_len_i tokens, so query token j sees positions <= kv_len_i - q_len_i + j:
//     out[t, h] = sum_p w_p v_p,  w = softmax over visible p of sm_scale * q[t, h] . k_p,
// k_p and v_p of kv head h / (q_heads / kv_heads).  A query token that sees
// nothing gets zeros.
//
// One warp per query token and head: 32 tokens at a time, a score per lane in
// fp32, running maximum and sum, then the values token by token, D / 32
// dimensions per lane.
#include "lq_attn_paged.cuh"
#include "lq_q4.cuh"

namespace lq {
namespace q4 {

struct AttnArgs {
  attn::Args a;
  const uint32_t* kc;
  const uint32_t* vc;
  const uint32_t* ks;
  const uint32_t* vs;
  int log2_group, dim;
};

template <int D, bool F32>
__global__ void __launch_bounds__(128) attn_rows_kernel(const __grid_constant__ AttnArgs qa) {
  using namespace attn;
  constexpr int E = D / 32;
  const Args& a = qa.a;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, bs1 = (1 << a.log2_bs) - 1, groups = D >> qa.log2_group;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.batch; i += blockDim.x)
      if ((int64_t)a.kv_lens[i] > ((int64_t)a.width << a.log2_bs)) raise_flag(a.status, LQ_DEV_RANGE);
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= a.total_q * a.q_heads) return;
  const int t = (int)(item / a.q_heads), head = (int)(item % a.q_heads), h = head / a.group;
  // the request that owns the token
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  while (lo + 1 < a.batch && a.cu_q[lo + 1] <= t) ++lo;
  const Request r = load_request(a, lo);
  int past = 0;
  if (t >= r.q0 && t < r.q0 + r.q_len) past = min(r.shown + (t - r.q0) + 1, r.len);
  const int32_t* table = a.table + lo * a.ldt;
  const int64_t at_q = (int64_t)t * a.ldq + (int64_t)head * D, at_out = (int64_t)t * a.ldo + (int64_t)head * D;
  float mx = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int t0 = 0; t0 < past; t0 += 32) {
    const int p = t0 + lane, blk = p < past ? table[p >> a.log2_bs] : -1;
    const bool ok = (unsigned)blk < (unsigned long long)a.num_blocks;
    if (p < past && !ok) raise_flag(a.status, LQ_DEV_RANGE);
    const int64_t row = ((((int64_t)blk * a.kv_heads + h) << a.log2_bs) + (p & bs1));
    float x = -INFINITY;
    if (ok) {
      float sum = 0.f;
      for (int c = 0; c < D; c += 8) {
        float v[8];
        values8(qa.kc[row * (D / 8) + c / 8], qa.ks[row * groups + (c >> qa.log2_group)], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float q;
          if constexpr (F32) q = reinterpret_cast<const float*>(a.q)[at_q + c + e];
          else q = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.q)[at_q + c + e] << 16);
          sum = fmaf(q, v[e], sum);
        }
      }
      x = sum * a.scale_log2;
    }
    float top = x;
    for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float to = fmaxf(mx, top), f = mx == -INFINITY ? 0.f : ex2(mx - to);
    const float w = ok ? ex2(x - to) : 0.f;
    mx = to;
    float sum = w;
    for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    l = fmaf(l, f, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    const uint32_t there = __ballot_sync(0xffffffffu, ok);
    for (int i = 0; i < 32; ++i) {
      const int64_t from = __shfl_sync(0xffffffffu, row, i);
      const float wt = __shfl_sync(0xffffffffu, w, i);
      if (there >> i & 1) {
        float v[8];
        const int c = lane * E;
        values8(qa.vc[from * (D / 8) + c / 8], qa.vs[from * groups + (c >> qa.log2_group)], v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float x8 = v[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) x8 = (c & 7) + e == k ? v[k] : x8;
          o[e] = fmaf(wt, x8, o[e]);
        }
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (F32) reinterpret_cast<float*>(a.out)[at_out + lane * E + e] = o[e] * inv;
    else reinterpret_cast<__nv_bfloat16*>(a.out)[at_out + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
  }
}

template <int D>
lq_status launch_rows(const AttnArgs& qa, bool f32, void* stream) {
  const int64_t grid = (qa.a.total_q * qa.a.q_heads + 3) / 4;
  return f32 ? serve::launch(attn_rows_kernel<D, true>, (unsigned)grid, 128, 0, stream, qa)
             : serve::launch(attn_rows_kernel<D, false>, (unsigned)grid, 128, 0, stream, qa);
}

}  // namespace q4
}  // namespace lq

using namespace lq;

extern "C" size_t lq_attention_paged_q4_workspace_size(int batch, int64_t total_q, int q_heads, int kv_heads,
                                                       int head_dim) {
  return lq_attention_paged_workspace_size(batch, total_q, q_heads, kv_heads, head_dim);
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
  q4::AttnArgs qa;
  attn::Args& a = qa.a;
  a = attn::Args{};
  a.q = q_dev; a.ldq = ldq; a.total_q = total_q; a.cu_q = cu_q_dev; a.kv_lens = kv_lens_dev; a.batch = batch;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width; a.num_blocks = num_blocks;
  a.log2_bs = serve::log2_of(block_size); a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads;
  a.scale_log2 = sm_scale * 1.4426950408889634f; a.out = out_dev; a.ldo = ldo; a.status = dev_status_dev;
  qa.kc = reinterpret_cast<const uint32_t*>(k_cache_dev); qa.vc = reinterpret_cast<const uint32_t*>(v_cache_dev);
  qa.ks = reinterpret_cast<const uint32_t*>(k_scales_dev); qa.vs = reinterpret_cast<const uint32_t*>(v_scales_dev);
  qa.log2_group = serve::log2_of(group_size); qa.dim = head_dim;
  const bool f32 = dtype == LQ_F32;
  switch (head_dim) {
    case 64: return q4::launch_rows<64>(qa, f32, stream);
    case 128: return q4::launch_rows<128>(qa, f32, stream);
    default: return q4::launch_rows<256>(qa, f32, stream);
  }
}
