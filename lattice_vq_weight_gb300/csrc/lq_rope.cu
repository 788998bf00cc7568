// RMS norm of every query and key head and the rotary position rotation, in
// one pass over q and k.
//
// Per token t and head: y = x * rsqrt(mean(x^2) + eps) * w (w the head's norm
// weights, shared by all heads of its kind), then the first rot dimensions are
// rotated pairwise by the token's angles, (a, b) -> (a cos - b sin, b cos + a
// sin); a pair is (i, i + rot/2), or (2i, 2i + 1) when interleaved.  Everything
// between the load and the one rounding of the result is fp32.
//
// The pass is bound by HBM for a prompt and by latency for a decode step, and
// at HBM speed an SM has few instructions for each value, so the layout saves
// those: eight dimensions per lane, chosen so that rotation partners meet in
// one lane (lane i of a head holds 4 i .. 4 i + 3 and the four dimensions
// rot/2 further; two 8-byte bf16 loads, 128 bytes per head and load) and no
// value is exchanged but the norm's sum.  A head takes the smallest
// power-of-two group of lanes that holds it (two heads of 128 per warp).  A
// warp handles IT rounds of heads of one token and one kind (query or key)
// with all their loads in flight at once, and forms the products of cosine,
// sine and weight once for all of them.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace rope {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Args {
  const void* q;
  const void* k;
  void* qo;
  void* ko;
  int64_t ldq, ldk, ldqo, ldko;
  int q_heads, kv_heads, dim, rot, interleaved;
  int64_t tokens, max_pos;
  int units_per_token, q_units;
  const float* qw;
  const float* kw;
  float eps, inv_dim;
  const int32_t* positions;
  const float* cos_sin;      // [max_pos x rot]: rot/2 cosines, then rot/2 sines
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* v) {
  if constexpr (BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  } else {
    const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, float a, float b, float c, float d) {
  if constexpr (BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(a, b, c, d);
  }
}

// G: lanes per head (a power of two, >= dim / 8); IT: rounds of 32 / G heads
// per warp; INTER: interleaved pairs.
template <bool BF16, int G, int IT, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(Args a) {
  constexpr int H = 32 / G;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1);
  const bool in_head = 8 * sub < a.dim;
  const bool rotates = 8 * sub < a.rot;
  const int half = a.rot >> 1;
  // this lane's dimensions: o0 .. o0 + 3 and o1 .. o1 + 3
  const int o0 = (!INTER && rotates) ? 4 * sub : 8 * sub;
  const int o1 = (!INTER && rotates) ? half + 4 * sub : 8 * sub + 4;
  pdl_wait();
  pdl_launch();
  const unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const unsigned t = u / (unsigned)a.units_per_token;
  if (t >= a.tokens) return;                      // whole warps only
  int unit = (int)(u - t * (unsigned)a.units_per_token);
  const bool is_q = unit < a.q_units;
  if (!is_q) unit -= a.q_units;
  const int heads = is_q ? a.q_heads : a.kv_heads;
  const int h0 = unit * (IT * H) + lane / G;
  const void* src = is_q ? a.q : a.k;
  void* dst = is_q ? a.qo : a.ko;
  const int64_t from = t * (is_q ? a.ldq : a.ldk) + (int64_t)h0 * a.dim;
  const int64_t to = t * (is_q ? a.ldqo : a.ldko) + (int64_t)h0 * a.dim;
  const int pos = __ldg(a.positions + t);

  float v[IT][8];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    if (h0 + it * H < heads && in_head) {
      load4<BF16>(src, from + it * H * a.dim + o0, v[it]);
      load4<BF16>(src, from + it * H * a.dim + o1, v[it] + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] = 0.f;
    }
  }

  // y[e] = r (c[e] v[e] + s[e] v[partner of e]): the weights ride along
  float c[8], s[8];
  const float* w = is_q ? a.qw : a.kw;
  {
    float wv[8];
    if (w != nullptr && in_head) {
      load4<false>(w, o0, wv);
      load4<false>(w, o1, wv + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) wv[e] = 1.f;
    }
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    if (!pos_ok && lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (rotates && pos_ok) {
      load4<false>(a.cos_sin, (int64_t)pos * a.rot + 4 * sub, cs);
      load4<false>(a.cos_sin, (int64_t)pos * a.rot + half + 4 * sub, sn);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = INTER ? 2 * i : i, q = INTER ? 2 * i + 1 : i + 4;
      c[p] = cs[i] * wv[p];
      c[q] = cs[i] * wv[q];
      s[p] = -sn[i] * wv[q];
      s[q] = sn[i] * wv[p];
    }
  }

#pragma unroll
  for (int it = 0; it < IT; ++it) {
    float r = 1.f;
    if (w != nullptr) {                           // the same in the whole warp
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x = fmaf(v[it][e], v[it][e], x);
#pragma unroll
      for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      r = rsqrtf(fmaf(x, a.inv_dim, a.eps));
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = INTER ? e ^ 1 : e ^ 4;
      y[e] = r * fmaf(s[e], v[it][p], c[e] * v[it][e]);
    }
    if (h0 + it * H < heads && in_head) {
      store4<BF16>(dst, to + it * H * a.dim + o0, y[0], y[1], y[2], y[3]);
      store4<BF16>(dst, to + it * H * a.dim + o1, y[4], y[5], y[6], y[7]);
    }
  }
}

template <bool BF16, int G>
lq_status launch_rope(Args& a, int sms, void* stream) {
  constexpr int H = 32 / G;
  auto units = [&](int it) { return (a.q_heads + it * H - 1) / (it * H) + (a.kv_heads + it * H - 1) / (it * H); };
  // four rounds per warp keep four heads' loads in flight; a call whose warps
  // would not fill the SMs twice takes one round per warp
  const bool wide = a.tokens * units(4) >= (int64_t)sms * 2 * kWarps;
  const int it = wide ? 4 : 1;
  a.units_per_token = units(it);
  a.q_units = (a.q_heads + it * H - 1) / (it * H);
  const int64_t grid = (a.tokens * a.units_per_token + kWarps - 1) / kWarps;
  if (grid > INT32_MAX / kWarps) return LQ_ERR_SHAPE;
  const unsigned n = (unsigned)grid;
  if (a.interleaved)
    return wide ? serve::launch(norm_rope_kernel<BF16, G, 4, true>, n, kThreads, 0, stream, a)
                : serve::launch(norm_rope_kernel<BF16, G, 1, true>, n, kThreads, 0, stream, a);
  return wide ? serve::launch(norm_rope_kernel<BF16, G, 4, false>, n, kThreads, 0, stream, a)
              : serve::launch(norm_rope_kernel<BF16, G, 1, false>, n, kThreads, 0, stream, a);
}

template <bool BF16>
lq_status launch_dim(Args& a, int sms, void* stream) {
  const int lanes = a.dim / 8;
  if (lanes <= 8) return launch_rope<BF16, 8>(a, sms, stream);
  if (lanes <= 16) return launch_rope<BF16, 16>(a, sms, stream);
  return launch_rope<BF16, 32>(a, sms, stream);
}

}  // namespace rope
}  // namespace lq

using namespace lq;

extern "C" lq_status lq_qk_norm_rope(const void* q_dev, int64_t ldq, int q_heads, const void* k_dev, int64_t ldk,
                                     int kv_heads, int dtype, int64_t tokens, int head_dim, const float* q_weight_dev,
                                     const float* k_weight_dev, float eps, const int32_t* positions_dev,
                                     const float* cos_sin_dev, int64_t max_pos, int rot_dim, int interleaved,
                                     void* q_out_dev, int64_t ldqo, void* k_out_dev, int64_t ldko,
                                     int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_qk_norm_rope");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  if (head_dim <= 0 || head_dim > 256 || head_dim % 8 != 0) return LQ_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > head_dim) return LQ_ERR_SHAPE;
  if (rot_dim % 16 != 0) return LQ_ERR_UNSUPPORTED;
  if (q_heads < 0 || kv_heads < 0 || q_heads > 1024 || kv_heads > 1024 || tokens < 0 || max_pos < 0)
    return LQ_ERR_SHAPE;
  if (!(eps >= 0.f)) return LQ_ERR_ARG;
  const int64_t esize = dtype == LQ_BF16 ? 2 : 4;
  const int64_t qc = (int64_t)q_heads * head_dim, kc = (int64_t)kv_heads * head_dim;
  if (q_heads > 0 && (ldq < qc || ldqo < qc || (ldq * esize) % 16 != 0 || (ldqo * esize) % 16 != 0)) return LQ_ERR_SHAPE;
  if (kv_heads > 0 && (ldk < kc || ldko < kc || (ldk * esize) % 16 != 0 || (ldko * esize) % 16 != 0))
    return LQ_ERR_SHAPE;
  if (tokens == 0 || q_heads + kv_heads == 0) return LQ_OK;
  if (q_heads > 0 && (q_dev == nullptr || q_out_dev == nullptr || !aligned16(q_dev) || !aligned16(q_out_dev)))
    return LQ_ERR_ARG;
  if (kv_heads > 0 && (k_dev == nullptr || k_out_dev == nullptr || !aligned16(k_dev) || !aligned16(k_out_dev)))
    return LQ_ERR_ARG;
  if (!aligned16(q_weight_dev) || !aligned16(k_weight_dev) || !aligned4(dev_status_dev)) return LQ_ERR_ARG;
  if (positions_dev == nullptr || !aligned4(positions_dev)) return LQ_ERR_ARG;
  if (rot_dim > 0 && (cos_sin_dev == nullptr || !aligned16(cos_sin_dev))) return LQ_ERR_ARG;
  rope::Args a;
  a.q = q_dev; a.k = k_dev; a.qo = q_out_dev; a.ko = k_out_dev;
  a.ldq = ldq; a.ldk = ldk; a.ldqo = ldqo; a.ldko = ldko;
  a.q_heads = q_heads; a.kv_heads = kv_heads; a.dim = head_dim; a.rot = rot_dim; a.interleaved = interleaved != 0;
  a.tokens = tokens; a.max_pos = max_pos;
  a.qw = q_weight_dev; a.kw = k_weight_dev; a.eps = eps; a.inv_dim = 1.0f / (float)head_dim;
  a.positions = positions_dev; a.cos_sin = cos_sin_dev; a.status = dev_status_dev;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  return dtype == LQ_BF16 ? rope::launch_dim<true>(a, sms, stream) : rope::launch_dim<false>(a, sms, stream);
}
