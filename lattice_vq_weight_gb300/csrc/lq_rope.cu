// RMS norm of every query and key head and the rotary position rotation, in
// one pass over q and k.
//
// Per token t and head: y = x * rsqrt(mean(x^2) + eps) * w (w the head's norm
// weights, shared by all heads of its kind), then the first rot dimensions are
// rotated pairwise by the token's angles, (a, b) -> (a cos - b sin, b cos + a
// sin); a pair is (i, i + rot/2), or (2i, 2i + 1) when interleaved.  Everything
// between the load and the one rounding of the result is fp32.
//
// The pass is bound by HBM for a prompt and by latency for a decode step, so
// the layout is chosen for wide loads and few dependent steps: eight
// consecutive dimensions per lane (one 16-byte bf16 load), a head in the
// smallest power-of-two group of lanes that holds it (two heads of 128 per
// warp), the norm by shuffles within the group, and the rotation partner
// rot/2 dimensions away by shuffles too -- no shared memory, no barrier.  A
// warp takes IT x 32/group heads of one token with all their loads in flight
// at once, so a lane's cos and sin values are loaded once for IT heads.
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
  int64_t tokens, units, max_pos;
  int units_per_token;
  const float* qw;
  const float* kw;
  float eps, inv_dim;
  const int32_t* positions;
  const float* cos_sin;      // [max_pos x rot]: rot/2 cosines, then rot/2 sines
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
    const float4 x = f[0], y = f[1];
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      u[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// G: lanes per head (a power of two, >= dim / 8); IT: rounds of 32 / G heads
// per warp.
template <bool BF16, int G, int IT>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(Args a) {
  constexpr int H = 32 / G;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1);
  const bool in_head = 8 * sub < a.dim;
  const bool rotates = 8 * sub < a.rot;
  const int half = a.rot >> 1;
  pdl_wait();
  pdl_launch();
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= a.units) return;                       // whole warps only
  const int64_t t = u / a.units_per_token;
  const int h0 = (int)(u - t * a.units_per_token) * (IT * H) + lane / G;
  const int heads = a.q_heads + a.kv_heads;

  float v[IT][8];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int h = h0 + it * H;
    if (h < heads && in_head) {
      if (h < a.q_heads) load8<BF16>(a.q, t * a.ldq + (int64_t)h * a.dim + 8 * sub, v[it]);
      else load8<BF16>(a.k, t * a.ldk + (int64_t)(h - a.q_heads) * a.dim + 8 * sub, v[it]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] = 0.f;
    }
  }

  // this lane's angles: element e of the lane belongs to pair i(e), as its
  // first member (sign of sin -) or its second (+)
  float cs[8], sn[8];
  const int pos = __ldg(a.positions + t);
  const bool pos_ok = pos >= 0 && pos < a.max_pos;
  if (!pos_ok && lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
  if (rotates && pos_ok) {
    const float* row = a.cos_sin + (int64_t)pos * a.rot;
    if (a.interleaved) {
      const float4 c = *reinterpret_cast<const float4*>(row + 4 * sub);
      const float4 s = *reinterpret_cast<const float4*>(row + half + 4 * sub);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = cc[e >> 1];
        sn[e] = (e & 1) ? ss[e >> 1] : -ss[e >> 1];
      }
    } else {
      const bool second = 8 * sub >= half;
      const int i0 = 8 * sub - (second ? half : 0);
      load8<false>(row, i0, cs);
      load8<false>(row, half + i0, sn);
#pragma unroll
      for (int e = 0; e < 8; ++e) sn[e] = second ? sn[e] : -sn[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) { cs[e] = 1.f; sn[e] = 0.f; }
  }
  // the lane holding the partner dimensions (half style)
  int partner = lane;
  if (!a.interleaved && rotates) partner = (8 * sub >= half) ? lane - (half >> 3) : lane + (half >> 3);

#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int h = h0 + it * H;
    const bool is_q = h < a.q_heads, ok = h < heads && in_head;
    const float* w = is_q ? a.qw : a.kw;
    // the sum in every lane, also where this kind of head is not normed: a
    // warp may hold both kinds, and its shuffles are not to diverge
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[it][e], v[it][e], s);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (w != nullptr && ok) {
      const float r = rsqrtf(fmaf(s, a.inv_dim, a.eps));
      float wv[8];
      load8<false>(w, 8 * sub, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[it][e] = v[it][e] * r * wv[e];
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float far = __shfl_sync(0xffffffffu, v[it][e], partner);
      const float other = a.interleaved ? v[it][e ^ 1] : far;
      y[e] = rotates ? fmaf(other, sn[e], v[it][e] * cs[e]) : v[it][e];
    }
    if (ok) {
      if (is_q) store8<BF16>(a.qo, t * a.ldqo + (int64_t)h * a.dim + 8 * sub, y);
      else store8<BF16>(a.ko, t * a.ldko + (int64_t)(h - a.q_heads) * a.dim + 8 * sub, y);
    }
  }
}

template <bool BF16, int G>
lq_status launch_rope(Args& a, int sms, void* stream) {
  constexpr int H = 32 / G;
  const int heads = a.q_heads + a.kv_heads;
  // four rounds per warp keep four loads per lane in flight; a call whose
  // warps would not fill the SMs twice takes one round per warp
  const bool wide = a.tokens * ((heads + 4 * H - 1) / (4 * H)) >= (int64_t)sms * 2 * kWarps;
  const int it = wide ? 4 : 1;
  a.units_per_token = (heads + it * H - 1) / (it * H);
  a.units = a.tokens * a.units_per_token;
  const int64_t grid = (a.units + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return LQ_ERR_SHAPE;
  return wide ? serve::launch(norm_rope_kernel<BF16, G, 4>, (unsigned)grid, kThreads, 0, stream, a)
              : serve::launch(norm_rope_kernel<BF16, G, 1>, (unsigned)grid, kThreads, 0, stream, a);
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
