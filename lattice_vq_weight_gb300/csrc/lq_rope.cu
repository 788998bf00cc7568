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
// power-of-two group of lanes that holds it (two heads of 128 per warp).  A unit is IT
// rounds of heads of one token and one kind (query or key), whose loads are in
// flight at once and which share the products of cosine, sine and weight.  A
// warp goes from unit to unit with the next one's values, the angles of the
// next one's position and the position after that under way: one unit per warp
// measured 81 us for a prompt of 8191 tokens and 72 heads of 128 (now 59), most of
// it the latency of position, angles and values one after the other.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <type_traits>

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

// Four values as loaded.
template <bool BF16>
struct Four {
  uint32_t w[BF16 ? 2 : 4];
};
template <bool BF16>
__device__ __forceinline__ Four<BF16> fetch4(const void* p, int64_t i) {
  Four<BF16> f;
  if constexpr (BF16) {
    const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
    f.w[0] = x.x; f.w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + i);
    f.w[0] = x.x; f.w[1] = x.y; f.w[2] = x.z; f.w[3] = x.w;
  }
  return f;
}
// Values 2 i and 2 i + 1 of it.
template <bool BF16>
__device__ __forceinline__ float2 pair_of(const Four<BF16>& f, int i) {
  if constexpr (BF16) return make_float2(__uint_as_float(f.w[i] << 16), __uint_as_float(f.w[i] & 0xFFFF0000u));
  else return make_float2(__uint_as_float(f.w[2 * i]), __uint_as_float(f.w[2 * i + 1]));
}

// A unit of work: token, kind, first head of this lane's group.
struct Unit {
  unsigned t;
  int h0, heads;
  bool is_q;
};

// The heads of a unit whose position is outside the table: normed, not turned.
// (On its own and after the others, so that the usual units pay nothing for it.)
template <bool BF16, int G, int IT>
__device__ __noinline__ void norm_only(const Args& a, const Unit& u) {
  constexpr int H = 32 / G;
  const int sub = threadIdx.x & (G - 1);
  const float* w = u.is_q ? a.qw : a.kw;
  const void* src = u.is_q ? a.q : a.k;
  void* dst = u.is_q ? a.qo : a.ko;
  const int64_t from = u.t * (u.is_q ? a.ldq : a.ldk) + (int64_t)u.h0 * a.dim + 8 * sub;
  const int64_t to = u.t * (u.is_q ? a.ldqo : a.ldko) + (int64_t)u.h0 * a.dim + 8 * sub;
#pragma unroll 1
  for (int it = 0; it < IT; ++it) {
    const bool here = u.h0 + it * H < u.heads && 8 * sub < a.dim;
    float x[8] = {}, wv[8], q = 0.f;
    if (here) {
      load4<BF16>(src, from + it * H * a.dim, x);
      load4<BF16>(src, from + it * H * a.dim + 4, x + 4);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q = fmaf(x[e], x[e], q);
      wv[e] = w != nullptr && here ? w[8 * sub + e] : 1.f;
    }
#pragma unroll
    for (int o = G / 2; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    const float r = w != nullptr ? rsqrtf(fmaf(q, a.inv_dim, a.eps)) : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r * (wv[e] * x[e]);
    if (here) {
      store4<BF16>(dst, to + it * H * a.dim, x[0], x[1], x[2], x[3]);
      store4<BF16>(dst, to + it * H * a.dim + 4, x[4], x[5], x[6], x[7]);
    }
  }
}

// G: lanes per head (a power of two, >= dim / 8); IT: rounds of 32 / G heads
// per unit; INTER: interleaved pairs; PART: only the first dimensions are turned.
template <bool BF16, int G, int IT, bool INTER, bool PART>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(Args a) {
  constexpr int H = 32 / G;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1);
  const bool in_head = 8 * sub < a.dim;
  const bool rotates = PART ? 8 * sub < a.rot : in_head;
  const int half = a.rot >> 1;
  // this lane's dimensions: o0 .. o0 + 3 and o1 .. o1 + 3
  const int o0 = (!INTER && rotates) ? 4 * sub : 8 * sub;
  const int o1 = (!INTER && rotates) ? half + 4 * sub : 8 * sub + 4;
  const unsigned units = (unsigned)a.units, warps = gridDim.x * kWarps;
  auto unit_of = [&](unsigned u) {
    Unit x;
    x.t = u / (unsigned)a.units_per_token;
    int i = (int)(u - x.t * (unsigned)a.units_per_token);
    x.is_q = i < a.q_units;
    if (!x.is_q) i -= a.q_units;
    x.heads = x.is_q ? a.q_heads : a.kv_heads;
    x.h0 = i * (IT * H) + lane / G;
    return x;
  };
  auto fetch = [&](const Unit& x, Four<BF16> (&v)[IT][2]) {
    const void* src = x.is_q ? a.q : a.k;
    const int64_t from = x.t * (x.is_q ? a.ldq : a.ldk) + (int64_t)x.h0 * a.dim;
#pragma unroll
    for (int it = 0; it < IT; ++it)
      if (x.h0 + it * H < x.heads && in_head) {
        v[it][0] = fetch4<BF16>(src, from + it * H * a.dim + o0);
        v[it][1] = fetch4<BF16>(src, from + it * H * a.dim + o1);
      }
  };
  auto angles = [&](int pos, float (&cs)[4], float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
    if (rotates && pos >= 0 && pos < a.max_pos) {
      load4<false>(a.cos_sin, (int64_t)pos * a.rot + 4 * sub, cs);
      load4<false>(a.cos_sin, (int64_t)pos * a.rot + half + 4 * sub, sn);
    }
  };
  pdl_wait();
  pdl_launch();

  unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= units) return;                         // whole warps only
  Unit now = unit_of(u), next = unit_of(min(u + warps, units - 1));
  Four<BF16> v[IT][2], vn[IT][2];
  float cs[4], sn[4], csn[4], snn[4];
  bool outside = false;                           // a position was
  int pos = a.positions[now.t], pos_next = a.positions[next.t];
  fetch(now, v);
  angles(pos, cs, sn);
  for (;;) {
    const bool more = u + warps < units;
    Unit after = next;
    int pos_after = pos_next;
    if (more) {
      fetch(next, vn);
      angles(pos_next, csn, snn);
      after = unit_of(min(u + 2 * warps, units - 1));
      pos_after = a.positions[after.t];
    }

    // y[e] = r (c[e] v[e] + s[e] v[partner of e]): the weights ride along
    float2 c[4], s[4];
    const float* w = now.is_q ? a.qw : a.kw;
    {
      float wv[8];
      if (w != nullptr && in_head) {
        load4<false>(w, o0, wv);
        load4<false>(w, o1, wv + 4);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = 1.f;
      }
      float cc[8], ss[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = INTER ? 2 * i : i, q = INTER ? 2 * i + 1 : i + 4;
        cc[p] = cs[i] * wv[p];
        cc[q] = cs[i] * wv[q];
        ss[p] = -sn[i] * wv[q];
        ss[q] = sn[i] * wv[p];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[e] = make_float2(cc[2 * e], cc[2 * e + 1]);
        s[e] = make_float2(ss[2 * e], ss[2 * e + 1]);
      }
    }
    if (!(pos >= 0 && pos < a.max_pos)) {           // left to the pass below
      now.heads = 0;
      outside = true;
    }
    void* dst = now.is_q ? a.qo : a.ko;
    const int64_t to = now.t * (now.is_q ? a.ldqo : a.ldko) + (int64_t)now.h0 * a.dim;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const bool here = now.h0 + it * H < now.heads && in_head;
      float2 x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = here ? pair_of<BF16>(v[it][e >> 1], e & 1) : make_float2(0.f, 0.f);
      float r = 1.f;
      if (w != nullptr) {                         // the same in the whole warp
        float2 q = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) q = fma2(x[e], x[e], q);
        float z = q.x + q.y;
#pragma unroll
        for (int o = G / 2; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        r = rsqrtf(fmaf(z, a.inv_dim, a.eps));
      }
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = INTER ? make_float2(x[e].y, x[e].x) : x[e ^ 2], cx = mul2(c[e], x[e]);
        // (a value that is not turned has no partner: 0 times an infinite one would be NaN)
        y[e] = mul2(r2, !PART || rotates ? fma2(s[e], p, cx) : cx);
      }
      if (here) {
        store4<BF16>(dst, to + it * H * a.dim + o0, y[0].x, y[0].y, y[1].x, y[1].y);
        store4<BF16>(dst, to + it * H * a.dim + o1, y[2].x, y[2].y, y[3].x, y[3].y);
      }
    }
    if (!more) break;
    u += warps;
    now = next;
    next = after;
    pos = pos_next;
    pos_next = pos_after;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      v[it][0] = vn[it][0];
      v[it][1] = vn[it][1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) { cs[i] = csn[i]; sn[i] = snn[i]; }
  }
  if (outside) {
    if (lane == 0) raise_flag(a.status, LQ_DEV_RANGE);
#pragma unroll 1
    for (u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += warps) {
      const Unit x = unit_of(u);
      const int p = a.positions[x.t];
      if (!(p >= 0 && p < a.max_pos)) norm_only<BF16, G, IT>(a, x);
    }
  }
}

template <bool BF16, int G>
lq_status launch_rope(Args& a, int sms, void* stream) {
  constexpr int H = 32 / G;
  auto units = [&](int it) { return (a.q_heads + it * H - 1) / (it * H) + (a.kv_heads + it * H - 1) / (it * H); };
  // four rounds per unit (two for fp32, whose values take twice the registers);
  // one where that would leave SMs without a unit per warp
  constexpr int kMost = BF16 ? 4 : 2;
  const int it = a.tokens * units(kMost) >= (int64_t)sms * kWarps ? kMost : 1;
  a.units_per_token = units(it);
  a.q_units = (a.q_heads + it * H - 1) / (it * H);
  a.units = a.tokens * a.units_per_token;
  if (a.units > INT32_MAX / 2) return LQ_ERR_SHAPE;
  int64_t grid = (a.units + kWarps - 1) / kWarps;
  if (grid > (int64_t)sms * 3) grid = (int64_t)sms * 3;
  const unsigned n = (unsigned)grid;
  auto go = [&](auto inter, auto part) {
    constexpr bool I = decltype(inter)::value, P = decltype(part)::value;
    if (it == 1) return serve::launch(norm_rope_kernel<BF16, G, 1, I, P>, n, kThreads, 0, stream, a);
    return serve::launch(norm_rope_kernel<BF16, G, kMost, I, P>, n, kThreads, 0, stream, a);
  };
  const std::true_type yes;
  const std::false_type no;
  if (a.rot < a.dim) return a.interleaved ? go(yes, yes) : go(no, yes);
  return a.interleaved ? go(yes, no) : go(no, no);
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
  if (q_heads > 0 && (ldq < qc || ldqo < qc || (ldq * esize) % 16 != 0 || (ldqo * esize) % 16 != 0))
    return LQ_ERR_SHAPE;
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
