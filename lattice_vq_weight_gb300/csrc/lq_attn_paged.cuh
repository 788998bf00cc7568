// Shared by the kernels of the paged attention: the split kernel for few query
// rows (lq_attn_paged.cu) and the one for many (lq_attn_paged_tiles.cu).  Internal
// to the library.
#pragma once

#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lq_device.cuh"
#include "lq_host.h"
#include "lq_serve.cuh"
#include "lq_tma.cuh"

namespace lq {
namespace attn {

// What a piece of a row tile belongs to: request (its first query token and
// how many it has), row tile, kv head, and whether the piece begins or ends the
// tile's tokens.  valid: 0 no piece, 1 in its warp's ring, 2 in global memory.
struct Tag {
  int i, rt, h, q0, q_len;
  int valid, starts, ends;
};

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
  const int8_t* vc;
  const float* ks;
  const float* vs;
  int64_t num_blocks;
  int log2_bs, q_heads, kv_heads, group;
  float scale_log2;          // sm_scale * log2(e)
  void* out;
  int64_t ldo;
  float* part;               // partial results of the CTAs
  Tag* meta;                 // and what they belong to, two for each CTA
  int32_t* status;
};

constexpr long long kWaitCycles = 2000000000ll;   // about one second
// Where value scales may be far apart (the kernel for many rows; rows_apart of the
// split kernel) a row carries two exponents, both whole numbers: `mx`, the values'
// (its weights are 2^(x - mx + kShift), x the exponent that holds the value scale),
// and `un`, the unit of its sum of weights 2^un, near the largest score.  Their
// difference is about the log2 of the value scales that matter, whatever those
// are, so neither sum can leave fp32's range.  A weight goes into the sum as
// weight / value scale times one factor per row, 2^(mx - kShift - un) (`unit_of`).

// 2^k of a whole number, subnormal ones too; 0 where that is too small and for NaN.
__device__ __forceinline__ float pow2(float k) {
  const int e = (int)fminf(fmaxf(k, -150.f), 127.f);
  return __int_as_float(e >= -126 ? (e + 127) << 23 : (1 << 23) >> (-126 - e));
}

// Softmax weights are held times 2^8 relative to the running maximum, and the
// maximum may be behind by up to 2^7: the largest is then 2^15, in fp16's
// range, and weights down to 2^-22 of the maximum are normal numbers.
constexpr float kShift = 8.f;
constexpr float kLead = 7.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a value scale: -inf of 0, subnormal scales too.
__device__ __forceinline__ float log2_scale(float v) {
  return v < 7.88860905e-31f ? lg2(v * 18446744073709551616.f) - 64.f : lg2(v);       // 2^-100, 2^64
}

// The factor of a row's weights over value scales in its sum.
__device__ __forceinline__ float unit_of(float mx, float un) { return pow2(mx - kShift - un); }

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What pack_f16 left out, again as fp16: the two together carry 22 bits.
__device__ __forceinline__ uint32_t rest_f16(uint32_t packed, float lo, float hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_f16(lo - f.x, hi - f.y);
}

// Two codes, offset to unsigned bytes (code + 128) and placed by `sel`, as
// fp16 numbers: 0x6400 + byte is 1024 + byte, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t bytes, uint32_t sel) {
  const uint32_t h = __byte_perm(bytes, 0x64646464u, sel);
  const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Floats of the workspace per SM: of the split kernel's CTA two pieces and one for
// each of up to 16 warps, of up to 16 rows with their maxima, sums and units.  What
// the kernel for many rows leaves is less (one piece per CTA, at most a CTA per SM
// when there are any).
constexpr int work_floats(int head_dim) { return (2 + 16) * 16 * (head_dim + 3); }

// One request's share of the work: query rows (token j, head of the group)
// numbered j * group + head for each kv head.
struct Request {
  int q0, q_len, len;        // len: cached tokens, cut at the block table's end
  int shown;                 // position that query token 0 sees last
};

__device__ __forceinline__ Request load_request(const Args& a, int i) {
  Request r;
  const int q0 = a.cu_q[i], q1 = a.cu_q[i + 1], len = a.kv_lens[i];
  r.q0 = q0 < 0 ? 0 : q0;
  const int64_t end = q1 < a.total_q ? q1 : a.total_q;
  r.q_len = end > r.q0 ? (int)(end - r.q0) : 0;
  r.shown = (len > 0 ? len : 0) - r.q_len;
  const int64_t most = (int64_t)a.width << a.log2_bs;
  r.len = len < 0 ? 0 : (len < most ? len : (int)most);
  return r;
}

// Tensor map of a cache's codes as lines of 128 bytes, copied in boxes of
// `lines` of them, at most 256, in the 128-byte swizzle.
bool encode_cache(CUtensorMap* map, const void* codes, int64_t bytes, int lines);

// One CTA per SM; the merge looks at all of them with one thread each.
int cta_count();
// Bytes of the workspace that hold the CTAs' Tags, in front of their pieces.
size_t meta_bytes(int ctas);

// The kernel for many query rows (lq_attn_paged_tiles.cu): its units of work
// (pairs of row tiles of a kv head, at most so many) and the CTAs that share one.
struct TilePlan {
  int64_t units;
  int splits;
};
// most_tokens: positions that any request can have.
TilePlan plan_tiles(int batch, int64_t total_q, int group, int kv_heads, int head_dim, int64_t most_tokens, int sms);
lq_status launch_attn_tiles(const Args& a, const int8_t* kc, const int8_t* vc, int64_t cache_bytes, int head_dim,
                            const TilePlan& plan, void* stream);

}  // namespace attn
}  // namespace lq
