// Verification of drafted tokens against the target's probabilities, with the
// random numbers given by the caller (speculative sampling: Leviathan et al.
// 2023, Chen et al. 2023).
//
// Request b brings n_b drafted tokens x_0 .. x_{n-1}, drawn from the draft
// distributions q_i, and the target's distributions p_0 .. p_n.  Token i is
// accepted while u_i q_i(x_i) < p_i(x_i); with a accepted, the token after them
// is drawn from max(p_a - q_a, 0) if a < n and from p_n otherwise (from p_a
// when no weight is left).  A draft without distributions (NULL) is one that
// takes its token for certain: q_i is one at x_i and zero elsewhere.
//
// The draw inverts a cumulative sum over the vocabulary.  Its weights are
// whole numbers, floor(2^36 w), so their sums do not depend on the order or the
// split of the summation and the drawn token is a function of the inputs alone:
// the first v whose inclusive sum exceeds floor(u * total), u's 24 bits taken
// as a whole number.  (A weight below 2^-36 counts as zero, 1e-11 of the mass.)
//
// A CTA per request: the acceptance tests in the first warp, then each warp
// sums its share of the vocabulary, the warp in whose share the drawn token
// lies finds it by scanning that share again.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace verify {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct Args {
  const int32_t* tokens;
  const int32_t* lens;
  int batch, max_draft;
  int64_t vocab;
  const void* p;
  int64_t p_req, p_row;
  const void* q;
  int64_t q_req, q_row;
  const float* u_accept;
  const float* u_sample;
  int32_t* out;
  int32_t* accepted;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + i) << 16);
  else return __ldg(reinterpret_cast<const float*>(p) + i);
}

// floor(2^36 w) of a weight in [0, 4]; NaN and negative weights count as zero.
__device__ __forceinline__ unsigned long long whole(float w) {
  return w > 0.f ? __float2ull_rz(fminf(w, 4.f) * 68719476736.f) : 0ull;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_kernel(Args a) {
  __shared__ int s_acc, s_found;
  __shared__ unsigned long long part[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  pdl_wait();
  pdl_launch();
  int n = a.lens != nullptr ? __ldg(a.lens + b) : a.max_draft;
  if (n < 0 || n > a.max_draft) {
    if (tid == 0) raise_flag(a.status, LQ_DEV_RANGE);
    n = n < 0 ? 0 : a.max_draft;
  }
  if (warp == 0) {
    int acc = n;
    for (int i0 = 0; i0 < n && acc == n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int64_t x = __ldg(a.tokens + (int64_t)b * a.max_draft + i);
        ok = false;
        if (x >= 0 && x < a.vocab) {
          const float p = at<BF16>(a.p, b * a.p_req + i * a.p_row + x);
          const float q = a.q != nullptr ? at<BF16>(a.q, b * a.q_req + i * a.q_row + x) : 1.f;
          ok = __fmul_rn(__ldg(a.u_accept + (int64_t)b * a.max_draft + i), q) < p;
        } else {
          raise_flag(a.status, LQ_DEV_RANGE);
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, !ok);
      if (no) acc = i0 + __ffs(no) - 1;
    }
    if (lane == 0) {
      s_acc = acc;
      s_found = -1;
    }
  }
  __syncthreads();
  const int acc = s_acc;
  bool rest = acc < n;
  const int64_t pr = b * a.p_req + acc * a.p_row, qr = b * a.q_req + acc * a.q_row;
  const int64_t gone = (rest && a.q == nullptr) ? __ldg(a.tokens + (int64_t)b * a.max_draft + acc) : -1;
  const int64_t share = (a.vocab + kWarps - 1) / kWarps;
  const int64_t v0 = min(a.vocab, warp * share), v1 = min(a.vocab, v0 + share);
  auto weight = [&](int64_t v) {
    float w = at<BF16>(a.p, pr + v);
    if (!(w <= 3.402823466e38f)) raise_flag(a.status, LQ_DEV_NONFINITE);
    if (rest) w = a.q != nullptr ? w - at<BF16>(a.q, qr + v) : (v == gone ? 0.f : w);
    return whole(w);
  };
  unsigned long long total = 0, before = 0;
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long sum = 0;
    for (int64_t v = v0 + lane; v < v1; v += 32) sum += weight(v);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before = total;
      total += part[w];
    }
    if (total > 0 || !rest) break;
    rest = false;                        // nothing left of p - q: draw from p
  }
  if (total > 0) {
    float u = __ldg(a.u_sample + b);
    u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
    const unsigned long long k = (unsigned long long)(u * 16777216.f);
    const unsigned long long goal = (__umul64hi(total, k) << 40) | ((total * k) >> 24);
    if (goal >= before && goal < before + part[warp]) {
      unsigned long long run = before;
      for (int64_t c = v0; c < v1; c += 32) {
        const unsigned long long w = c + lane < v1 ? weight(c + lane) : 0ull;
        unsigned long long inc = w;
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + inc > goal);
        if (hit) {
          if (lane == 0) s_found = (int)(c + __ffs(hit) - 1);
          break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  } else if (tid == 0) {
    raise_flag(a.status, LQ_DEV_RANGE);
  }
  __syncthreads();
  for (int i = tid; i <= a.max_draft; i += kThreads)
    a.out[(int64_t)b * (a.max_draft + 1) + i] =
        i < acc ? __ldg(a.tokens + (int64_t)b * a.max_draft + i) : (i == acc ? s_found : -1);
  if (tid == 0) a.accepted[b] = acc;
}

}  // namespace verify
}  // namespace lq

using namespace lq;

extern "C" lq_status lq_verify_draft(const int32_t* draft_tokens_dev, const int32_t* draft_lens_dev, int batch,
                                     int max_draft, int64_t vocab, const void* target_probs_dev,
                                     int64_t target_req_stride, int64_t target_row_stride,
                                     const void* draft_probs_dev, int64_t draft_req_stride, int64_t draft_row_stride,
                                     int dtype, const float* u_accept_dev, const float* u_sample_dev,
                                     int32_t* out_tokens_dev, int32_t* accepted_dev, int32_t* dev_status_dev,
                                     void* stream) {
  LQ_NVTX_RANGE("lq_verify_draft");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  if (batch < 0 || batch > (1 << 20) || max_draft < 0 || max_draft > 1024 || vocab <= 0 ||
      vocab > (int64_t(1) << 24))
    return LQ_ERR_SHAPE;
  if (target_row_stride < 0 || target_req_stride < 0 || (max_draft > 0 && target_row_stride < vocab))
    return LQ_ERR_SHAPE;
  if (draft_probs_dev != nullptr && max_draft > 0 && (draft_row_stride < vocab || draft_req_stride < 0))
    return LQ_ERR_SHAPE;
  if (batch == 0) return LQ_OK;
  auto elem_aligned = [&](const void* p) { return dtype == LQ_BF16 ? serve::aligned2(p) : aligned4(p); };
  if (target_probs_dev == nullptr || !elem_aligned(target_probs_dev) || !elem_aligned(draft_probs_dev) ||
      u_sample_dev == nullptr || !aligned4(u_sample_dev) || out_tokens_dev == nullptr || !aligned4(out_tokens_dev) ||
      accepted_dev == nullptr || !aligned4(accepted_dev) || !aligned4(draft_lens_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  if (max_draft > 0 && (draft_tokens_dev == nullptr || u_accept_dev == nullptr || !aligned4(draft_tokens_dev) ||
                        !aligned4(u_accept_dev)))
    return LQ_ERR_ARG;
  verify::Args a;
  a.tokens = draft_tokens_dev; a.lens = draft_lens_dev; a.batch = batch; a.max_draft = max_draft; a.vocab = vocab;
  a.p = target_probs_dev; a.p_req = target_req_stride; a.p_row = target_row_stride;
  a.q = draft_probs_dev; a.q_req = draft_req_stride; a.q_row = draft_row_stride;
  a.u_accept = u_accept_dev; a.u_sample = u_sample_dev; a.out = out_tokens_dev; a.accepted = accepted_dev;
  a.status = dev_status_dev;
  return dtype == LQ_BF16
             ? serve::launch(verify::verify_kernel<true>, (unsigned)batch, verify::kThreads, 0, stream, a)
             : serve::launch(verify::verify_kernel<false>, (unsigned)batch, verify::kThreads, 0, stream, a);
}
