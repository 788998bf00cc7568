// Log probabilities of given tokens from the logits, with the entropy of the
// distribution, the token's rank and the most likely alternatives.
//
// With m = max x, d = x - m rounded to fp32, l = sum e^d and S = sum e^d d over a
// row x:
//     log p(v) = d_v - log l,    entropy = -sum p log p = log l - S / l,
//     rank(t) = the number of v with d_v > d_t, or d_v = d_t and v < t.
// S is negative, so the entropy's two terms do not cancel.  Alternatives are in
// the order of (d descending, token ascending): that of the log probabilities as
// they are given, in which logits that differ by less than d's last place are equal.
//
// One CTA per row, several passes over it.
#include "lq_device.cuh"
#include "lq_host.h"
#include "lq_serve.cuh"

#include <cmath>
#include <cuda_bf16.h>

namespace lq {
namespace score {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = LQ_MAX_ALTERNATIVES;

struct Args {
  const void* x;
  int64_t ld, rows, vocab;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* ranks;
  int top;
  int32_t* top_tokens;
  float* top_logprobs;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else return reinterpret_cast<const float*>(p)[i];
}

// A value and its token as one number, larger for the ones that come first.
__device__ __forceinline__ unsigned long long key_of(float x, uint32_t v) {
  uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);                 // -0 is 0
  b = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (unsigned long long)b << 32 | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

template <typename T, typename F>
__device__ __forceinline__ T over_cta(T x, T* sh, F f) {
  for (int o = 16; o; o >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
  for (int w = 1; w < kWarps; ++w) x = f(x, sh[w]);
  return x;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) score_kernel(Args a) {
  __shared__ float shf[kWarps];
  __shared__ int shi[kWarps];
  __shared__ unsigned long long shk[kWarps];
  pdl_wait();
  pdl_launch();
  const int64_t row = blockIdx.x;
  const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x) + row * a.ld * (BF16 ? 2 : 4);
  const auto add = [](float p, float q) { return p + q; };
  float m = -INFINITY;
  int bad = 0;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
    const float y = at<BF16>(x, v);
    bad |= !(y < INFINITY);
    m = fmaxf(m, y);
  }
  bad = over_cta(bad, shi, [](int p, int q) { return p | q; });
  m = over_cta(m, shf, [](float p, float q) { return fmaxf(p, q); });
  const int32_t token = a.tokens[row];
  const bool given = token >= 0 && token < a.vocab;
  if (threadIdx.x == 0) {
    if (bad) raise_flag(a.status, LQ_DEV_NONFINITE);
    else if (m == -INFINITY) raise_flag(a.status, LQ_DEV_RANGE);
    if (token >= a.vocab) raise_flag(a.status, LQ_DEV_RANGE);
  }
  const float base = m == -INFINITY ? 0.f : m;
  const unsigned long long own = given ? key_of(at<BF16>(x, token) - base, token) : ~0ull;
  float l = 0.f, s = 0.f;
  int before = 0;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
    const float y = at<BF16>(x, v), d = y - base, e = expf(d);
    l += e;
    if (e > 0.f) s = fmaf(e, d, s);
    before += key_of(d, (uint32_t)v) > own;
  }
  l = over_cta(l, shf, add);
  s = over_cta(s, shf, add);
  before = over_cta(before, shi, [](int p, int q) { return p + q; });
  const float log_l = l > 0.f ? logf(l) : 0.f;
  if (threadIdx.x == 0) {
    a.logprobs[row] = bad ? NAN : given ? value_of(own) - log_l : 0.f;
    if (a.entropy != nullptr) a.entropy[row] = bad ? NAN : l > 0.f ? log_l - s / l : 0.f;
    if (a.ranks != nullptr) a.ranks[row] = bad || !given ? -1 : before;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    unsigned long long best = 0;
    if (!bad)
      for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
        const unsigned long long key = key_of(at<BF16>(x, v) - base, (uint32_t)v);
        if (key < last && key > best) best = key;
      }
    best = over_cta(best, shk, [](unsigned long long p, unsigned long long q) { return p > q ? p : q; });
    last = best;
    if (threadIdx.x == 0) {
      a.top_tokens[row * a.top + k] = bad ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)best);
      a.top_logprobs[row * a.top + k] = bad ? NAN : value_of(best) - log_l;
    }
  }
}

}  // namespace score
}  // namespace lq

using namespace lq;

extern "C" lq_status lq_token_logprobs(const void* logits_dev, int64_t ld, int dtype, int64_t rows, int64_t vocab,
                                       const int32_t* tokens_dev, float* logprobs_dev, float* entropy_dev,
                                       int32_t* ranks_dev, int top, int32_t* top_tokens_dev,
                                       float* top_logprobs_dev, int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_token_logprobs");
  if (dtype != LQ_BF16 && dtype != LQ_F32) return LQ_ERR_DTYPE;
  if (rows < 0 || rows > (1 << 24) || vocab <= 0 || vocab > (int64_t(1) << 24) || (rows > 1 && ld < vocab) ||
      top < 0 || top > LQ_MAX_ALTERNATIVES || top > vocab)
    return LQ_ERR_SHAPE;
  if (rows == 0) return LQ_OK;
  const bool elem = dtype == LQ_BF16 ? serve::aligned2(logits_dev) : aligned4(logits_dev);
  if (logits_dev == nullptr || !elem || tokens_dev == nullptr || logprobs_dev == nullptr || !aligned4(tokens_dev) ||
      !aligned4(logprobs_dev) || !aligned4(entropy_dev) || !aligned4(ranks_dev) || !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  if (top > 0 && (top_tokens_dev == nullptr || top_logprobs_dev == nullptr || !aligned4(top_tokens_dev) ||
                  !aligned4(top_logprobs_dev)))
    return LQ_ERR_ARG;
  score::Args a;
  a.x = logits_dev; a.ld = ld; a.rows = rows; a.vocab = vocab; a.tokens = tokens_dev; a.logprobs = logprobs_dev;
  a.entropy = entropy_dev; a.ranks = ranks_dev; a.top = top; a.top_tokens = top_tokens_dev;
  a.top_logprobs = top_logprobs_dev; a.status = dev_status_dev;
  return dtype == LQ_BF16 ? serve::launch(score::score_kernel<true>, (unsigned)rows, score::kThreads, 0, stream, a)
                          : serve::launch(score::score_kernel<false>, (unsigned)rows, score::kThreads, 0, stream, a);
}
