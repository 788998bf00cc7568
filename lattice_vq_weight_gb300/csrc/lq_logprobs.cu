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
// A cluster of up to eight CTAs per row reads the row once: each CTA copies its
// share to shared memory in pieces (untiled bulk copies; the few elements before and
// after the 16-byte boundaries by ordinary loads) and takes maxima as they arrive, the
// CTAs agree on the row's maximum, and everything else, whose terms hang on it, comes
// from shared memory.  The exponentials, one fma, two additions, the rank's comparison
// and the unpacking make about 8 instructions an element, so rows stay bound by HBM as
// long as other CTAs of the SM load meanwhile.  Sums go through fixed trees: equal
// calls give equal bits.
//
// Alternatives: the k-th largest of 32 maxima, each over every 32nd 16-byte chunk of
// the share, is a bound that at least k elements reach and few others do; those are
// listed on the way and ranked by counting.  Where more reach it than there is room
// for (equal logits, large ones in step with the chunks), the k are taken one after
// the other instead.
#include "lq_device.cuh"
#include "lq_host.h"
#include "lq_serve.cuh"
#include "lq_tma.cuh"

#include <cmath>
#include <cuda_bf16.h>

namespace lq {
namespace score {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = LQ_MAX_ALTERNATIVES, kMaxCluster = 8;
constexpr int kPieces = 8;                     // copies that a share is split into
constexpr int kRoom = 1024;                    // candidates that are listed
constexpr int kByRank = 256;                   // and ordered by counting
constexpr int kMostBytes = 192 * 1024;         // of a share in shared memory at once
constexpr long long kWaitCycles = 2000000000ll;
typedef unsigned long long u64;

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
  int cluster;
  int64_t share;             // elements of a row per CTA
  int segment;               // of those in shared memory at once
};

// A value and its token as one number, larger for the ones that come first.
__device__ __forceinline__ u64 key_of(float x, uint32_t v) {
  uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);                 // -0 is 0
  b = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (u64)b << 32 | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}
// The number after x (x <= 0).
__device__ __forceinline__ float after(float x) {
  return x == 0.f ? __uint_as_float(1u) : __uint_as_float(__float_as_uint(x) - 1u);
}

template <bool BF16>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else return reinterpret_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[BF16 ? 8 : 4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    } else {
      v[e] = __uint_as_float(u[e]);
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// This CTA's shared address `p`, of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t theirs;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(theirs) : "r"(smem_addr(p)), "r"(rank));
  return theirs;
}
__device__ __forceinline__ void put(uint32_t to, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t to, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory");
}

__device__ __forceinline__ void copy_in(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// What a CTA finds in its share, for the cluster's first one.
struct Found {
  float l, s;
  int before, pad;
  u64 top[kMaxTop];
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) score_kernel(const __grid_constant__ Args a) {
  constexpr int E = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;
  extern __shared__ __align__(16) uint8_t image[];
  __shared__ uint64_t bars[kPieces];
  __shared__ float maxima[kWarps][32];
  __shared__ float sums[kWarps][2];
  __shared__ int counts[kWarps];
  __shared__ float tops[kMaxCluster];          // the CTAs' maxima
  __shared__ float bound;                      // of the candidates, a logit
  __shared__ int listed, timeout;
  __shared__ u64 list[kRoom], best[kMaxTop], round_best[kWarps];
  __shared__ Found found[kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = a.cluster, rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / ctas;

  if (tid == 0) {
    for (int p = 0; p < kPieces; ++p) mbar_init1(bars + p, 1);
    mbar_init_fence();
    timeout = 0;
  }
  if (ctas > 1) cluster_arrive();              // the others' shared memory is there once all have come here
  pdl_wait();
  pdl_launch();
  __syncthreads();

  const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x) + row * a.ld * kSize;
  const int64_t v0 = min(a.vocab, rank * a.share), v1 = min(a.vocab, v0 + a.share);
  const int segments = v1 > v0 ? (int)((v1 - v0 + a.segment - 1) / a.segment) : 1;

  // A segment: n elements from token base on, in 16-byte chunks of which the first
  // `skew` elements and those past the end are -inf.
  int64_t base = 0;
  int n = 0, skew = 0, chunks = 0, body = 0, per_piece = 0;
  uint32_t phase = 0;
  auto load = [&](int segment) {
    base = v0 + (int64_t)segment * a.segment;
    n = (int)min((int64_t)a.segment, v1 - base);
    const uint8_t* src = x + base * kSize;
    const int head = min(n, (int)((0u - (uint32_t)reinterpret_cast<uintptr_t>(src)) & 15u) / kSize);
    skew = head > 0 ? E - head : 0;
    body = (n - head) / E;                     // whole chunks
    chunks = (skew + n + E - 1) / E;
    per_piece = (body + kPieces - 1) / kPieces;
    const int first = skew > 0;
    if (tid < kPieces) {
      const int c0 = min(body, tid * per_piece), c1 = min(body, c0 + per_piece);
      mbar_expect_tx(bars + tid, (c1 - c0) * 16);
      if (c1 > c0) copy_in(image + (first + c0) * 16, src + head * kSize + c0 * 16, (c1 - c0) * 16, bars + tid);
    }
    // what lies outside the boundaries: first and last chunk
    if (warp == 1) {
      const uint32_t none = BF16 ? 0xFF80u : 0xFF800000u;
      const auto set = [&](int slot, uint32_t v) {
        if constexpr (BF16) reinterpret_cast<uint16_t*>(image)[slot] = (uint16_t)v;
        else reinterpret_cast<uint32_t*>(image)[slot] = v;
      };
      const auto get = [&](int i) -> uint32_t {
        if constexpr (BF16) return reinterpret_cast<const uint16_t*>(src)[i];
        else return reinterpret_cast<const uint32_t*>(src)[i];
      };
      if (first && lane < E) set(lane, lane >= skew && lane - skew < n ? get(lane - skew) : none);
      const int slot = (first + body) * E + lane;           // after the body
      if (lane < E && slot < chunks * E) set(slot, slot - skew < n ? get(slot - skew) : none);
    }
    __syncthreads();
  };
  // Runs f(chunk, its 16 bytes) over this thread's chunks as their pieces arrive.
  auto each = [&](auto f) {
    const int first = skew > 0;
#pragma unroll 1
    for (int p = 0; p < kPieces; ++p) {
      const int c0 = p == 0 ? 0 : first + min(body, p * per_piece);
      const int c1 = p == kPieces - 1 ? chunks : first + min(body, (p + 1) * per_piece);
      if (c0 >= c1) continue;
      if (!mbar_wait_bounded(bars + p, phase, kWaitCycles)) {
        timeout = 1;
        break;
      }
#pragma unroll 4
      for (int c = c0 + ((tid - c0) & (kThreads - 1)); c < c1; c += kThreads)
        f(c, reinterpret_cast<const uint4*>(image)[c]);
    }
  };
  // The largest logit of this thread's chunks.
  auto largest = [&]() {
    float m = -INFINITY;
    each([&](int, const uint4& w) {
      float v[E];
      unpack<BF16>(w, v);
#pragma unroll
      for (int e = 0; e < E; e += 2) m = fmaxf(m, fmaxf(v[e], v[e + 1]));
    });
    return m;
  };
  // From the threads' maxima the CTA's, and the bound under its candidates.
  auto bound_of = [&](float mine) {
    maxima[warp][lane] = mine;
    __syncthreads();
    float m = -INFINITY;
    if (warp == 0) {
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, maxima[w][lane]);
      if (a.top > 0) {
        int ahead = 0;                         // lanes whose maximum comes before this one's
#pragma unroll 8
        for (int o = 0; o < 32; ++o) {
          const float y = __shfl_sync(0xffffffffu, m, o);
          ahead += y > m || (y == m && o < lane);
        }
        if (ahead == a.top - 1) bound = m;
      }
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;                                  // in warp 0
  };

  // the row's maximum
  float mine = -INFINITY;
  for (int g = 0; g < segments; ++g) {
    if (g > 0) {
      fence_proxy_async_smem();
      __syncthreads();
      phase ^= 1;
    }
    load(g);
    mine = fmaxf(mine, largest());
  }
  float m = bound_of(mine);
  if (ctas > 1) {
    cluster_wait();
    if (warp == 0 && lane < ctas) put(peer(tops + rank, lane), m);
    cluster_arrive();
    cluster_wait();
  } else {
    if (tid == 0) tops[0] = m;
    __syncthreads();
  }
  m = tops[0];
  for (int r = 1; r < ctas; ++r) m = fmaxf(m, tops[r]);
  const float zero = m == -INFINITY ? 0.f : m;

  const int32_t token = a.tokens[row];
  const bool given = token >= 0 && token < a.vocab;
  const float dt = given ? at<BF16>(x, token) - zero : INFINITY;
  const float dt_after = given ? after(dt) : INFINITY;              // d > dt is d >= dt_after

  float2 l2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
  int before = 0, have = 0;                    // have: alternatives found in earlier segments
  for (int g = 0; g < segments; ++g) {
    if (segments > 1) {                        // the share again
      fence_proxy_async_smem();
      __syncthreads();
      phase ^= 1;
      load(g);
      bound_of(largest());
    }
    if (tid < have) list[tid] = best[tid];
    if (tid == 0) listed = have;
    __syncthreads();
    const float least = a.top > 0 ? bound - zero : INFINITY;
    const int64_t first = base - skew;         // token of the image's first slot
    each([&](int c, const uint4& w) {
      float v[E];
      unpack<BF16>(w, v);
      const int64_t t0 = first + (int64_t)c * E;
      const float2 shift = make_float2(-zero, -zero), log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
      float high = -INFINITY;
      // all of the chunk before the token, or all after it; the chunk that holds it and
      // those with slots that are no tokens are looked at one by one
      const bool apart = (token >= t0 && token < t0 + E) || c == 0 || c == chunks - 1;
      const float from = t0 < token ? dt : dt_after;
      int more = 0;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 d = add2(make_float2(v[e], v[e + 1]), shift);
        more += (d.x >= from) + (d.y >= from);
        v[e] = d.x;
        v[e + 1] = d.y;
        high = fmaxf(high, fmaxf(d.x, d.y));
        d = make_float2(max_nan(d.x, -1e30f), max_nan(d.y, -1e30f));       // -inf: no term, not 0 times itself
        float2 y = mul2(d, log2e);
        y = make_float2(ex2(y.x), ex2(y.y));
        l2 = add2(l2, y);
        s2 = fma2(y, d, s2);
      }
      if (apart) {
        more = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int64_t t = t0 + e;
          more += t >= base && t < base + n && (v[e] >= dt_after || (v[e] == dt && t < token));
        }
      }
      before += more;
      if (high >= least) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int64_t t = t0 + e;
          if (v[e] >= least && t >= base && t < base + n) {
            const int to = atomicAdd(&listed, 1);
            if (to < kRoom) list[to] = key_of(v[e], (uint32_t)t);
          }
        }
      }
    });
    __syncthreads();
    if (a.top > 0) {
      const int count = listed, k = min((int64_t)a.top, (int64_t)have + n);
      if (count <= kByRank) {
        const u64 key = tid < count ? list[tid] : 0;
        int ahead = 0;
#pragma unroll 8
        for (int i = 0; i < count; ++i) ahead += list[i] > key;
        __syncthreads();
        if (tid < count && ahead < k) best[ahead] = key;
      } else {
        // one after the other: the largest key below the last, of the list or, where it
        // has overflowed, of the earlier segments' and the whole segment
        u64 last = ~0ull;
        const int old = count <= kRoom ? count : have;
        u64 taken = 0;
        for (int i = 0; i < k; ++i) {
          u64 top = 0;
          for (int j = tid; j < old; j += kThreads)
            if (list[j] < last && list[j] > top) top = list[j];
          if (count > kRoom)
            each([&](int c, const uint4& w) {
              float v[E];
              unpack<BF16>(w, v);
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const int64_t t = first + (int64_t)c * E + e;
                const u64 key = key_of(v[e] - zero, (uint32_t)t);
                if (t >= base && t < base + n && key < last && key > top) top = key;
              }
            });
          for (int o = 16; o; o >>= 1) {
            const u64 y = __shfl_xor_sync(0xffffffffu, top, o);
            top = y > top ? y : top;
          }
          if (lane == 0) round_best[warp] = top;
          __syncthreads();
          for (int w = 0; w < kWarps; ++w) top = round_best[w] > top ? round_best[w] : top;
          __syncthreads();
          last = top;
          if (tid == i) taken = top;
        }
        if (tid < k) best[tid] = taken;
      }
      have = k;
      __syncthreads();
    }
  }

  // sums over the CTA, then over the cluster, in a fixed order
  float l = l2.x + l2.y, s = s2.x + s2.y;
  for (int o = 16; o; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    s += __shfl_xor_sync(0xffffffffu, s, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    sums[warp][0] = l;
    sums[warp][1] = s;
    counts[warp] = before;
  }
  __syncthreads();
  if (warp == 0) {
    l = s = 0.f;
    before = 0;
    for (int w = 0; w < kWarps; ++w) {
      l += sums[w][0];
      s += sums[w][1];
      before += counts[w];
    }
    Found* to = found + rank;
    if (ctas > 1) {
      if (lane == 0) {
        put(peer(&to->l, 0), l);
        put(peer(&to->s, 0), s);
        put(peer(&to->before, 0), __int_as_float(before));
      }
      if (lane < a.top) put(peer(&to->top[lane], 0), lane < have ? best[lane] : (u64)0);
    } else {
      if (lane == 0) {
        to->l = l;
        to->s = s;
        to->before = before;
      }
      if (lane < a.top) to->top[lane] = lane < have ? best[lane] : 0;
    }
  }
  if (ctas > 1) {
    cluster_arrive();
    if (rank != 0) {
      if (tid == 0 && timeout) raise_flag(a.status, LQ_DEV_TIMEOUT);
      return;
    }
    cluster_wait();
  } else {
    __syncthreads();
  }
  l = s = 0.f;
  before = 0;
  for (int r = 0; r < ctas; ++r) {
    l += found[r].l;
    s += found[r].s;
    before += found[r].before;
  }
  const bool bad = !(l < INFINITY);            // NaN: one among the logits, or +inf less itself
  const float log_l = l > 0.f ? logf(l) : 0.f;
  if (tid == 0) {
    if (timeout) raise_flag(a.status, LQ_DEV_TIMEOUT);
    if (bad) raise_flag(a.status, LQ_DEV_NONFINITE);
    else if (m == -INFINITY) raise_flag(a.status, LQ_DEV_RANGE);
    if (token >= a.vocab) raise_flag(a.status, LQ_DEV_RANGE);
    a.logprobs[row] = bad ? NAN : given ? dt - log_l : 0.f;
    if (a.entropy != nullptr) a.entropy[row] = bad ? NAN : l > 0.f ? log_l - s / l : 0.f;
    if (a.ranks != nullptr) a.ranks[row] = bad || !given ? -1 : before;
  }
  if (tid < a.top * ctas) {
    // an alternative's place: how many of all CTAs' lists come before it
    const u64 key = found[tid / a.top].top[tid % a.top];
    int ahead = 0;
    for (int r = 0; r < ctas; ++r)
      for (int i = 0; i < a.top; ++i) ahead += found[r].top[i] > key;
    if (key != 0 && ahead < a.top) {
      a.top_tokens[row * a.top + ahead] = bad ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)key);
      a.top_logprobs[row * a.top + ahead] = bad ? NAN : value_of(key) - log_l;
    }
  }
  if (bad && tid < a.top) {                    // (keys of NaN say nothing)
    a.top_tokens[row * a.top + tid] = -1;
    a.top_logprobs[row * a.top + tid] = NAN;
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
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  // As few CTAs per row as keep several shares on an SM, more where the rows alone
  // would leave SMs idle.
  const int64_t esize = dtype == LQ_BF16 ? 2 : 4, bytes = vocab * esize;
  int ctas = 1;
  while (ctas < score::kMaxCluster &&
         (bytes / ctas > 52 * 1024 || (rows * ctas < 2 * sms && bytes / ctas > 8 * 1024)))
    ctas *= 2;
  a.cluster = ctas;
  a.share = (vocab + ctas - 1) / ctas;
  a.segment = (int)(a.share < score::kMostBytes / esize ? a.share : score::kMostBytes / esize);
  const int smem = (int)(a.segment * esize) / 16 * 16 + 48;          // chunks at both ends may be partial
  const auto kernel = dtype == LQ_BF16 ? score::score_kernel<true> : score::score_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, score::kMostBytes + 48) !=
      cudaSuccess) {
    cudaGetLastError();
    return LQ_ERR_CUDA;
  }
  return serve::launch(kernel, (unsigned)(rows * ctas), score::kThreads, smem, stream, a, (unsigned)ctas);
}
