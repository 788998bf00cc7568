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
// as a whole number.  (A weight below 2^-36 counts as zero, 1e-11 of the mass, and
// one above 4, which no probability is, as 4: 2^24 of them then fit 64 bits.)
//
// A cluster of CTAs per request, up to eight by the vocabulary's size, so that
// a small batch still reads its rows with many SMs.  Every CTA runs the
// acceptance tests for itself (a few gathered values), sums its share of the
// row warp by warp, and reads the other CTAs' sums from their shared memory;
// the CTA in whose share the drawn token lies then looks again at the one
// warp's part of it that holds the token, all its threads at once.  Bound by
// reading the one row of p and of q that the request draws from.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

#include <cuda_bf16.h>

namespace lq {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct Args {
  const int32_t* tokens;
  const int32_t* lens;
  int batch, max_draft, cluster;
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
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else return reinterpret_cast<const float*>(p)[i];
}

// floor(2^36 w) of a weight in [0, 4]; NaN and negative weights count as zero.
// From the bits, mantissa shifted by exponent: the conversion instruction to 64
// bits would bound the kernel.
__device__ __forceinline__ unsigned long long whole(float w) {
  const uint32_t bits = __float_as_uint(fminf(fmaxf(w, 0.f), 4.f));       // (fmaxf of NaN and 0 is 0)
  const int e = (int)(bits >> 23);                                        // w = 1.m 2^(e - 127)
  const uint32_t top = bits << 8 | 0x80000000u;
  return e < 91 ? 0ull : ((unsigned long long)top << 32) >> (154 - e);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// The 64-bit word at this CTA's shared address `p`, of CTA `rank` of the cluster.
__device__ __forceinline__ unsigned long long peer_word(const unsigned long long* p, uint32_t rank) {
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t theirs;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(theirs) : "r"(mine), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(theirs) : "memory");
  return v;
}

// Shifts whose amount past 31, also a negative one, gives 0 (as PTX defines them).
__device__ __forceinline__ uint32_t shr0(uint32_t x, int by) {
  uint32_t y;
  asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
  return y;
}
__device__ __forceinline__ uint32_t shl0(uint32_t x, int by) {
  uint32_t y;
  asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
  return y;
}

// Sum of the weights of x - y: whole() without a branch or a 64-bit shift, the
// two words of the weight by shifts that leave 0 where there is nothing.
// `most` grows to the largest magnitude of x, as bits.
struct Sum {
  unsigned long long n = 0;
  uint32_t most = 0;
  __device__ __forceinline__ void add(float x, float y) {
    most = max(most, __float_as_uint(x) & 0x7FFFFFFFu);
    const uint32_t bits = __float_as_uint(fminf(fmaxf(x - y, 0.f), 4.f));
    const uint32_t top = bits << 8 | 0x80000000u;
    const int e = 122 - (int)(bits >> 23);
    const uint32_t hi = shr0(top, e + 32), lo = shr0(top, e) | shl0(top, -e);
    n += (unsigned long long)hi << 32 | lo;
  }
};

// A row's weights: p, or max(p - q, 0), or p without one token.
template <bool BF16>
struct Row {
  const void* p;
  const void* q;             // null: none
  int64_t gone;              // token left out, -1: none
  int32_t* status;
  __device__ __forceinline__ unsigned long long weight(int64_t v) const {
    return whole(v == gone ? 0.f : at<BF16>(p, v) - (q != nullptr ? at<BF16>(q, v) : 0.f));
  }
  // the sum over [v0, v1) of a warp's lanes; v0 a multiple of 8
  __device__ __forceinline__ unsigned long long sum(int64_t v0, int64_t v1, int lane) const {
    constexpr int E = BF16 ? 8 : 4;                // values per 16-byte load
    Sum n;
    int64_t v = v0;
    const uintptr_t low = reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q);
    if ((low & 15) == 0) {                         // rows that start at 16-byte boundaries
      const uint4* pv = reinterpret_cast<const uint4*>(p) + v0 / E + lane;
      const uint4* qv = reinterpret_cast<const uint4*>(q) + v0 / E + lane;
      const int steps = (int)(v1 > v0 ? (v1 - v0) / (32 * E) : 0);
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        const uint4 x = pv[32 * i];
        const uint4 y = q != nullptr ? qv[32 * i] : make_uint4(0, 0, 0, 0);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (BF16) {
            n.add(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16));
            n.add(__uint_as_float(xs[e] & 0xFFFF0000u), __uint_as_float(ys[e] & 0xFFFF0000u));
          } else {
            n.add(__uint_as_float(xs[e]), __uint_as_float(ys[e]));
          }
        }
      }
      v += (int64_t)steps * (32 * E);
    }
#pragma unroll 8
    for (v += lane; v < v1; v += 32) n.add(at<BF16>(p, v), q != nullptr ? at<BF16>(q, v) : 0.f);
    if (lane == 0 && gone >= v0 && gone < v1) n.n -= whole(at<BF16>(p, gone));
    for (int o = 16; o; o >>= 1) n.n += __shfl_xor_sync(0xffffffffu, n.n, o);
    if (n.most >= 0x7F800000u) raise_flag(status, LQ_DEV_NONFINITE);
    else if (n.most > 0x40800000u) raise_flag(status, LQ_DEV_RANGE);      // above 4
    return n.n;
  }
};

// Six CTAs per SM (40 registers a thread): 96 requests of eight CTAs are then
// one wave; with 48 registers and five they took 34 us instead of 26.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 6) verify_kernel(Args a) {
  __shared__ int s_acc;
  __shared__ unsigned long long part[kWarps], total_here, scan[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = a.cluster, rank = ctas > 1 ? (int)cluster_rank() : 0, b = blockIdx.x / ctas;
  pdl_wait();
  pdl_launch();
  int n = a.lens != nullptr ? a.lens[b] : a.max_draft;
  if (n < 0 || n > a.max_draft) {
    if (tid == 0) raise_flag(a.status, LQ_DEV_RANGE);
    n = n < 0 ? 0 : a.max_draft;
  }
  const int32_t* drafted = a.tokens + (int64_t)b * a.max_draft;
  if (warp == 0) {
    int acc = n;
    for (int i0 = 0; i0 < n && acc == n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int64_t x = drafted[i];
        ok = false;
        if (x >= 0 && x < a.vocab) {
          const float p = at<BF16>(a.p, b * a.p_req + i * a.p_row + x);
          const float q = a.q != nullptr ? at<BF16>(a.q, b * a.q_req + i * a.q_row + x) : 1.f;
          ok = __fmul_rn(a.u_accept[(int64_t)b * a.max_draft + i], q) < p;
        } else {
          raise_flag(a.status, LQ_DEV_RANGE);
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, !ok);
      if (no) acc = i0 + __ffs(no) - 1;
    }
    if (lane == 0) s_acc = acc;
  }
  __syncthreads();
  const int acc = s_acc;
  constexpr int64_t esize = BF16 ? 2 : 4;
  Row<BF16> row;
  row.p = reinterpret_cast<const uint8_t*>(a.p) + (b * a.p_req + acc * a.p_row) * esize;
  row.q = acc < n && a.q != nullptr ? reinterpret_cast<const uint8_t*>(a.q) + (b * a.q_req + acc * a.q_row) * esize
                                    : nullptr;
  row.gone = acc < n && a.q == nullptr ? drafted[acc] : -1;
  row.status = a.status;

  // shares of a multiple of 8 tokens: CTA by CTA, in each warp by warp
  const int64_t share = ((a.vocab + (int64_t)ctas * kWarps - 1) / ((int64_t)ctas * kWarps) + 7) & ~(int64_t)7;
  auto begin_of = [&](int w) { return min(a.vocab, ((int64_t)rank * kWarps + w) * share); };
  unsigned long long total = 0, before = 0;        // all CTAs', and those before this one
  for (int pass = 0; pass < 2; ++pass) {
    const unsigned long long mine = row.sum(begin_of(warp), begin_of(warp + 1), lane);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    unsigned long long here = 0;
    for (int w = 0; w < kWarps; ++w) here += part[w];
    if (ctas > 1) {
      if (tid == 0) total_here = here;
      cluster_sync();
      total = 0;
      for (int r = 0; r < ctas; ++r) {
        if (r == rank) before = total;
        total += peer_word(&total_here, (uint32_t)r);
      }
      cluster_sync();                              // read before anyone writes it again or leaves
    } else {
      total = here;
    }
    if (total > 0 || (row.q == nullptr && row.gone < 0)) break;
    row.q = nullptr;                               // nothing left of p - q: draw from p
    row.gone = -1;
    __syncthreads();
  }

  int32_t* out = a.out + (int64_t)b * (a.max_draft + 1);
  if (total > 0) {
    float u = a.u_sample[b];
    u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
    const unsigned long long k = (unsigned long long)(u * 16777216.f);
    const unsigned long long goal = (__umul64hi(total, k) << 40) | ((total * k) >> 24);
    // the warp's part that holds the token, if it lies in this CTA
    int w = 0;
    unsigned long long run = before;
    while (w < kWarps && goal >= run + part[w]) run += part[w++];
    if (goal >= before && w < kWarps) {
      // its tokens in runs, a run per thread; the sums before each thread's run
      const int64_t v0 = begin_of(w), v1 = begin_of(w + 1);
      const int64_t per = (v1 - v0 + kThreads - 1) / kThreads;
      const int64_t c0 = min(v1, v0 + tid * per), c1 = min(v1, c0 + per);
      unsigned long long sum = 0;
#pragma unroll 8
      for (int64_t v = c0; v < c1; ++v) sum += row.weight(v);
      unsigned long long inc = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      for (int i = 0; i < warp; ++i) inc += scan[i];
      unsigned long long at_run = run + inc - sum;
      if (goal >= at_run && goal < at_run + sum) {
        int64_t v = c0;
        for (; v < c1; ++v) {
          at_run += row.weight(v);
          if (at_run > goal) break;
        }
        out[acc] = (int32_t)v;
      }
    }
  } else if (rank == 0 && tid == 0) {
    out[acc] = -1;
    raise_flag(a.status, LQ_DEV_RANGE);
  }
  if (rank == 0) {
    for (int i = tid; i <= a.max_draft; i += kThreads)
      if (i != acc) out[i] = i < acc ? drafted[i] : -1;
    if (tid == 0) a.accepted[b] = acc;
  }
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
  // a CTA for every 4096 tokens of the vocabulary: shares of 2 or more 16-byte
  // loads per lane
  a.cluster = 1;
  while (a.cluster < verify::kMaxCluster && (int64_t)a.cluster * 4096 < vocab) a.cluster *= 2;
  const unsigned grid = (unsigned)batch * (unsigned)a.cluster;
  return dtype == LQ_BF16
             ? serve::launch(verify::verify_kernel<true>, grid, verify::kThreads, 0, stream, a, a.cluster)
             : serve::launch(verify::verify_kernel<false>, grid, verify::kThreads, 0, stream, a, a.cluster);
}
