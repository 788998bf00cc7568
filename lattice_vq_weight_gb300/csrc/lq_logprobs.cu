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
// A row is read once where a cluster's shared memory holds it (longer ones, in segments,
// twice; ranks among logits within 2^-70 of 0 or against masked tokens, and an overflowing
// list of candidates, read the row again).  A CTA, or a cluster of up to eight where a row is longer than
// one SM's shared memory or there are few rows, copies its share of a row to shared
// memory in four pieces (untiled bulk copies) and takes maxima as they arrive; the
// CTAs agree on the row's maximum, and everything else, whose terms hang on it, comes
// from shared memory: 7 to 8 instructions an element for the exponential, the sums and
// the rank's comparison (by saturating products: as compare and count it was the pipe of
// compares and integers that bound the kernel, 135 us for 2047 rows of 50001 to 106).
// CTAs stay for row after row: as soon as a piece has been read for the last time, a warp
// of its own copies the same piece of the next row over it, so that the loads run under
// the exponentials, and finishes the row before.  A cluster waits for itself once per row: the
// maxima of a row and the results of the row before cross together, and a row's results
// are put together by its CTAs in turn.  Sums go through fixed trees: equal calls give
// equal bits.
//
// Alternatives: the k-th largest of 32 maxima, each over every 32nd 16-byte chunk of
// the share, is a bound that at least k elements reach and few others do; those are
// listed on the way and ranked by counting.  Where more reach it than there is room
// for (equal logits, large ones in step with the chunks, rows of which a mask leaves so few
// that the bound is -inf), the k are taken one after the other instead, from the row itself:
// 96 rows of 128256 with 20 alternatives take 22 us, with all but 30 tokens masked 450.
//
// A row starts at any element: chunks at its ends are copied whole where that stays
// inside the matrix, and slots that are not the row's count as -inf.
#include "lq_device.cuh"
#include "lq_host.h"
#include "lq_logprobs_plan.h"
#include "lq_serve.cuh"
#include "lq_tma.cuh"

#include <atomic>
#include <cmath>
#include <cuda_bf16.h>

namespace lq {
namespace score {

constexpr int kWarps = kThreads / 32;          // and a warp that copies and finishes rows
constexpr int kMaxTop = LQ_MAX_ALTERNATIVES;
constexpr int kRoom = 512;                     // candidates that are listed
constexpr int kByRank = 256;                   // and ordered by counting
constexpr long long kWaitCycles = 2000000000ll;
constexpr float kHuge = 3.40282347e38f;        // the largest number
typedef unsigned long long u64;

struct Args : Division {
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

// 1 where x is above 0 (by 2^-127 or more), else 0, and where x is 0, k.
__device__ __forceinline__ float step_of(float x, float k) {
  float y;
  asm("fma.rn.sat.f32 %0, %1, 0f7F000000, %2;" : "=f"(y) : "f"(x), "f"(k));        // 2^127
  return y;
}

// Barrier of the warps that compute, and one that the last warp comes to without waiting.
__device__ __forceinline__ void sync_workers() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void sync_listed() { asm volatile("bar.sync 2, %0;" ::"n"(kThreads + 32) : "memory"); }
__device__ __forceinline__ void arrive_listed() { asm volatile("bar.arrive 2, %0;" ::"n"(kThreads + 32) : "memory"); }

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

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void copy_in(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// A segment of a CTA's share of a row: n elements from token `base` on, in `chunks`
// chunks of 16 bytes whose first `skew` slots and last ones may not be the row's.
struct View {
  const uint8_t* src;        // of the first chunk, at a 16-byte boundary
  int64_t base;
  int n, skew, chunks;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads + 32, 1) score_kernel(const __grid_constant__ Args a) {
  constexpr int E = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;
  extern __shared__ __align__(16) uint8_t image_bytes[];
  uint4* image = reinterpret_cast<uint4*>(image_bytes);
  __shared__ uint64_t full[kPieces], empty[kPieces];
  __shared__ float maxima[kWarps + 1][32];
  __shared__ float sums[kWarps + 1][2];
  __shared__ int counts[kWarps + 1];
  __shared__ float tops[2][kMaxCluster];       // the CTAs' maxima, of this row and the next
  __shared__ float bound;                      // of the candidates, a logit
  __shared__ int listed, timeout;
  __shared__ u64 list[kRoom], best[kMaxTop], round_best[kWarps];
  __shared__ float4 found[2][kMaxCluster];     // the CTAs' sums and counts
  __shared__ u64 keys[2][kMaxCluster * kMaxTop];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = a.cluster, rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int64_t clusters = gridDim.x / ctas, row0 = blockIdx.x / ctas;

  if (tid == 0) {
    for (int p = 0; p < kPieces; ++p) {
      mbar_init1(full + p, 1);
      mbar_init1(empty + p, kWarps);
    }
    mbar_init_fence();
    timeout = listed = 0;
  }
  if (ctas > 1) cluster_arrive();              // the others' shared memory is there once all have come here
  pdl_wait();
  pdl_launch();
  __syncthreads();

  const uint8_t* all = reinterpret_cast<const uint8_t*>(a.x);
  const uint8_t* all_end = all + ((a.rows - 1) * a.ld + a.vocab) * kSize;
  const int64_t v0 = min(a.vocab, rank * a.share), v1 = min(a.vocab, v0 + a.share);
  const int segments = v1 > v0 ? (int)((v1 - v0 + a.segment - 1) / a.segment) : 1;

  auto view = [&](int64_t row, int segment) {
    View w;
    w.base = v0 + (int64_t)segment * a.segment;
    w.n = (int)min((int64_t)a.segment, v1 - w.base);
    const uint8_t* src = all + (row * a.ld + w.base) * kSize;
    const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(src) & 15u;
    w.src = src - low;
    w.skew = w.n > 0 ? (int)low / kSize : 0;
    w.chunks = (w.skew + w.n + E - 1) / E;
    return w;
  };
  // Every wait is bounded (about a second of clock cycles).  A thread whose wait has run out
  // waits no more, lets no piece go and starts no copy, so that the CTA's rows, garbage now,
  // soon come to their end and no piece is copied whose last copy is still under way.
  bool waited = true;                          // until then
  auto wait_for = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity, waited ? kWaitCycles : 0)) {
      timeout = 1;
      waited = false;
    }
  };
  int started = 0;                             // copies, by the last warp's lane 0: of piece 0, 1, ... in turn
  // The last warp copies piece p; its barrier completes a phase even if there is nothing to
  // copy.  The matrix's own first and last chunk, where not all of it is inside, come by
  // single loads.
  auto start = [&](const View& w, int p) {
    int c0 = min(w.chunks, p * a.per_piece), c1 = min(w.chunks, c0 + a.per_piece);
    const bool single0 = c0 == 0 && c1 > 0 && w.src < all;
    const bool single1 = c1 == w.chunks && c1 > c0 && w.src + (int64_t)w.chunks * 16 > all_end;
    if (single0 || single1) {
      const int slot = (lane < E && single0 ? 0 : w.chunks - 1) * E + (lane & (E - 1));
      if (lane < 2 * E && (lane < E ? single0 : single1) && (unsigned)(slot - w.skew) < (unsigned)w.n) {
        if constexpr (BF16)
          reinterpret_cast<uint16_t*>(image)[slot] = reinterpret_cast<const uint16_t*>(w.src)[slot];
        else
          reinterpret_cast<uint32_t*>(image)[slot] = reinterpret_cast<const uint32_t*>(w.src)[slot];
      }
      fence_proxy_async_smem();                // before the copy that comes here next
      __syncwarp();
      c0 += single0;
      c1 = max(c0, c1 - (single1 && (c1 > c0)));
    }
    if (lane == 0 && waited) {
      ++started;
      mbar_expect_tx(full + p, (c1 - c0) * 16);
      if (c1 > c0) copy_in(image + c0, w.src + (int64_t)c0 * 16, (c1 - c0) * 16, full + p);
    }
  };
  // Runs f(c, values of chunks c, c + kThreads, ...) over this thread's chunks of piece p,
  // several at a time, whole warps together (chunks past the piece: -inf).  The share's
  // first and last chunk, some of whose slots may not be the row's, are left out: the last
  // warp looks after them.
  auto each = [&](const View& w, int p, auto f) {
    constexpr int B = BF16 ? 2 : 4;
    const int c1 = min(w.chunks - 1, (p + 1) * a.per_piece);
    int c = max(1, p * a.per_piece) + warp * 32;            // lane 0's
#pragma unroll 1
    for (; c + 31 + (B - 1) * kThreads < c1; c += B * kThreads) {
      uint4 u[B];
      float v[B][E];
#pragma unroll
      for (int b = 0; b < B; ++b) u[b] = image[c + lane + b * kThreads];
#pragma unroll
      for (int b = 0; b < B; ++b) unpack<BF16>(u[b], v[b]);
      f(c, v);
    }
    constexpr uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll 1
    for (; c < c1; c += kThreads) {
      uint4 u = make_uint4(none, none, none, none);
      if (c + lane < c1) u = image[c + lane];
      float v[1][E];
      unpack<BF16>(u, v[0]);
      f(c, v);
    }
  };
  // The slot of the first or last chunk that a lane of the last warp looks after, -1 if
  // none: E lanes for each.
  auto edge_slot = [&](const View& w) {
    const int c = lane < E ? 0 : w.chunks - 1, slot = c * E + (lane & (E - 1));
    const bool mine = lane < 2 * E && w.chunks > 0 && (lane < E || c > 0);
    return mine && (unsigned)(slot - w.skew) < (unsigned)w.n ? slot : -1;
  };
  // The largest logit of this thread's chunks, as they arrive.
  auto largest = [&](const View& w, uint32_t parity) {
    float m = -INFINITY;
    if (warp == kWarps) {
      for (int p = 0; p < kPieces; ++p) wait_for(full + p, parity);
      const int slot = edge_slot(w);
      return slot >= 0 ? at<BF16>(image, slot) : m;
    }
#pragma unroll 1
    for (int p = 0; p < kPieces; ++p) {
      wait_for(full + p, parity);
      each(w, p, [&](int, auto& v) {
        constexpr int B = sizeof(v) / sizeof(v[0]);
        float h[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          h[b] = fmaxf(v[b][0], v[b][1]);
#pragma unroll
          for (int e = 2; e < E; e += 2) h[b] = fmaxf(h[b], fmaxf(v[b][e], v[b][e + 1]));
        }
#pragma unroll
        for (int b = 0; b < B; ++b) m = fmaxf(m, h[b]);
      });
    }
    return m;
  };
  // From the threads' maxima the CTA's (in warp 0), and the bound under its candidates.
  auto bound_of = [&](float mine) {
    maxima[warp][lane] = mine;
    __syncthreads();
    float m = -INFINITY;
    if (warp == 0) {
#pragma unroll
      for (int q = 0; q <= kWarps; ++q) m = fmaxf(m, maxima[q][lane]);
      int ahead = 0;                           // lanes whose maximum comes before this one's
      if (a.top > 1) {
#pragma unroll
        for (int o = 0; o < 32; ++o) {
          const float y = __shfl_sync(0xffffffffu, m, o);
          ahead += (y > m) | ((y == m) & (o < lane));
        }
        if (ahead == a.top - 1) bound = m;
      }
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (a.top == 1 && lane == 0) bound = m;
    }
    return m;
  };

  // The row before, which the last warp finishes once the cluster has met again.
  int64_t last_row = -1;
  int last_token = -1;
  float last_m = 0.f, last_dt = 0.f;
  auto finish = [&](int slot) {
    float l = 0.f, s = 0.f;
    int before = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r < ctas) {
        const float4 f = found[slot][r];
        l += f.x;
        s += f.y;
        before += __float_as_int(f.z);
      }
    }
    const bool bad = !(l < INFINITY);          // NaN: one among the logits, or +inf less itself
    const bool given = last_token >= 0 && last_token < a.vocab;
    const float log_l = l > 0.f ? logf(l) : 0.f;
    if (lane == 0) {
      if (bad) raise_flag(a.status, LQ_DEV_NONFINITE);
      else if (last_m == -INFINITY) raise_flag(a.status, LQ_DEV_RANGE);
      if (last_token >= a.vocab) raise_flag(a.status, LQ_DEV_RANGE);
      a.logprobs[last_row] = bad ? NAN : given ? last_dt - log_l : 0.f;
      if (a.entropy != nullptr) a.entropy[last_row] = bad ? NAN : l > 0.f ? log_l - s / l : 0.f;
      if (a.ranks != nullptr) a.ranks[last_row] = bad || !given ? -1 : before;
    }
    for (int i = lane; i < a.top * ctas; i += 32) {
      // an alternative's place: how many of every CTA's, which are in order, come before it
      const u64 key = keys[slot][i];
      int ahead[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) ahead[r] = 0;
#pragma unroll
      for (int step = kMaxTop; step; step >>= 1)
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const int to = ahead[r] + step;
          if (r < ctas && to <= a.top && keys[slot][r * a.top + to - 1] > key) ahead[r] = to;
        }
      int place = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) place += ahead[r];
      if (bad ? i < a.top : key != 0 && place < a.top) {
        const int64_t to = last_row * a.top + (bad ? i : place);
        a.top_tokens[to] = bad ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)key);
        a.top_logprobs[to] = bad ? NAN : value_of(key) - log_l;
      }
    }
  };

  int use = 0;                                 // copies of whole segments so far
  if (segments == 1 && warp == kWarps) {
    const View w = view(row0, 0);
    for (int p = 0; p < kPieces; ++p) start(w, p);
  }
  if (ctas > 1) cluster_wait();
  int it = 0;
  auto logit_of = [&](int64_t row, int32_t token) {
    return token >= 0 && token < a.vocab ? at<BF16>(all + row * a.ld * kSize, token) : 0.f;
  };
  int32_t next_token = a.tokens[row0];
  float next_xt = logit_of(row0, next_token);
  for (int64_t row = row0; row < a.rows; row += clusters, ++it) {
    // the next row's token and logit are fetched under this row's work
    const int32_t token = next_token;
    const bool given = token >= 0 && token < a.vocab;
    const float xt = next_xt;
    const bool more = row + clusters < a.rows;
    if (more) next_token = a.tokens[row + clusters];
    // segment g, once everyone has read what was there; its phase
    View w = view(row, 0);
    auto load = [&](int g) {
      if (segments > 1) {
        __syncthreads();
        w = view(row, g);
        if (warp == kWarps)
          for (int p = 0; p < kPieces; ++p) start(w, p);
      }
      return (uint32_t)use++ & 1u;
    };
    // the row's maximum
    uint32_t parity = 0;
    float mine = -INFINITY;
    for (int g = 0; g < segments; ++g) {
      parity = load(g);
      mine = fmaxf(mine, largest(w, parity));
    }
    float m = bound_of(mine);
    if (ctas > 1) {
      if (warp == 0 && lane < ctas) put(peer(&tops[it & 1][rank], lane), m);
      cluster_arrive();
      cluster_wait();
    } else {
      if (tid == 0) tops[it & 1][0] = m;
      __syncthreads();
    }
    m = tops[it & 1][0];
#pragma unroll
    for (int r = 1; r < kMaxCluster; ++r)
      if (r < ctas) m = fmaxf(m, tops[it & 1][r]);
    if (warp == kWarps && it > 0 && (it - 1) % ctas == rank) finish((it - 1) & 1);
    const float zero = m == -INFINITY ? 0.f : m;
    const float dt = given ? xt - zero : kHuge;
    // Counting by step_of needs differences of 2^-127 or more, and tokens above the least
    // number: other rows' ranks are counted one by one.
    const bool odd_rank = given && (fabsf(zero) < 8.4703295e-22f || dt <= -kHuge);         // 2^-70

    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, s2[2] = {l2[0], l2[0]};
    float2 n2[2] = {l2[0], l2[0]};             // elements before the token
    float before = 0.f;                        // and what they are off by
    int have = 0, odd = 0;                     // alternatives found in earlier segments
    for (int g = 0; g < segments; ++g) {
      if (segments > 1) {                      // the share again
        parity = load(g);
        bound_of(largest(w, parity));
      }
      if (g == 0 && more) next_xt = logit_of(row + clusters, next_token);
      if (segments > 1) __syncthreads();       // the bound
      const float least = a.top > 0 ? bound - zero : INFINITY;
      // the token's slot of the image, or one before or behind all
      const int64_t far = token - w.base + w.skew;
      const int slot = far < 0 ? -1 : far < w.chunks * E ? (int)far : w.chunks * E;
      auto note = [&](float d, int at_slot) {  // a candidate
        const int to = atomicAdd(&listed, 1);
        if (to < kRoom) list[to] = key_of(d, (uint32_t)(w.base + at_slot - w.skew));
      };
      if (warp == kWarps) {
        // The chunks at the ends, a slot per lane; and the rank by whole chunks before and
        // behind the token, which the workers count, is not that of the slots of the chunk
        // that holds it: they are counted one by one, what the workers count taken off.
        const int edge = edge_slot(w), c = slot / E;
        if (edge >= 0) {
          const float d = at<BF16>(image, edge) - zero, dc = max_nan(d, -kHuge), y = ex2(dc * 1.4426950408889634f);
          l2[0].x += y;
          s2[0].x = fmaf(y, dc, s2[0].x);
          before += (float)((d > dt) | ((d == dt) & (edge < slot)));
          if (d >= least) note(d, edge);
        }
        if (slot >= 0 && c > 0 && c < w.chunks - 1 && lane < E) {
          const float d = at<BF16>(image, c * E + lane) - zero;
          before += (float)((d > dt) | ((d == dt) & (c * E + lane < slot)));
          before -= step_of(max_nan(d, -kHuge) - dt, c * E < slot ? 1.f : 0.f);
        }
        __syncwarp();
        arrive_listed();
        if (segments == 1 && more) {
          const View next = view(row + clusters, 0);
          for (int p = 0; p < kPieces; ++p) {
            wait_for(empty + p, (uint32_t)it & 1u);         // all have read the piece
            start(next, p);
          }
        }
        continue;
      }
      const float2 shift = make_float2(-zero, -zero), token_at = make_float2(-dt, -dt);
      const float2 log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll 1
      for (int p = 0; p < kPieces; ++p) {
        const int c1 = min(w.chunks - 1, (p + 1) * a.per_piece);
        each(w, p, [&](int c, auto& v) {
          constexpr int B = sizeof(v) / sizeof(v[0]);
          float high = -INFINITY;
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const float equal = (c + lane + b * kThreads) * E < slot ? 1.f : 0.f;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              float2 d = add2(make_float2(v[b][e], v[b][e + 1]), shift);
              high = fmaxf(high, fmaxf(d.x, d.y));
              d = make_float2(max_nan(d.x, -kHuge), max_nan(d.y, -kHuge));   // -inf: no term, not 0 times itself
              const float2 over = add2(d, token_at);
              n2[b & 1] = add2(n2[b & 1], make_float2(step_of(over.x, equal), step_of(over.y, equal)));
              float2 y = mul2(d, log2e);
              y = make_float2(ex2(y.x), ex2(y.y));
              l2[b & 1] = add2(l2[b & 1], y);
              s2[b & 1] = fma2(y, d, s2[b & 1]);
            }
          }
          // lanes with candidates, seldom: the warp looks at one's slots together
          for (uint32_t hit = __ballot_sync(0xffffffffu, high >= least); hit; hit &= hit - 1) {
            const int chunk = c + __ffs(hit) - 1 + lane / E * kThreads, to = chunk * E + lane % E;
            if (lane < B * E && chunk < c1) {
              const float d = at<BF16>(image, to) - zero;
              if (d >= least) note(d, to);
            }
          }
        });
        __syncwarp();
        if (lane == 0 && waited) arrive(empty + p);
      }
      if (odd_rank) {
        const uint8_t* src = all + (row * a.ld + w.base) * kSize;
        for (int j = tid; j < w.n; j += kThreads) {
          const float d = at<BF16>(src, j) - zero;
          odd += (d > dt) | ((d == dt) & (w.base + j < token));
        }
      }
      sync_listed();
      if (a.top > 0) {
        const int count = listed, k = (int)min((int64_t)a.top, (int64_t)have + w.n);
        if (count <= kByRank) {
          if (warp <= (count - 1) >> 5) {
            const u64 key = tid < count ? list[tid] : 0;
            int ahead = 0;
#pragma unroll 8
            for (int i = 0; i < count; ++i) ahead += list[i] > key;
            if (tid < count && ahead < k) best[ahead] = key;
          }
        } else {
          // one after the other: the largest key below the last, of the list or, where it
          // has overflowed, of the earlier segments' and the whole segment
          u64 last = ~0ull, taken = 0;
          const int old = count <= kRoom ? count : have;
          const uint8_t* src = all + (row * a.ld + w.base) * kSize;
          for (int i = 0; i < k; ++i) {
            u64 top = 0;
            for (int j = tid; j < old; j += kThreads)
              if (list[j] < last && list[j] > top) top = list[j];
            if (count > kRoom)
              for (int j = tid; j < w.n; j += kThreads) {
                const u64 key = key_of(at<BF16>(src, j) - zero, (uint32_t)(w.base + j));
                if (key < last && key > top) top = key;
              }
            for (int o = 16; o; o >>= 1) {
              const u64 y = __shfl_xor_sync(0xffffffffu, top, o);
              top = y > top ? y : top;
            }
            if (lane == 0) round_best[warp] = top;
            sync_workers();
            for (int q = 0; q < kWarps; ++q) top = round_best[q] > top ? round_best[q] : top;
            sync_workers();
            last = top;
            if (tid == i) taken = top;
          }
          if (tid < k) best[tid] = taken;
        }
        have = k;
        sync_workers();
        // the next list begins with these, if it is one of the same row
        const int keep = g + 1 < segments ? have : 0;
        if (tid < keep) list[tid] = best[tid];
        if (tid == 0) listed = keep;
      }
    }

    // sums over the CTA in a fixed order, to the one of the cluster whose turn it is
    {
      // (whole numbers: at most 2^20 of a thread's, and 2^24 in all)
      int n = (int)((n2[0].x + n2[0].y) + (n2[1].x + n2[1].y) + before);
      if (odd_rank) n = odd;
      float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y), s = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
      n = __reduce_add_sync(0xffffffffu, n);
      for (int o = 16; o; o >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      if (lane == 0) {
        sums[warp][0] = l;
        sums[warp][1] = s;
        counts[warp] = n;
      }
      __syncthreads();
    }
    if (warp == 0) {
      float l = lane <= kWarps ? sums[lane][0] : 0.f, s = lane <= kWarps ? sums[lane][1] : 0.f;
      const int n = __reduce_add_sync(0xffffffffu, lane <= kWarps ? counts[lane] : 0);
      for (int o = 16; o; o >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      const int turn = it % ctas;
      const u64 key = lane < have ? best[lane] : 0;
      if (ctas > 1) {
        if (lane == 0) {
          const uint32_t to = peer(&found[it & 1][rank], turn);
          put(to, l);
          put(to + 4, s);
          put(to + 8, __int_as_float(n));
        }
        if (lane < a.top) put(peer(&keys[it & 1][rank * a.top + lane], turn), key);
      } else {
        if (lane == 0) found[it & 1][0] = make_float4(l, s, __int_as_float(n), 0.f);
        if (lane < a.top) keys[it & 1][lane] = key;
      }
    }
    last_row = row;
    last_token = token;
    last_m = m;
    last_dt = dt;
  }
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == kWarps && it > 0 && (it - 1) % ctas == rank) finish((it - 1) & 1);
  if (warp == kWarps && lane == 0 && timeout) {
    // let the last copy of each piece land before the CTA ends
    for (int p = 0; p < kPieces; ++p) {
      const int copies = (started + kPieces - 1 - p) / kPieces;
      if (copies > 0) mbar_wait_bounded(full + p, (uint32_t)(copies - 1) & 1u, kWaitCycles / 8);
    }
  }
  if (tid == 0 && timeout) raise_flag(a.status, LQ_DEV_TIMEOUT);
}

// The kernels may use all of the shared memory that a share can take.
bool prepare() {
  for (auto kernel : {score_kernel<true>, score_kernel<false>})
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
  return true;
}

// Clusters of so many CTAs that the current device holds at once, one CTA per SM (fewer
// than the SMs allow: a cluster lies within one of their groups); 0 on an error.
int most_clusters(int ctas) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];
  int device = 0, n = 0;
  if (cudaGetDevice(&device) == cudaSuccess && device < kDevices && (n = known[device][ctas].load()) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads + 32);
  cfg.dynamicSmemBytes = kMostBytes;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, score_kernel<true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (device < kDevices) known[device][ctas].store(n);
  return n;
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
  if (!score::prepare()) return LQ_ERR_CUDA;
  score::Args a;
  a.x = logits_dev; a.ld = ld; a.rows = rows; a.vocab = vocab; a.tokens = tokens_dev; a.logprobs = logprobs_dev;
  a.entropy = entropy_dev; a.ranks = ranks_dev; a.top = top; a.top_tokens = top_tokens_dev;
  a.top_logprobs = top_logprobs_dev; a.status = dev_status_dev;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  score::Plan plan;
  if (!score::make_plan(rows, vocab, dtype == LQ_BF16 ? 2 : 4,
                        [&](int c) { return c == 1 ? sms : score::most_clusters(c); }, &plan))
    return LQ_ERR_CUDA;
  static_cast<score::Division&>(a) = plan.d;
  const auto kernel = dtype == LQ_BF16 ? score::score_kernel<true> : score::score_kernel<false>;
  return serve::launch(kernel, (unsigned)(plan.clusters * plan.d.cluster), score::kThreads + 32, plan.d.chunks * 16, stream,
                       a, (unsigned)plan.d.cluster);
}
