// Block tables and slot maps of a paged KV cache, built on the GPU from the
// requests' lengths.
//
// Request i holds c_i cached tokens and brings n_i new ones; with blocks of bs
// tokens it has have_i = ceil(c_i / bs) blocks and needs need_i = ceil((c_i +
// n_i) / bs).  Its new blocks are the free-list entries f_i .. f_i + need_i -
// have_i - 1, f the exclusive prefix sum of need - have over the requests, and
// new token t of request i (the batch's tokens are numbered request after
// request, cu the prefix sum of n) has position p = c_i + t - cu_i and slot
// table[i][p / bs] * bs + p % bs.
//
// One launch.  The prefix sums are the only coupling between requests, and
// they need just the 8 bytes of lengths per request, so every CTA computes
// them for itself in shared memory instead of waiting for another launch, and
// then writes its share of the table rows (a warp per row) and of the tokens
// (four to a thread; their requests by search in cu).  A block that
// another CTA writes in this launch is never read back from the table: it is
// taken from the free list.
#include "lq_host.h"
#include "lq_device.cuh"
#include "lq_serve.cuh"

namespace lq {
namespace plan {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Args {
  const int32_t* cached;
  const int32_t* fresh;      // new tokens per request
  int batch, log2_bs;
  const int32_t* free_blocks;
  int64_t num_free;
  int32_t* table;
  int64_t ldt;
  int width;
  int32_t* cu;               // [batch + 1]
  int32_t* kv_lens;          // [batch]
  int64_t* slots;            // [max_tokens]
  int32_t* positions;        // [max_tokens]
  int64_t max_tokens;
  int32_t* used;
  int32_t* status;
};

__device__ __forceinline__ int clip_len(int32_t v) { return v < 0 ? 0 : v; }

__global__ void __launch_bounds__(kThreads) plan_kernel(Args a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* cu = plan_smem;                     // [batch + 1]
  int32_t* fs = plan_smem + a.batch + 1;       // [batch + 1]: first free-list entry
  __shared__ long long wsum[kWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs1 = (1 << a.log2_bs) - 1;
  pdl_wait();
  pdl_launch();

  // prefix sums: each thread owns a run of requests
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int i0 = min(a.batch, tid * per), i1 = min(a.batch, i0 + per);
  long long sn = 0, sb = 0;
  bool bad = false;
  for (int i = i0; i < i1; ++i) {
    const int32_t rc = a.cached[i], rn = a.fresh[i];
    const long long c = clip_len(rc), n = clip_len(rn);
    const long long need = (c + n + bs1) >> a.log2_bs;
    bad |= rc < 0 || rn < 0 || c + n > INT32_MAX || need > a.width;
    sn += n;
    sb += need - ((c + bs1) >> a.log2_bs);
  }
  long long en = sn, eb = sb;                  // inclusive over the warp
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, en, o), y = __shfl_up_sync(0xffffffffu, eb, o);
    if (lane >= o) { en += x; eb += y; }
  }
  if (lane == 31) { wsum[warp][0] = en; wsum[warp][1] = eb; }
  __syncthreads();
  long long tn = 0, tb = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) { en += tn; eb += tb; }
    tn += wsum[w][0];
    tb += wsum[w][1];
  }
  en -= sn;
  eb -= sb;
  auto clip = [](long long v) { return (int32_t)(v < INT32_MAX ? v : INT32_MAX); };
  for (int i = i0; i < i1; ++i) {
    const long long c = clip_len(a.cached[i]), n = clip_len(a.fresh[i]);
    cu[i] = clip(en);
    fs[i] = clip(eb);
    if (blockIdx.x == 0) {
      a.cu[i] = clip(en);
      a.kv_lens[i] = clip(c + n);
    }
    en += n;
    eb += ((c + n + bs1) >> a.log2_bs) - ((c + bs1) >> a.log2_bs);
  }
  if (tid == 0) {
    cu[a.batch] = clip(tn);
    if (blockIdx.x == 0) {
      a.cu[a.batch] = clip(tn);
      a.used[0] = clip(tb);
      bad |= tn > a.max_tokens || tb > a.num_free;
    }
  }
  if (blockIdx.x == 0 && bad) raise_flag(a.status, LQ_DEV_RANGE);
  __syncthreads();

  // table rows: blocks held stay, new ones come from the free list, -1 after
  for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < a.batch; i += (int64_t)gridDim.x * kWarps) {
    const long long c = clip_len(a.cached[i]), n = clip_len(a.fresh[i]);
    const long long have = (c + bs1) >> a.log2_bs, need = (c + n + bs1) >> a.log2_bs;
    int32_t* row = a.table + i * a.ldt;
    for (long long j = have + lane; j < a.width; j += 32) {
      const long long f = (long long)fs[i] + j - have;
      row[j] = (j < need && f < a.num_free) ? a.free_blocks[f] : -1;
    }
  }

  // tokens, 128 neighbouring ones per warp and turn: the first of a lane's four
  // finds its request by binary search, the others go on from there
  const int64_t total = min((long long)cu[a.batch], (long long)a.max_tokens);
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * 128; t0 < a.max_tokens;
       t0 += (int64_t)gridDim.x * kWarps * 128) {
    int lo = 0, hi = a.batch;                  // last i with cu[i] <= t: empty requests are skipped
    if (t0 + lane < total) {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t0 + lane) lo = mid; else hi = mid;
      }
    }
    long long slot[4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      slot[i] = -1;
      pos[i] = 0;
      if (t < total) {
        while (cu[lo + 1] <= t) ++lo;          // (cu[batch] > t)
        const long long c = clip_len(a.cached[lo]);
        const long long p = c + t - cu[lo];
        const long long have = (c + bs1) >> a.log2_bs, j = p >> a.log2_bs;
        int32_t blk = -1;
        if (j < a.width) {
          const long long f = (long long)fs[lo] + j - have;
          if (j < have) blk = a.table[(int64_t)lo * a.ldt + j];
          else if (f < a.num_free) blk = a.free_blocks[f];
        }
        if (blk >= 0) slot[i] = ((long long)blk << a.log2_bs) + (p & bs1);
        pos[i] = (int)(p < INT32_MAX ? p : INT32_MAX);
      }
    }
    // (stored last: the four tokens' loads need not wait for each other's stores)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (t >= a.max_tokens) break;
      a.slots[t] = slot[i];
      a.positions[t] = pos[i];
    }
  }
}

}  // namespace plan
}  // namespace lq

using namespace lq;

extern "C" lq_status lq_kv_plan(const int32_t* cached_lens_dev, const int32_t* new_lens_dev, int batch, int block_size,
                                const int32_t* free_blocks_dev, int64_t num_free, int32_t* block_table_dev,
                                int64_t table_stride, int table_width, int32_t* cu_new_dev, int32_t* kv_lens_dev,
                                int64_t* slots_dev, int32_t* positions_dev, int64_t max_tokens, int32_t* used_dev,
                                int32_t* dev_status_dev, void* stream) {
  LQ_NVTX_RANGE("lq_kv_plan");
  if (!serve::valid_block_size(block_size)) return LQ_ERR_UNSUPPORTED;
  if (batch < 0 || batch > LQ_MAX_REQUESTS || table_width < 0 || table_stride < table_width || num_free < 0 ||
      max_tokens < 0 || max_tokens > INT32_MAX)
    return LQ_ERR_SHAPE;
  if (cu_new_dev == nullptr || used_dev == nullptr || !aligned4(cu_new_dev) || !aligned4(used_dev) ||
      !aligned4(dev_status_dev))
    return LQ_ERR_ARG;
  if (batch > 0 && (cached_lens_dev == nullptr || new_lens_dev == nullptr || kv_lens_dev == nullptr ||
                    !aligned4(cached_lens_dev) || !aligned4(new_lens_dev) || !aligned4(kv_lens_dev)))
    return LQ_ERR_ARG;
  if (batch > 0 && table_width > 0 && (block_table_dev == nullptr || !aligned4(block_table_dev))) return LQ_ERR_ARG;
  if (num_free > 0 && (free_blocks_dev == nullptr || !aligned4(free_blocks_dev))) return LQ_ERR_ARG;
  if (max_tokens > 0 && (slots_dev == nullptr || positions_dev == nullptr || !serve::aligned8(slots_dev) ||
                         !aligned4(positions_dev)))
    return LQ_ERR_ARG;
  plan::Args a;
  a.cached = cached_lens_dev; a.fresh = new_lens_dev; a.batch = batch; a.log2_bs = serve::log2_of(block_size);
  a.free_blocks = free_blocks_dev; a.num_free = num_free;
  a.table = block_table_dev; a.ldt = table_stride; a.width = table_width;
  a.cu = cu_new_dev; a.kv_lens = kv_lens_dev; a.slots = slots_dev; a.positions = positions_dev;
  a.max_tokens = max_tokens; a.used = used_dev; a.status = dev_status_dev;
  const int sms = device_sm_count();
  if (sms <= 0) return LQ_ERR_CUDA;
  const size_t smem = (size_t)(2 * (size_t)batch + 2) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    if (cudaFuncSetAttribute(plan::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return LQ_ERR_CUDA;
    }
  }
  // a CTA per kWarps table rows or kWarps x 128 tokens, at most two per SM
  int64_t grid = (batch + plan::kWarps - 1) / plan::kWarps;
  const int64_t by_tokens = (max_tokens + plan::kWarps * 128 - 1) / (plan::kWarps * 128);
  if (by_tokens > grid) grid = by_tokens;
  if (grid > 2 * (int64_t)sms) grid = 2 * (int64_t)sms;
  if (grid < 1) grid = 1;
  return serve::launch(plan::plan_kernel, (unsigned)grid, plan::kThreads, smem, stream, a);
}
